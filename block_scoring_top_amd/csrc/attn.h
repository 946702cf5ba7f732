// attn.h - what the attention kernels share: arguments, softmax state, the
// joining of splits.
#pragma once

#include <type_traits>
#include <utility>

#include "kernels.h"
#include "kv4.h"

namespace bs {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <class F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
// f(0) .. f(N-1) with the index a constant (conversion builtins take their
// byte selector as an immediate).
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>());
}

// Maximum / sum over the four 16-lane rows of a wave, per lane of a row.
__device__ __forceinline__ float rows_max(float x) {
  const uint32_t u = __float_as_uint(x);
  auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t v = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
  auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float rows_sum(float x) {
  const uint32_t u = __float_as_uint(x);
  auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t v = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// A maximum to subtract: 0 in place of -inf, so that -inf scores give 0 and
// not NaN.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }

// The 16-bit values of a pair of packed pairs, transposed: lo holds both low
// halves, hi both high halves.
__device__ __forceinline__ uint32_t pair_lo(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t pair_hi(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Nonzero if either 16-bit half of x is an infinity or a NaN: the exponent
// field of ones carries into the sign position.
template <class T>
__device__ __forceinline__ uint32_t nonfinite_pair(uint32_t x) {
  return ((x & T::kExpMask) + T::kExpLsb) & 0x80008000u;
}

// A pair with infinities and NaN replaced by zeros (clean), and 0/1 marks of
// the halves that are +inf or NaN (plus) and -inf or NaN (minus).
template <class T>
__device__ __forceinline__ void split_nonfinite(uint32_t x, uint32_t& clean, uint32_t& plus, uint32_t& minus) {
  clean = plus = minus = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t v = (x >> (16 * h)) & 0xFFFFu, mag = v & 0x7FFFu;
    if (mag < T::kInfBits) clean |= v << (16 * h);
    if (mag > T::kInfBits || v == T::kInfBits) plus |= T::kOne << (16 * h);
    if (mag > T::kInfBits || v == (T::kInfBits | 0x8000u)) minus |= T::kOne << (16 * h);
  }
}

// What visible infinities and NaN add to a sum: counts of +inf-or-NaN and of
// -inf-or-NaN terms.
__device__ __forceinline__ float nonfinite_term(float plus, float minus) {
  return plus > 0.f ? (minus > 0.f ? NAN : INFINITY) : (minus > 0.f ? -INFINITY : 0.f);
}

__device__ __forceinline__ void wave_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace bs
