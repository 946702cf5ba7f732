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

// All ones in the 16-bit halves whose bit 15 is set.
__device__ __forceinline__ uint32_t spread_halves(uint32_t x) { return ((x >> 15) & 0x00010001u) * 0xFFFFu; }
// The bits of a where sel is set, of b elsewhere.
__device__ __forceinline__ uint32_t bit_select(uint32_t sel, uint32_t a, uint32_t b) { return (a & sel) | (b & ~sel); }
// All ones if bit i of x is set, else 0.
__device__ __forceinline__ uint32_t bit_mask(uint32_t x, int i) { return (uint32_t)__builtin_amdgcn_sbfe((int)x, i, 1); }

// A pair with infinities and NaN replaced by zeros (clean), and marks for
// them: 1 for +inf, 64 for -inf, 65 for NaN, exact in both 16-bit types.  This
// and what follows are written without comparisons: their lane masks, dozens
// of them at once, would not fit the scalar registers.
template <class T>
__device__ __forceinline__ void split_nonfinite(uint32_t x, uint32_t& clean, uint32_t& marks) {
  constexpr uint32_t mant = 0x7FFF7FFFu & ~T::kExpMask, both = 0x00010001u;
  const uint32_t bad = spread_halves(nonfinite_pair<T>(x));
  const uint32_t nan = spread_halves(((x & mant) + 0x7FFF7FFFu) & 0x80008000u);
  clean = x & ~bad;
  marks = bad & bit_select(nan, T::k65 * both, bit_select(spread_halves(x), T::k64 * both, T::kOne * both));
}

// What visible infinities and NaN add to a sum, from the sum of the marks of
// at most 32 keys: its 64s count -inf and NaN, the rest +inf and NaN.
__device__ __forceinline__ float nonfinite_term(float n) {
  const float minus = floorf(n * (1.f / 64)), plus = n - 64.f * minus;
  const uint32_t p = 0u - (uint32_t)(int)fminf(plus, 1.f), q = 0u - (uint32_t)(int)fminf(minus, 1.f);
  return __uint_as_float(p & 0x7F800000u) + __uint_as_float(q & 0xFF800000u);
}

// Bit k (0 .. 63) set where position p0 + k is seen by a row at position t.
__device__ __forceinline__ uint64_t visible_bits(int p0, int t, int window, int sinks) {
  auto below = [](int64_t n) -> uint64_t {  // bits 0 .. n-1
    const int c = (int)(n < 0 ? 0 : n > 64 ? 64 : n);
    return c == 0 ? 0 : ~0ull >> (64 - c);
  };
  return below((int64_t)t + 1 - p0) & (~below((int64_t)t - window + 1 - p0) | below((int64_t)sinks - p0));
}

__device__ __forceinline__ void wave_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace bs
