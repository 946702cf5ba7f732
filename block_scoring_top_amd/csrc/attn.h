// attn.h - what the attention kernels share: arguments, softmax state, the
// joining of splits.
#pragma once

#include <type_traits>
#include <utility>

#include "kernels.h"
#include "kv4.h"

namespace bs {

// How far (in log2) a score may exceed the running maximum before that moves.
constexpr float kSlack = 8.f;
// Running maxima past this are exact to no more than 2^-4 (in log2), and more
// than that lies between a score's product with the scale as the maximum has it
// and as an fma holds it: weights are then of the rounded products.  Of the
// others they left fp16's range from scores of 2^26 on, and FP32's from 2^31.
constexpr float kHugeScore = 0x1p20f;
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

// The maximum that passes NaN on (v_maximum3_f32).  fmaxf would first have to
// quieten each operand, one instruction apiece.
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Maximum / sum over the four 16-lane rows of a wave, per lane of a row.
__device__ __forceinline__ float rows_max(float x) {
  const uint32_t u = __float_as_uint(x);
  auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t v = __float_as_uint(max_nan(__uint_as_float(a[0]), __uint_as_float(a[1])));
  auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max_nan(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float rows_sum(float x) {
  const uint32_t u = __float_as_uint(x);
  auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t v = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// A row's sums of weights, relative to its running maximum and raised by
// 2^T::kRaise, which the output's division cancels: x of the weights in
// FP32 (for lse), y of the weights as rounded for their product with V.  The
// output is divided by y: the rounding of a weight that dominates its row then
// cancels.  Over 52 drawn calls the outputs' error against 64 bits is 1.16
// times that of an FP32 form rounded once (at most 1.33); with x in y's place
// it was 1.19 (1.42), for 2% less time in the prefill kernel.
typedef f32x2_t Sums;

// sums += the rounding of 8 weights packed in p.
template <class T>
__device__ __forceinline__ float add_rounded(const u32x4_t& p, float sum) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = T::dot2(p[i], T::kOne * 0x00010001u, sum);
  return sum;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// A maximum to subtract: 0 in place of -inf, so that -inf scores give 0 and
// not NaN.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }

// x * scale rounded, whatever it is used in.
__device__ __forceinline__ float rounded_product(float x, float scale) {
  float y = x * scale;
  asm("" : "+v"(y));
  return y;
}

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

// Marks for the infinities and NaN of a pair, 0 for other values: 1 for +inf,
// 64 for -inf, 65 for NaN, exact in both 16-bit types.  This and what follows
// are written without comparisons: their lane masks, dozens of them at once,
// would not fit the scalar registers.
template <class T>
__device__ __forceinline__ uint32_t nonfinite_marks(uint32_t x) {
  constexpr uint32_t mant = 0x7FFF7FFFu & ~T::kExpMask, both = 0x00010001u;
  const uint32_t nan = spread_halves(((x & mant) + 0x7FFF7FFFu) & 0x80008000u);
  return spread_halves(nonfinite_pair<T>(x)) &
         bit_select(nan, T::k65 * both, bit_select(spread_halves(x), T::k64 * both, T::kOne * both));
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

// Where part i of n items in `parts` parts begins, the sizes differing by one at
// most (32-bit: a 64-bit division is a hundred scalar instructions).
__device__ __forceinline__ int part_start(uint32_t n, uint32_t parts, uint32_t i) {
  const uint32_t q = n / parts, r = n - q * parts;
  return (int)(q * i + min(i, r));
}

// The LDS address behind a generic pointer into shared memory.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)p;
}

__device__ __forceinline__ void wave_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

// A workspace region that splits exchange results through: relaxed
// device-scope accesses only (performed at the device's coherence point, not
// in an XCD's L2), so no cache write-back is needed.
struct SplitBuffer {
  __amdgpu_buffer_rsrc_t rs;
  __device__ __forceinline__ SplitBuffer(float* p, uint32_t bytes)
      : rs(__builtin_amdgcn_make_buffer_rsrc(p, (short)0, bytes, 0x00020000)) {}
  static constexpr int kSc1 = 16;
  // Past every workspace (32 MiB): a load from there is refused by the
  // buffer's bounds and gives zeros.
  static constexpr uint32_t kNowhere = 1u << 30;
  __device__ __forceinline__ void store4(uint32_t off, const f32x4_t& v) const {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rs, off, 0, kSc1);
  }
  __device__ __forceinline__ f32x4_t load4(uint32_t off) const {
    return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, kSc1));
  }
};

// Called by every lane of a workgroup whose partial result is stored: true in
// the workgroup that is the last of its group's nsplit to arrive (its counter
// is then zero again).  `arrived` is in LDS.
__device__ __forceinline__ bool last_of_group(uint32_t* counters, uint32_t group, int nsplit, int tid, uint32_t& arrived) {
  __builtin_amdgcn_s_waitcnt(0);  // this lane's stores have been performed
  __syncthreads();
  if (tid == 0) {
    arrived = __hip_atomic_fetch_add(&counters[group], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (arrived == (uint32_t)nsplit - 1)
      __hip_atomic_store(&counters[group], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return arrived == (uint32_t)nsplit - 1;
}

// Joins the partial results of nsplit workgroups in split order.  A partial
// (step bytes) holds [cols][D] products, then [cols] (maximum, sums, 0).  A thread takes
// 4 channels of UNITS columns at a time, the loads of BATCH splits of each in
// flight together (past the last split: zeros, as a split read again with weight
// 0 might hold infinities; past the last column: its own again, not written).
template <int D, int THREADS, int UNITS, int BATCH, class F>
__device__ __forceinline__ void join_batches(const SplitBuffer& sb, uint32_t first, uint32_t step, int cols, int ncols,
                                             int nsplit, int tid, F write) {
  const int n = ncols * (D / 4);
  for (int u0 = tid; u0 < n; u0 += THREADS * UNITS) {
    uint32_t ml[UNITS], oo[UNITS];
    float mm[UNITS];
    Sums ll[UNITS];
    f32x4_t o[UNITS];
#pragma unroll
    for (int v = 0; v < UNITS; ++v) {
      const int u = u0 + v * THREADS < n ? u0 + v * THREADS : u0;
      const int cc = u / (D / 4), d = (u % (D / 4)) * 4;
      ml[v] = first + (cols * D + 4 * cc) * 4, oo[v] = first + (cc * D + d) * 4;
      mm[v] = -INFINITY, ll[v] = Sums{0.f, 0.f}, o[v] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    for (int i = 0; i < nsplit; i += BATCH) {
      f32x4_t x[UNITS][BATCH], y[UNITS][BATCH];
#pragma unroll
      for (int v = 0; v < UNITS; ++v)
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const bool there = i + k < nsplit;
          const uint32_t at = there ? (i + k) * step : SplitBuffer::kNowhere;
          x[v][k] = sb.load4(ml[v] + at), y[v][k] = sb.load4(oo[v] + at);
          x[v][k].x = there ? x[v][k].x : -INFINITY;
        }
#pragma unroll
      for (int v = 0; v < UNITS; ++v) {
        float nm = mm[v];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) nm = fmaxf(nm, x[v][k].x);
        const float nf = finite_max(nm), f = exp2_fast(mm[v] - nf);
        ll[v] *= f, o[v] *= f;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const float g = exp2_fast(x[v][k].x - nf);
          ll[v] += x[v][k].yz * g, o[v] += y[v][k] * g;
        }
        mm[v] = nm;
      }
    }
#pragma unroll
    for (int v = 0; v < UNITS; ++v) {
      const int u = u0 + v * THREADS;
      if (u < n) write(u / (D / 4), (u % (D / 4)) * 4, o[v], mm[v], ll[v]);
    }
  }
}

// A pass over the columns is a memory latency: 2 or 4 go at once where that many
// are needed and have few splits each.
template <int D, int THREADS, int COLS, class F>
__device__ __forceinline__ void join_splits(const SplitBuffer& sb, uint32_t first, uint32_t step, int ncols, int nsplit,
                                            int tid, F write) {
  constexpr int MOST = COLS * (D / 4) / THREADS;
  const bool passes = ncols * (D / 4) > THREADS;
  if (nsplit > 8) {
    join_batches<D, THREADS, 1, 16>(sb, first, step, COLS, ncols, nsplit, tid, write);
  } else if (MOST > 1 && passes) {
    if (MOST > 2 && nsplit <= 4)
      join_batches<D, THREADS, (MOST > 2 ? 4 : 1), 4>(sb, first, step, COLS, ncols, nsplit, tid, write);
    else
      join_batches<D, THREADS, (MOST > 1 ? 2 : 1), 8>(sb, first, step, COLS, ncols, nsplit, tid, write);
  } else if (nsplit > 4) {
    join_batches<D, THREADS, 1, 8>(sb, first, step, COLS, ncols, nsplit, tid, write);
  } else {
    join_batches<D, THREADS, 1, 4>(sb, first, step, COLS, ncols, nsplit, tid, write);
  }
}

// The natural logarithm of a row's sum of weights, -inf for an empty row: m is
// its maximum (log2), the sum relative to that and raised.
template <class T>
__device__ __forceinline__ float row_lse(float m, float sum) {
  return sum == 0.f ? -INFINITY : (m + (__builtin_amdgcn_logf(sum) - T::kRaise)) * kLn2;
}

// Stores 4 channels of a joined column and (with the first) its lse.
template <class T>
__device__ __forceinline__ void write_joined(typename T::elem* dst, int d, const f32x4_t& o, float m, const Sums& l, float* lse) {
  const float inv = l.y == 0.f ? 0.f : 1.f / l.y;
  *reinterpret_cast<u32x2_t*>(dst + d) = u32x2_t{T::pack(o.x * inv, o.y * inv), T::pack(o.z * inv, o.w * inv)};
  if (lse != nullptr && d == 0) *lse = row_lse<T>(m, l.x);
}

}  // namespace bs
