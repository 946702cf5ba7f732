// kv8.hip - the 8-bit KV cache: rows quantised as they are written, and read
// back.
//
// Store.  A page's scale belongs to all its tokens, so the rows of a call that
// lie in one page are one workgroup's work, for one kv head: with m their largest
// finite magnitude (K and V apart),
//   e = the least with m <= 448 * 2^e;  a call that writes the page's first slot
//   sets the page's scale to 2^e, any other raises it to 2^e if it is below,
//   and then the codes of the page's other slots are rounded to the new scale;
//   code = x * 2^-e rounded to the nearest E4M3 value, ties to even.
// Load: code * scale.
//
// Streams without reuse: HBM bounds them at the prefill sizes and the launch at
// the decode ones.  A workgroup keeps its rows in registers between the maximum
// and the rounding, so they are read once: 2 * D lanes, half of them for K, 8
// channels of a row a lane and up to 8 rows each.  Which rows share a page is
// found from the slots: those of a page lie within 64 consecutive rows of the
// call, so the first of them looks at the 63 before it (it is the first) and at
// the 63 behind it (they are its mates).
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "kv8.h"

namespace bs {

namespace {

static_assert(kPage == 64, "a slot is a page times 64 and an offset");
constexpr int kSpan = 64;  // rows that a page's rows lie within: as many as a page has slots

// 8 channels as FP32 values.
template <class T>
struct Values {
  float v[8];
  __device__ __forceinline__ explicit Values(const Chunk<T>& x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, Bf16>::value) {
        v[2 * i] = __uint_as_float(x.v[i] << 16), v[2 * i + 1] = __uint_as_float(x.v[i] & 0xFFFF0000u);
      } else {
        const f16x2_t h = __builtin_bit_cast(f16x2_t, (uint32_t)x.v[i]);
        v[2 * i] = (float)h.x, v[2 * i + 1] = (float)h.y;
      }
    }
  }
};
template <>
struct Values<F32> {
  float v[8];
  __device__ __forceinline__ explicit Values(const Chunk<F32>& x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x.v[i];
  }
};

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kDppQuadXor1, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kDppQuadXor2, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kDppRowHalfMirror, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kDppRowMirror, 0xF, 0xF, false));
  return max(max(readlane(x, 0), readlane(x, 16)), max(readlane(x, 32), readlane(x, 48)));
}

}  // namespace

// S: rows of the call whose runs (rows of one page) a workgroup takes if they
// begin there, one run after the other: S rows a group, `groups` from group0 on.
//
// In a prompt's rows every fourth group of 16 begins a run.  Consecutive
// workgroups go to the 8 XCDs in turn, so groups 4 apart are neighbours in the
// grid: with the groups in order, two XCDs did all the work (8,192 rows x 8
// heads of 128: 31.5 us).
template <class T, int D, int S>
__global__ __launch_bounds__(2 * D) void kv8_store_kernel(const typename T::elem* __restrict__ k,
                                                          const typename T::elem* __restrict__ v, int64_t ld_k,
                                                          int64_t ld_v, const int32_t* __restrict__ slots,
                                                          int32_t num_tok, int32_t hkv, int32_t num_slots,
                                                          uint8_t* codes, float* scales, uint32_t group0, uint32_t groups) {
  constexpr int LANES = D / 8, ROWS = D / LANES, PASSES = kPage / ROWS;  // of a row; rows at a time
  static_assert(ROWS == 8 && PASSES == 8, "D lanes for K, D for V");
  constexpr int HALF_WAVES = D / 64;  // waves that work on K (V)
  __shared__ int32_t sl[kSpan - 1 + S + kSpan - 1];
  __shared__ int32_t mate_row[kSpan], mate_slot[kSpan];
  __shared__ uint32_t tops[2][HALF_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.y, which = wave / HALF_WAVES;
  const int r0 = tid % D / LANES, j = tid % LANES;
  uint32_t group = blockIdx.x;
  if constexpr (S == 16) {
    const uint32_t quarter = (groups + 3) / 4;
    group = group % quarter * 4 + group / quarter;
    if (group >= groups) return;
  }
  const int64_t first = ((int64_t)group0 + group) * S;
  const typename T::elem* src = (which ? v : k) + h * D + j * 8;
  const int64_t ld = which ? ld_v : ld_k;

  // The slots around; -1 for those that are none.
  for (int i = tid; i < kSpan - 1 + S + kSpan - 1; i += 2 * D) {
    const int64_t t = first - (kSpan - 1) + i;
    const int32_t s = t >= 0 && t < num_tok ? slots[t] : -1;
    sl[i] = s >= 0 && s < num_slots ? s : -1;
  }
  __syncthreads();
  // Which of the S rows begin a run.
  uint64_t begins;
  if constexpr (S == 1) {
    const int s = sl[kSpan - 1];
    const int x = sl[lane < kSpan - 1 ? lane : 0];
    begins = s >= 0 && ballot(x >= 0 && x >> 6 == s >> 6) == 0 ? 1 : 0;
  } else {
    static_assert(S == 16, "four lanes a row, 16 of the 63 rows before it each");
    const int r = lane & 15, s = sl[kSpan - 1 + r];
    bool seen = s < 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int back = (lane >> 4) * 16 + i + 1;
      const int x = sl[back < kSpan ? kSpan - 1 + r - back : kSpan - 2 + r];
      seen |= x >= 0 && x >> 6 == s >> 6;
    }
    const uint64_t b = ballot(seen);
    begins = ~(b | b >> 16 | b >> 32 | b >> 48) & 0xFFFFu;
  }
  for (; begins != 0; begins &= begins - 1) {
    const int at = kSpan - 1 + __builtin_ctzll(begins);
    const int page = __builtin_amdgcn_readfirstlane(sl[at]) >> 6;
    // The run's rows, in order (every wave for itself; wave 0 notes them down).
    const int s = sl[at + lane];
    const bool mine = s >= 0 && s >> 6 == page;
    const uint64_t mask = ballot(mine);
    const int n = __popcll(mask), passes = (n + ROWS - 1) / ROWS;
    const bool anew = ballot(mine && (s & 63) == 0) != 0;
    if (wave == 0 && mine) {
      const int m = lanes_below(mask);
      mate_row[m] = at - (kSpan - 1) + lane, mate_slot[m] = s & 63;
    }
    float* const scale_at = scales + ((int64_t)page * hkv + h) * 2 + which;
    const float was = *scale_at;
    __syncthreads();

    auto run = [&](auto passes_c) {
      constexpr int P = decltype(passes_c)::value;
      // Lanes past the last row take it again.
      Chunk<T> x[P];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (i < passes) x[i].load(src + (first + mate_row[min(i * ROWS + r0, n - 1)]) * ld);
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (i < passes) top = max(top, x[i].top());
      // Infinities and NaN are left out of the maximum, in a second look if there are any.
      bool careful = false;
      if (ballot(top >= 0x7F800000u)) {
        careful = true, top = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (i >= passes) continue;
          const Values<T> y(x[i]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint32_t u = __float_as_uint(y.v[c]) & 0x7FFFFFFFu;
            top = max(top, u < 0x7F800000u ? u : 0u);
          }
        }
      }
      top = wave_max_u32(top);
      if (lane == 0) tops[which][wave % HALF_WAVES] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < HALF_WAVES; ++w) top = max(top, tops[which][w]);
      int e = kv8_exponent(top);
      const int old = min(max((int)(__float_as_uint(was) >> 23), kExpMin8), kExpMax8);
      const bool raised = !anew && e > old;
      if (!anew) e = max(e, old);
      const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
      careful = careful || e == kExpMax8;  // values past 448 scales

      uint8_t* const page_codes = codes + (((int64_t)page * kPage * hkv + h) * 2 + which) * D + j * 8;
      const int64_t step = (int64_t)hkv * 2 * D;
      auto write = [&](auto careful_c) {
        constexpr bool CAREFUL = decltype(careful_c)::value;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int m = i * ROWS + r0;
          if (i >= passes) continue;
          const Values<T> y(x[i]);
          u32x2_t c;
          c.x = kv8_codes<true, CAREFUL>(kv8_codes<false, CAREFUL>(0u, y.v[0] * inv, y.v[1] * inv), y.v[2] * inv, y.v[3] * inv);
          c.y = kv8_codes<true, CAREFUL>(kv8_codes<false, CAREFUL>(0u, y.v[4] * inv, y.v[5] * inv), y.v[6] * inv, y.v[7] * inv);
          if (m < n) *reinterpret_cast<u32x2_t*>(page_codes + mate_slot[m] * step) = c;
        }
      };
      if (careful)
        write(std::true_type());
      else
        write(std::false_type());
      if (raised) {
        const uint64_t written = wave_or64(mine ? 1ull << (s & 63) : 0);
        const float f = __uint_as_float((uint32_t)max(127 + old - e, 0) << 23);  // 2^-127 and less: 0
        u32x2_t c[PASSES];
#pragma unroll
        for (int i = 0; i < PASSES; ++i) c[i] = *reinterpret_cast<u32x2_t*>(page_codes + (i * ROWS + r0) * step);
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i][w], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i][w], true);
            c[i][w] = kv8_codes<true, true>(kv8_codes<false, true>(0u, a.x * f, a.y * f), b.x * f, b.y * f);
          }
          const int m = i * ROWS + r0;
          if ((written >> m & 1) == 0) *reinterpret_cast<u32x2_t*>(page_codes + m * step) = c[i];
        }
      }
      if ((anew || raised) && tid % D == 0) *scale_at = __uint_as_float((uint32_t)e << 23);
    };
    // Few rows (decode, verify) by code of their own: what runs once a workgroup
    // is fetched as it runs.
    if (passes == 1)
      run(std::integral_constant<int, 1>());
    else
      run(std::integral_constant<int, PASSES>());
    __syncthreads();  // the lists are free again
  }
}

// A lane takes 8 channels of a row; a row's lanes go through its heads, K then
// V of each.
template <class T, int D>
__global__ __launch_bounds__(256) void kv8_load_kernel(const uint8_t* __restrict__ codes,
                                                       const float* __restrict__ scales, int32_t num_slots,
                                                       const int32_t* __restrict__ slots, int32_t n, int32_t hkv,
                                                       typename T::elem* __restrict__ k,
                                                       typename T::elem* __restrict__ v, int64_t ld_k, int64_t ld_v) {
  constexpr uint32_t LANES = D / 8;
  const uint32_t id = blockIdx.x * 256 + threadIdx.x, per_row = hkv * 2 * LANES;  // a launch has at most 2^31 lanes
  const uint32_t t = id / per_row, u = id % per_row, h = u / (2 * LANES), which = u / LANES & 1, j = u % LANES;
  if (t >= (uint32_t)n) return;
  const int32_t slot = slots[t];
  u32x2_t c = {0, 0};
  float s = 1.f;
  if (slot >= 0 && slot < num_slots) {
    c = *reinterpret_cast<const u32x2_t*>(codes + (((int64_t)slot * hkv + h) * 2 + which) * D + j * 8);
    s = scales[((int64_t)(slot >> 6) * hkv + h) * 2 + which];
  }
  Chunk<T> x;
  if constexpr (std::is_same<T, F32>::value) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[w], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[w], true);
      x.v[4 * w] = a.x * s, x.v[4 * w + 1] = a.y * s, x.v[4 * w + 2] = b.x * s, x.v[4 * w + 3] = b.y * s;
    }
  } else {
    x.v = u32x4_t{T::template from_fp8<0>(c.x, s), T::template from_fp8<1>(c.x, s), T::template from_fp8<0>(c.y, s),
                  T::template from_fp8<1>(c.y, s)};
  }
  x.store((which ? v + (int64_t)t * ld_v : k + (int64_t)t * ld_k) + h * D + j * 8);
}

namespace {

// From here on a workgroup of the store takes the runs of 16 rows: those of a
// prompt are a page's 64, and one workgroup a row would mostly find that it has
// no run.
constexpr int kManyTokens = 2048;

template <class F>
int by_type_and_dim(int32_t dtype, int32_t d, F f) {
  auto dim = [&](auto t) {
    if (d == 64) return f(t, std::integral_constant<int, 64>());
    if (d == 128) return f(t, std::integral_constant<int, 128>());
    return f(t, std::integral_constant<int, 256>());
  };
  if (dtype == BS_BF16) return dim(Bf16());
  if (dtype == BS_F16) return dim(F16());
  return dim(F32());
}

}  // namespace

int launch_kv8_store(const void* k, const void* v, int32_t dtype, int64_t ld_k, int64_t ld_v, const int32_t* slots,
                     int32_t num_tok, int32_t hkv, int32_t d, uint8_t* codes, float* scales, int32_t num_slots,
                     hipStream_t stream) {
  return by_type_and_dim(dtype, d, [&](auto t, auto dim) {
    typedef decltype(t) T;
    typedef typename T::elem elem;
    constexpr int D = decltype(dim)::value;
    auto go = [&](auto rows) {
      constexpr int S = decltype(rows)::value;
      const int64_t groups = ((int64_t)num_tok + S - 1) / S, most = ((int64_t)1 << 31) / (2 * D);  // of a launch
      for (int64_t g = 0; g < groups; g += most) {
        const uint32_t n = (uint32_t)std::min(most, groups - g);
        hipLaunchKernelGGL((kv8_store_kernel<T, D, S>), dim3(S == 16 ? (n + 3) / 4 * 4 : n, hkv), dim3(2 * D), 0, stream,
                           static_cast<const elem*>(k), static_cast<const elem*>(v), ld_k, ld_v, slots, num_tok, hkv,
                           num_slots, codes, scales, (uint32_t)g, n);
        if (hipGetLastError() != hipSuccess) return (int)BS_ERR_LAUNCH;
      }
      return (int)BS_OK;
    };
    return num_tok < kManyTokens ? go(std::integral_constant<int, 1>()) : go(std::integral_constant<int, 16>());
  });
}

int launch_kv8_load(const uint8_t* codes, const float* scales, int32_t num_slots, const int32_t* slots,
                    int32_t num_slot_ids, int32_t hkv, int32_t d, void* k, void* v, int32_t dtype, int64_t ld_k,
                    int64_t ld_v, hipStream_t stream) {
  return by_type_and_dim(dtype, d, [&](auto t, auto dim) {
    typedef decltype(t) T;
    typedef typename T::elem elem;
    constexpr int D = decltype(dim)::value;
    const int64_t lanes = (int64_t)2 * hkv * (D / 8), most = std::max<int64_t>(1, ((int64_t)1 << 31) / lanes);
    for (int64_t r = 0; r < num_slot_ids; r += most) {
      const int64_t n = std::min<int64_t>(most, num_slot_ids - r);
      hipLaunchKernelGGL((kv8_load_kernel<T, D>), dim3((uint32_t)((n * lanes + 255) / 256)), dim3(256), 0, stream, codes,
                         scales, num_slots, slots + r, (int32_t)n, hkv, static_cast<elem*>(k) + r * ld_k,
                         static_cast<elem*>(v) + r * ld_v, ld_k, ld_v);
      if (hipGetLastError() != hipSuccess) return (int)BS_ERR_LAUNCH;
    }
    return (int)BS_OK;
  });
}

}  // namespace bs
