// kv8.hip - the 8-bit KV cache: rows quantised as they are written, and read
// back.
//
// Store.  A page's scale belongs to all its tokens, so the rows of a call that
// lie in one page are one workgroup's work, for each kv head: with m their largest
// finite magnitude (K and V apart),
//   e = the least with m <= 448 * 2^e;  a call that writes the page's first slot
//   sets the page's scale to 2^e, any other raises it to 2^e if it is below,
//   and then the codes of the page's other slots are rounded to the new scale;
//   code = x * 2^-e rounded to the nearest E4M3 value, ties to even.
// Load: code * scale.
//
// Streams without reuse: HBM bounds them at the prefill sizes and the launch at
// the decode ones (8,192 tokens x 8 heads of 128: 12.0 and 9.2 us, 4.2 and 5.5
// TB/s; 64 tokens x 2 heads 3.9 and 2.8).  A workgroup keeps its rows in registers
// between the maximum and the rounding, so they are read once: 2 * D lanes, half of
// them for K, 8 channels of a row a lane.  Which rows share a page (a run) is found
// from the slots: they lie within 64 consecutive rows of the call, so a wave that
// holds the 64 slots before its group and the 128 from there on sees all of every
// run that begins in the group.  A run of up to 8 rows takes the lanes of one row,
// beside 7 others (decode, verify), a longer one the workgroup (2,000 tokens of a page
// each, 2 heads of 128: 5.6 us, 15.4 with one run after the other).
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

// 8 values as codes.  Not CAREFUL: all are finite and of at most 448 scales, and the
// hardware's scaled conversion takes two at a time.
template <bool CAREFUL, class T>
__device__ __forceinline__ u32x2_t kv8_codes(const Chunk<T>& x, float scale) {
  u32x2_t c;
  if constexpr (CAREFUL) {
    const Values<T> y(x);
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));
#pragma unroll
    for (int w = 0; w < 2; ++w)
      c[w] = kv8_pack<true>(kv8_pack<false>(0u, y.v[4 * w] * inv, y.v[4 * w + 1] * inv), y.v[4 * w + 2] * inv, y.v[4 * w + 3] * inv);
  } else {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      i16x2_t two = {0, 0};
      if constexpr (std::is_same<T, F32>::value) {
        two = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(two, x.v[4 * w], x.v[4 * w + 1], scale, false);
        two = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(two, x.v[4 * w + 2], x.v[4 * w + 3], scale, true);
      } else {
        two = T::template to_fp8<0>(two, x.v[2 * w], scale);
        two = T::template to_fp8<1>(two, x.v[2 * w + 1], scale);
      }
      c[w] = __builtin_bit_cast(uint32_t, two);
    }
  }
  return c;
}

// The largest of N neighbouring lanes' values, in each of them.
template <int N>
__device__ __forceinline__ uint32_t lanes_max_u32(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kDppQuadXor1, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kDppQuadXor2, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kDppRowHalfMirror, 0xF, 0xF, false));
  if (N > 8) x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kDppRowMirror, 0xF, 0xF, false));
  if (N == 32) x = max(x, (uint32_t)__shfl_xor((int)x, 16));
  if (N == 64) x = max(max(readlane(x, 0), readlane(x, 16)), max(readlane(x, 32), readlane(x, 48)));
  return x;
}

// The largest magnitude of n <= N rows of 8 channels; without infinities and NaN, if there
// are any in the wave (careful is set then).
template <class T, int N>
__device__ __forceinline__ uint32_t largest(const Chunk<T> (&x)[N], int n, bool& careful) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) top = max(top, x[i].top());
  if (ballot(top >= 0x7F800000u) != 0) {
    careful = true, top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i >= n) continue;
      const Values<T> y(x[i]);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t u = __float_as_uint(y.v[c]) & 0x7FFFFFFFu;
        top = max(top, u < 0x7F800000u ? u : 0u);
      }
    }
  }
  return top;
}

// A run of at most ROWS rows, of each a lane has 8 channels.
template <class T, int ROWS>
struct ShortRun {
  static constexpr int N = ROWS;
  Chunk<T> x[N];
  int slot[N], n, page;  // in the page; rows
  uint64_t written;      // the slots, as bits
  float was;             // scale
  bool there, anew;
};

// A page's scale (its biased exponent): what its new rows need and, unless the page begins
// anew, no less than it was.
struct Scale {
  int e, old;
  bool raised;
  __device__ __forceinline__ Scale(uint32_t top, float was, bool anew) {
    e = kv8_exponent(top), old = min(max((int)(__float_as_uint(was) >> 23), kExpMin8), kExpMax8);
    raised = !anew && e > old;
    if (!anew) e = max(e, old);
  }
  __device__ __forceinline__ float value() const { return __uint_as_float((uint32_t)e << 23); }
};

// Rows first, first + step, ... (N of them) of a page, but for those that `written` names, from scale 2^old to 2^e.
template <int N>
__device__ __forceinline__ void rescale(uint8_t* codes, int64_t row_bytes, int first, int step, uint64_t written, int old, int e) {
  const float f = __uint_as_float((uint32_t)max(127 + old - e, 0) << 23);  // 2^-127 and less: 0
  codes += first * row_bytes, written >>= first;
#pragma unroll 1
  for (int n = 0; n < N; n += 8, codes += 8 * step * row_bytes, written >>= 8 * step & 63) {
    u32x2_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = *reinterpret_cast<u32x2_t*>(codes + i * step * row_bytes);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i][w], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i][w], true);
        c[i][w] = kv8_pack<true>(kv8_pack<false>(0u, a.x * f, a.y * f), b.x * f, b.y * f);
      }
      if ((written >> i * step & 1) == 0) *reinterpret_cast<u32x2_t*>(codes + i * step * row_bytes) = c[i];
    }
  }
}

}  // namespace

// S: rows of the call whose runs (rows of one page) a workgroup takes if they
// begin there: S rows a group, `groups` from group0 on.  Long runs go one after
// the other, all lanes on each; short ones (decode, verify) side by side, a row's
// lanes on each.
//
// In a prompt's rows every (64 / S)th group begins a run.  Consecutive
// workgroups go to the 8 XCDs in turn, so groups that far apart are neighbours in
// the grid: with the groups in order, two XCDs did all the work (8,192 rows x 8
// heads of 128, S = 16: 31.5 us).
template <class T, int D, int S>
__global__ __launch_bounds__(2 * D) void kv8_store_kernel(const typename T::elem* __restrict__ k,
                                                          const typename T::elem* __restrict__ v, int64_t ld_k,
                                                          int64_t ld_v, const int32_t* __restrict__ slots,
                                                          int32_t num_tok, int32_t hkv, int32_t num_slots,
                                                          uint8_t* codes, float* scales, uint32_t group0, uint32_t groups) {
  constexpr int LANES = D / 8, ROWS = D / LANES;  // of a row; rows at a time
  static_assert(ROWS == 8, "D lanes for K, D for V");
  constexpr int HALF_WAVES = D / 64;              // waves that work on K (V)
  constexpr int PASSES = kPage / ROWS, SHORT = 8;  // rows a lane of a long run; rows of a short run
  __shared__ int32_t list_row[kSpan], list_slot[kSpan];  // a long run's rows
  __shared__ uint32_t tops[2][HALF_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.y, which = wave / HALF_WAVES;
  const int r0 = tid % D / LANES, j = tid % LANES;
  const uint32_t apart = (groups + kSpan / S - 1) / (kSpan / S);
  const uint32_t group = blockIdx.x % apart * (kSpan / S) + blockIdx.x / apart;
  if (group >= groups) return;
  const int64_t first = ((int64_t)group0 + group) * S;
  const typename T::elem* src = (which ? v : k) + h * D + j * 8;
  const int64_t ld = which ? ld_v : ld_k, row_bytes = (int64_t)hkv * 2 * D;
  auto scale_of = [&](int page) { return scales + ((int64_t)page * hkv + h) * 2 + which; };
  auto codes_of = [&](int page) { return codes + (((int64_t)page * kPage * hkv + h) * 2 + which) * D + j * 8; };

  // The slots of the 64 rows before and of 128 from the first on; -1 for those that are none.
  auto slot_of = [&](int64_t t) {
    const int32_t x = t >= 0 && t < num_tok ? slots[t] : -1;
    return x >= 0 && x < num_slots ? x : -1;
  };
  const int before = slot_of(first - kSpan + lane), here = slot_of(first + lane), behind = slot_of(first + kSpan + lane);
  const int here_page = here >> 6, before_page = before >> 6, behind_page = behind >> 6;
  const uint64_t begins_page = ballot(here >= 0 && (here & 63) == 0), begins_behind = ballot(behind >= 0 && (behind & 63) == 0);
  int runs = 0, most = 0;  // short runs, and the most rows of one
  u32x4_t my_rows = {0, 0, 0, 0};  // lane i: the rows of short run i, as bits, and its page
  int my_page = 0;
  for (uint64_t left = ballot(here >= 0) & ((1ull << S) - 1); left != 0;) {
    // The first row left, its page, and the page's rows among the 64 from that row on.
    const int at = __builtin_ctzll(left), page = readlane(here_page, at);
    const uint64_t mask = ballot(here_page == page), late = ballot(behind_page == page) & ((1ull << at) - 1);
    left &= ~mask;
    if (ballot(before_page == page) != 0) continue;  // the run began before
    const int n = __popcll(mask) + __popcll(late);
    if (n <= SHORT) {
      my_rows = lane == runs ? u32x4_t{(uint32_t)mask, (uint32_t)(mask >> 32), (uint32_t)late, (uint32_t)(late >> 32)} : my_rows;
      my_page = lane == runs ? page : my_page;
      ++runs, most = max(most, n);
      continue;
    }
    const bool anew = ((mask & begins_page) | (late & begins_behind)) != 0;
    if (wave == 0) {
      const int m = lanes_below(mask), l = __popcll(mask) + lanes_below(late);
      if (mask >> lane & 1) list_row[m] = lane, list_slot[m] = here & 63;
      if (late >> lane & 1) list_row[l] = kSpan + lane, list_slot[l] = behind & 63;
    }
    const float was = *scale_of(page);
    __syncthreads();
    const int passes = (n + ROWS - 1) / ROWS;
    Chunk<T> x[PASSES];  // lanes past the last row take it again
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
      if (i < passes) x[i].load(src + (first + list_row[min(i * ROWS + r0, n - 1)]) * ld);
    bool careful = false;
    uint32_t top = lanes_max_u32<64>(largest(x, passes, careful));
    if (lane == 0) tops[which][wave % HALF_WAVES] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < HALF_WAVES; ++w) top = max(top, tops[which][w]);
    const Scale sc(top, was, anew);
    uint8_t* const at0 = codes_of(page);
    auto write = [&](auto careful_c) {
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int m = i * ROWS + r0;
        if (i >= passes) continue;
        const u32x2_t c = kv8_codes<decltype(careful_c)::value>(x[i], sc.value());
        if (m < n) *reinterpret_cast<u32x2_t*>(at0 + list_slot[m] * row_bytes) = c;
      }
    };
    if (careful || sc.e == kExpMax8)  // values past 448 scales
      write(std::true_type());
    else
      write(std::false_type());
    if (sc.raised) rescale<PASSES>(at0, row_bytes, r0, ROWS, wave_or64(lane < n ? 1ull << list_slot[lane] : 0), sc.old, sc.e);
    if ((anew || sc.raised) && tid % D == 0) *scale_of(page) = sc.value();
    __syncthreads();  // the list is free again
  }
  // Short run q + r0.
  auto fetch = [&](int q, auto& run) {
    run.there = q + r0 < runs;
    const int r = min(q + r0, runs - 1);
    run.page = __shfl(my_page, r), run.was = *scale_of(run.page);
    uint64_t mask = (uint32_t)__shfl((int)my_rows.x, r) | (uint64_t)(uint32_t)__shfl((int)my_rows.y, r) << 32;
    uint64_t late = (uint32_t)__shfl((int)my_rows.z, r) | (uint64_t)(uint32_t)__shfl((int)my_rows.w, r) << 32;
    run.anew = ((mask & begins_page) | (late & begins_behind)) != 0;
    run.n = __popcll(mask) + __popcll(late), run.written = 0;
    int row = 0, at = 0;  // in the group; in the cache
#pragma unroll
    for (int i = 0; i < run.N; ++i) {
      if (i >= most) continue;
      // The next row; without one, the last again.
      const bool now = mask != 0;
      const int bit = __builtin_ctzll(now ? mask : late | 1ull << 63);
      const int s_here = __shfl(here, bit), s_behind = __shfl(behind, bit);
      row = now ? bit : late != 0 ? kSpan + bit : row, at = now ? s_here : late != 0 ? s_behind : at;
      run.x[i].load(src + (first + row) * ld);
      run.slot[i] = at & 63, run.written |= 1ull << run.slot[i];
      mask &= mask - 1;  // 0 stays 0
      late = now ? late : late & (late - 1);
    }
  };
  auto finish = [&](auto& run) {
    bool careful = false;
    const Scale sc(lanes_max_u32<LANES>(largest(run.x, most, careful)), run.was, run.anew);
    uint8_t* const at0 = codes_of(run.page);
    auto write = [&](auto careful_c) {
#pragma unroll
      for (int i = 0; i < run.N; ++i) {
        if (i >= most) continue;
        const u32x2_t c = kv8_codes<decltype(careful_c)::value>(run.x[i], sc.value());
        if (run.there && i < run.n) *reinterpret_cast<u32x2_t*>(at0 + run.slot[i] * row_bytes) = c;
      }
    };
    if (careful || ballot(sc.e == kExpMax8) != 0)
      write(std::true_type());
    else
      write(std::false_type());
    if (run.there && (run.anew || sc.raised) && j == 0) *scale_of(run.page) = sc.value();
    // Pages whose scale grew, one after the other, by the whole wave.
    for (uint64_t grown = ballot(run.there && sc.raised && j == 0); grown != 0; grown &= grown - 1) {
      const int l = __builtin_ctzll(grown);
      const uint64_t w = readlane((uint32_t)run.written, l) | (uint64_t)readlane((uint32_t)(run.written >> 32), l) << 32;
      rescale<LANES>(codes_of((int)readlane(run.page, l)), row_bytes, lane / LANES, 64 / LANES, w, (int)readlane(sc.old, l),
                     (int)readlane(sc.e, l));
    }
  };
  if (most <= 2) {  // decode: several runs' loads in flight
    constexpr int TOGETHER = S / ROWS > 4 ? 4 : S / ROWS > 1 ? S / ROWS : 1;
    for (int q = 0; q < runs; q += ROWS * TOGETHER) {
      ShortRun<T, 2> run[TOGETHER];
#pragma unroll
      for (int i = 0; i < TOGETHER; ++i) fetch(q + i * ROWS, run[i]);
#pragma unroll
      for (int i = 0; i < TOGETHER; ++i) finish(run[i]);
    }
  } else {
    for (int q = 0; q < runs; q += ROWS) {
      ShortRun<T, SHORT> run;
      fetch(q, run);
      finish(run);
    }
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

// Rows of a group: 8, and 16 from here on (bf16, us: 64 x 1 tokens of 2 heads of 128
// 3.9 and 5.4, 512 x 1 of 8 heads 4.6 and 5.7, 2,000 x 1 8.8 and 8.0, 400 x 6 12.6 and 8.4,
// one prompt of 600 4.5 and 4.4, of 1,500 6.3 and 5.0, of 8,192 15.2 and 12.0; 32 rows: 8.2,
// 8.9, 10.4, 6.9, 4.4, 5.0, 11.1).
constexpr int kManyTokens = 1024;

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
      constexpr int S = decltype(rows)::value, APART = kSpan / S;
      const int64_t groups = ((int64_t)num_tok + S - 1) / S, most = ((int64_t)1 << 31) / (2 * D) - APART;  // of a launch
      for (int64_t g = 0; g < groups; g += most) {
        const uint32_t n = (uint32_t)std::min(most, groups - g);
        hipLaunchKernelGGL((kv8_store_kernel<T, D, S>), dim3((n + APART - 1) / APART * APART, hkv), dim3(2 * D), 0, stream,
                           static_cast<const elem*>(k), static_cast<const elem*>(v), ld_k, ld_v, slots, num_tok, hkv,
                           num_slots, codes, scales, (uint32_t)g, n);
        if (hipGetLastError() != hipSuccess) return (int)BS_ERR_LAUNCH;
      }
      return (int)BS_OK;
    };
    return num_tok < kManyTokens ? go(std::integral_constant<int, 8>()) : go(std::integral_constant<int, 16>());
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
