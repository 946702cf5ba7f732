// attn_prefill.h - attention over a sliding window and the first tokens, for
// many query rows of a request (attn_window's prefill form).
//
// The same sums as attn_gather.h, 4*D flops per (query vector, key): with many
// rows a key, the matrix cores and the softmax between their two products
// bound it.  A workgroup takes 32 * NW (row, head) pairs that share a kv head
// (the heads of a group packed beside the rows, so that a tile spans few
// positions) and walks the pages of its keys; a page is a tile of 64 keys:
//   * K and V pages are copied from HBM straight into LDS (16-bit pools), or
//     loaded into registers, converted and written there (codes), one page
//     ahead, two buffers, one barrier a page;
//   * S^T = K q^T with v_mfma_f32_32x32x16: a lane holds one query vector and
//     16 of every 32 keys, so the row maximum and sum need one exchange
//     between the wave's halves;
//   * O^T += V^T P^T: the accumulator of S^T is the B operand of the second
//     product with its keys in a fixed order (8*(i/4) + 4*half + i%4), and the
//     A operand is read from the row-major V tile in that order with the
//     transposing LDS loads; P never leaves its lane;
//   * the running maximum moves only when a score exceeds it by more than
//     kSlack (in log2), so the accumulators are hardly ever rescaled; P stays
//     below 2^(kSlack + kRaise), inside FP32 and both 16-bit types;
//   * P is rounded to the 16-bit operand type for the product (relative
//     2^-8 in bf16, as the output's own rounding);
//   * K rows are XOR-swizzled by 16-byte slices with key mod 16, V rows with
//     2 * (key mod 8), so that both kinds of LDS reads spread over the banks;
//   * pages that every row of a wave sees are not masked at all, pages that
//     none sees are skipped by the wave.
// Consecutive row blocks of one kv head run on one XCD, whose L2 then holds
// their window.
//
// Measured (calls back to back; under the profiler in brackets): 8,192 rows, window 4,096, 16 query / 2 kv
// heads of 128, bf16: 278 to 289 us (301 to 335), 950 to 988 TFLOP/s (an
// 8,192-cubed library product: 1,258), matrix cores busy for 49% of the cycles
// and vector units for 35%, at a clock that falls to 2.0 GHz.  5 ragged requests
// over the 4-bit cache in fp16, 28.7 GFLOP: 51 us (59).
#pragma once

#include "attn.h"

namespace bs {

struct PrefillArgs {
  const void* q;
  int64_t ld_q;
  const uint8_t *a, *b;
  int64_t ld_kv;
  int32_t num_pages, num_rows, hq, hkv, gb, hblocks;
  const int32_t *page_table, *req_row_ptr, *row_pos;
  int32_t pt_stride, max_rows, rows_per_tile, tiles_per_req, window, sinks;
  float scale_log2;  // of the scores, not below 0
  uint32_t flip;     // sign bits to turn in q: the scale was negative
  void* out;
  int64_t ld_out;
  float* lse;
  bool latest_first;        // a request's last rows start first
  uint32_t groups, nsplit;  // row blocks times head blocks; parts that a block's pages are split into
  float* partial;           // nsplit > 1: per (group, part) [cols][D] products, then [cols] (maximum, sums, 0)
};

// Which rows and heads a group is.  False: none.
struct PrefillGroup {
  int b, kvh, h0, heads, row0, nrows;
  __device__ __forceinline__ bool locate(const PrefillArgs& a, uint32_t group) {
    const int i_tile = group % a.tiles_per_req, rest = group / a.tiles_per_req;
    const int hb = rest % (a.hkv * a.hblocks), G = a.hq / a.hkv, hin = (hb % a.hblocks) * a.gb;
    b = rest / (a.hkv * a.hblocks), kvh = hb / a.hblocks;
    heads = min(a.gb, G - hin), h0 = kvh * G + hin;
    const int ra = max(a.req_row_ptr[b], 0);
    const int rb = (int)min((int64_t)min(a.req_row_ptr[b + 1], a.num_rows), (int64_t)ra + a.max_rows);
    const int last = ((rb > ra ? rb - ra : 0) + a.rows_per_tile - 1) / a.rows_per_tile - 1;
    if (i_tile > last) return false;
    row0 = ra + (a.latest_first ? last - i_tile : i_tile) * a.rows_per_tile, nrows = min(a.rows_per_tile, rb - row0);
    return true;
  }
};

template <class T>
__device__ __forceinline__ f32x16_t mfma32(const u32x4_t& a, const u32x4_t& b, const f32x16_t& c) {
  if constexpr (std::is_same<T, Bf16>::value)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

typedef int16_t i16x4_t __attribute__((ext_vector_type(4)));

// Four consecutive rows of one 16-bit column: the 16 lanes of a block give the
// addresses of 4 rows x 16 columns (8 bytes each) and lane c of the block
// receives column c.
__device__ __forceinline__ u32x2_t lds_read_tr(const uint8_t* p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) i16x4_t*)(uintptr_t)(uint32_t)(uintptr_t)p));
}

template <class T, int FORM, int D, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void attn_prefill_kernel(const PrefillArgs a) {
  constexpr bool FP4 = FORM == kForm4, FP8 = FORM == kForm8, CODES = FP4 || FP8;
  constexpr int ROW = D * 2;                // bytes of a key in LDS
  constexpr int NS = D / 8;                 // its 16-byte slices
  constexpr int KSWZ = NS < 16 ? NS - 1 : 15, VSWZ = NS < 16 ? NS - 1 : 15;
  constexpr int KS = D / 16, DT = D / 32;   // steps of the products
  constexpr int THREADS = 64 * NW;
  __shared__ __attribute__((aligned(1024))) uint8_t kv[2][2][kPage * ROW];  // buffer, K or V

  const int tid = threadIdx.x, lane = tid & 63, n32 = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Block b runs on XCD b mod 8: eight consecutive ids on one XCD (their rows
  // share most of their window in its L2), the next eight on the next.
  const uint32_t id = blockIdx.x / 64 * 64 + blockIdx.x % 8 * 8 + blockIdx.x / 8 % 8;
  if (id >= a.groups * a.nsplit) return;
  const uint32_t group = id % a.groups, split = id / a.groups;
  PrefillGroup w;
  if (!w.locate(a, group)) return;
  const int b = w.b, kvh = w.kvh, h0 = w.h0, heads = w.heads, row0 = w.row0, nrows = w.nrows;

  // Positions: of the workgroup's rows, of the wave's, of the lane's.
  int lo = 0x7FFFFFFF, hi = -1;
  for (int r = lane; r < nrows; r += 64) {
    const int t = a.row_pos[row0 + r];
    lo = min(lo, t < 0 ? 0x7FFFFFFF : t), hi = max(hi, t);
  }
  const int col = wave * 32 + n32, rr = col / a.gb, hh = col % a.gb;
  const bool ok = rr < nrows && hh < heads;
  const int t = ok ? a.row_pos[row0 + rr] : -1;
  int wlo = ok ? (t < 0 ? -1 : t) : 0x7FFFFFFF, whi = t, wfirst = t < 0 ? 0x7FFFFFFF : t;
  for (int o = 32; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor(lo, o)), hi = max(hi, __shfl_xor(hi, o));
    wlo = min(wlo, __shfl_xor(wlo, o)), whi = max(whi, __shfl_xor(whi, o)), wfirst = min(wfirst, __shfl_xor(wfirst, o));
  }
  const int tmin = __builtin_amdgcn_readfirstlane(lo), tmax = __builtin_amdgcn_readfirstlane(hi);
  // The wave's last position that all of its rows see, its last and its first
  // position.
  const int w_all = __builtin_amdgcn_readfirstlane(wlo), w_last = __builtin_amdgcn_readfirstlane(whi);
  const int w_first = __builtin_amdgcn_readfirstlane(wfirst);
  const int last = (int)min((int64_t)min(tmax, 0x7FFFFF00), (int64_t)a.pt_stride * kPage - 1);
  const int ns = max(0, min(a.sinks, last + 1)), sink_pages = (ns + kPage - 1) / kPage;
  const int wp0 = max(max(0, tmin - a.window + 1) / kPage, sink_pages);
  const int all_tiles = last < 0 ? 0 : sink_pages + max(0, last / kPage - wp0 + 1);
  const int tile0 = part_start(all_tiles, a.nsplit, split), tiles = part_start(all_tiles, a.nsplit, split + 1);
  const int32_t* ptab = a.page_table + (int64_t)b * a.pt_stride;

  u32x4_t qf[KS];
  {
    const typename T::elem* src = static_cast<const typename T::elem*>(a.q) + (int64_t)(row0 + (ok ? rr : 0)) * a.ld_q +
                                  (h0 + (ok ? hh : 0)) * D + 8 * half;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const u32x4_t x = *reinterpret_cast<const u32x4_t*>(src + 16 * ks);
      qf[ks] = ok ? x ^ a.flip : u32x4_t{0, 0, 0, 0};
    }
  }

  f32x16_t acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
  float m = -INFINITY;    // running maximum (scaled)
  Sums l = {0.f, 0.f};    // this half's share of the sums

  auto page_pos = [&](int i) { return i < sink_pages ? i : wp0 + (i - sink_pages); };
  // Next tile from `i` on whose page is one; `page` receives its id.
  auto next_tile = [&](int i, int& page) {
    for (; i < tiles; ++i) {
      page = ptab[page_pos(i)];
      if (page >= 0 && page < a.num_pages) break;
    }
    return i;
  };

  // 4-bit (8-bit): what a thread holds of the next page: 32 (16) channels, 16
  // bytes of codes, and their scale, of K or V, UNITS times.
  constexpr int PARTS = FP8 ? D / 8 : D / 16, PIECES = kPage * PARTS, UNITS = CODES ? (PIECES + THREADS - 1) / THREADS : 1;
  static_assert(CODES || kPage * NS % THREADS == 0, "the copies fill whole waves");
  u32x4_t codes[UNITS];
  uint32_t scale[UNITS];
  auto issue = [&](int page, int buf) {
    if constexpr (FP4) {
      const uint64_t rec = (uint64_t)a.hkv * D;
      const uint8_t* c0 = a.a + (uint64_t)page * kPage * rec + kvh * D;
      const uint8_t* s0 = a.b + (uint64_t)page * kPage * (rec / 16) + kvh * (D / 16);
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int x = u * THREADS + tid, key = x / (D / 16), part = x % (D / 16);
        if (PIECES % THREADS != 0 && x >= PIECES) continue;
        codes[u] = *reinterpret_cast<const u32x4_t*>(c0 + (uint64_t)key * rec + part * 16);
        scale[u] = s0[(uint64_t)key * (rec / 16) + part];
      }
    } else if constexpr (FP8) {
      const uint64_t rec = (uint64_t)a.hkv * 2 * D;
      const uint8_t* c0 = a.a + (uint64_t)page * kPage * rec + kvh * 2 * D;
      const uint32_t* s0 = reinterpret_cast<const uint32_t*>(a.b) + ((uint64_t)page * a.hkv + kvh) * 2;
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int x = u * THREADS + tid, key = x / PARTS, part = x % PARTS;
        if (PIECES % THREADS != 0 && x >= PIECES) continue;
        codes[u] = *reinterpret_cast<const u32x4_t*>(c0 + (uint64_t)key * rec + part * 16);
        scale[u] = s0[part >= PARTS / 2];
      }
    } else {
      const uint32_t rec = (uint32_t)(a.ld_kv * 2), bytes = rec * (kPage - 1) + D * 2;
      const uint64_t at = (uint64_t)page * kPage * (uint64_t)a.ld_kv * 2 + kvh * D * 2;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const uint64_t p = reinterpret_cast<uint64_t>(which ? a.b : a.a) + at;
        const u32x4_t rs = {(uint32_t)p, (uint32_t)(p >> 32), bytes, 0};
        const uint32_t dst = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)(&kv[buf][which][0]);
#pragma unroll
        for (int j = 0; j < kPage * NS / THREADS; ++j) {
          const int x = j * THREADS + tid, key = x / NS, s = x % NS;
          const int f = which ? (2 * key) & VSWZ : key & KSWZ;
          lds_dma_b128(rs, key * rec + (uint32_t)(s ^ f) * 16, dst + (j * THREADS + wave * 64) * 16);
        }
      }
    }
  };
  auto settle = [&](int buf) {
    if constexpr (FP4) {
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int x = u * THREADS + tid, key = x / (D / 16), part = x % (D / 16);
        if (PIECES % THREADS != 0 && x >= PIECES) continue;
        const int which = part >= D / 32, s = (part % (D / 32)) * 4, f = which ? (2 * key) & VSWZ : key & KSWZ;
        uint8_t* row = &kv[buf][which][key * ROW];
        const float sc = kv4_scale(scale[u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = codes[u][i];
          *reinterpret_cast<u32x4_t*>(row + ((s + i) ^ f) * 16) =
              u32x4_t{T::template from_fp4<0>(w, sc), T::template from_fp4<1>(w, sc), T::template from_fp4<2>(w, sc),
                      T::template from_fp4<3>(w, sc)};
        }
      }
    } else if constexpr (FP8) {
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int x = u * THREADS + tid, key = x / PARTS, part = x % PARTS;
        if (PIECES % THREADS != 0 && x >= PIECES) continue;
        const int which = part >= PARTS / 2, s = (part % (PARTS / 2)) * 2, f = which ? (2 * key) & VSWZ : key & KSWZ;
        uint8_t* row = &kv[buf][which][key * ROW];
        const float sc = __uint_as_float(scale[u]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w0 = codes[u][2 * i], w1 = codes[u][2 * i + 1];
          *reinterpret_cast<u32x4_t*>(row + ((s + i) ^ f) * 16) =
              u32x4_t{T::template from_fp8<0>(w0, sc), T::template from_fp8<1>(w0, sc), T::template from_fp8<0>(w1, sc),
                      T::template from_fp8<1>(w1, sc)};
        }
      }
    } else {
      wait_vmcnt<0>();
    }
  };

  const uint32_t k_row = n32 * ROW, k_swz = n32 & KSWZ;
  const int v_key = 4 * half + ((lane & 15) >> 2), v_cc = lane & 3;
  uint32_t v_off[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) {
    const int s = 4 * d + 2 * ((lane >> 4) & 1) + (v_cc >> 1);
    v_off[d] = v_key * ROW + ((s ^ ((2 * v_key) & VSWZ)) * 16) + (v_cc & 1) * 8;
  }
  // V^T's fragment of 16 keys from kb on, channels 32*d .. +31.
  auto v_frag = [&](const uint8_t* vt, int kb, int d) {
    const u32x2_t x = lds_read_tr(vt + v_off[d] + kb * ROW), y = lds_read_tr(vt + v_off[d] + (kb + 8) * ROW);
    return u32x4_t{x.x, x.y, y.x, y.y};
  };

  // Does every row of the wave see all of the page at p0?  Any of it?
  auto all_seen = [&](int p0) {
    return p0 + kPage - 1 <= w_all && (p0 > w_last - a.window || p0 + kPage - 1 < a.sinks);
  };
  auto any_seen = [&](int p0) { return p0 <= w_last && (p0 + kPage - 1 > w_first - a.window || p0 < a.sinks); };

  auto compute = [&](auto masked_c, auto careful_c, int p0, int buf) {
    constexpr bool MASKED = decltype(masked_c)::value, CAREFUL = MASKED && decltype(careful_c)::value;
    const uint8_t *kt = kv[buf][0], *vt = kv[buf][1];
    f32x16_t s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[j][i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const u32x4_t kf = *reinterpret_cast<const u32x4_t*>(kt + j * 32 * ROW + k_row + (((2 * ks + half) ^ k_swz) * 16));
        s[j] = mfma32<T>(kf, qf[ks], s[j]);
      }
    }
    if constexpr (!MASKED) {
      // Eight fragments of K in flight: left alone, two are.
      __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
#pragma unroll
      for (int k = 0; k < 2 * KS - 8; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x008, 8, 0);
    }
    // Bits of the lane's keys that its row sees: key 32*j + 8*(i/4) +
    // 4*half + i%4 at bit 8*(i/4) + i%4 of word j.
    uint32_t vis[2] = {0, 0};
    if constexpr (MASKED) {
      const uint64_t v = visible_bits(p0, t, a.window, a.sinks) >> (4 * half);
      vis[0] = (uint32_t)v, vis[1] = (uint32_t)(v >> 32);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[j][i] = __uint_as_float(
              bit_select(bit_mask(vis[j], 8 * (i >> 2) + (i & 3)), __float_as_uint(s[j][i]), 0xFF800000u));
    }
    float mx = max_nan(s[0][0], s[1][0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) mx = max_nan(max_nan(mx, s[0][i]), s[1][i]);
    {
      const uint32_t u = __float_as_uint(mx);
      auto x = __builtin_amdgcn_permlane32_swap(u, u, false, false);
      mx = rounded_product(max_nan(__uint_as_float(x[0]), __uint_as_float(x[1])), a.scale_log2);
    }
    if (ballot(mx - m > kSlack)) {
      const float mn = fmaxf(m, mx);
      const float f = exp2_fast(m - finite_max(mn));
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d) acc[d] *= f;
      m = mn;
    }
    float scale = a.scale_log2, base = finite_max(m);  // of the weights
    if constexpr (decltype(careful_c)::value) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[j][i] = rounded_product(s[j][i], scale) - base;
      scale = 1.f, base = 0.f;
    }
    u32x4_t pf[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float p[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) p[i] = exp2_fast(__builtin_fmaf(s[j][i], scale, T::kRaise - base));
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 16; i += 4) x += (p[i] + p[i + 1]) + (p[i + 2] + p[i + 3]);
      l.x += x;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        pf[2 * j + g] = u32x4_t{T::pack(p[8 * g], p[8 * g + 1]), T::pack(p[8 * g + 2], p[8 * g + 3]),
                                T::pack(p[8 * g + 4], p[8 * g + 5]), T::pack(p[8 * g + 6], p[8 * g + 7])};
        l.y = add_rounded<T>(pf[2 * j + g], l.y);
      }
    }
    // Careful: infinities and NaN in V at positions that only some rows see are
    // taken out of the product (0 * inf is NaN), and what the rows that see them
    // must show is added after it.
    uint32_t bad = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        u32x4_t v = v_frag(vt, 16 * g, d);
        if constexpr (CAREFUL) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = nonfinite_pair<T>(v[i]);
            bad |= x, v[i] &= ~spread_halves(x);
          }
        }
        acc[d] = mfma32<T>(v, pf[g], acc[d]);
      }
    if constexpr (CAREFUL) {
      if (ballot(bad != 0)) {
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          const uint32_t w = (g < 2 ? vis[0] : vis[1]) >> (16 * (g & 1));
          u32x4_t see;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = 2 * i, at = 8 * (k >> 2) + (k & 3);
            see[i] = (bit_mask(w, at) & T::kOne) | (bit_mask(w, at + 1) & (T::kOne << 16));
          }
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            const u32x4_t v = v_frag(vt, 16 * g, d);
            u32x4_t marks;
#pragma unroll
            for (int i = 0; i < 4; ++i) marks[i] = nonfinite_marks<T>(v[i]);
            f32x16_t n;
#pragma unroll
            for (int i = 0; i < 16; ++i) n[i] = 0.f;
            n = mfma32<T>(marks, see, n);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[d][i] += nonfinite_term(n[i]);
            __builtin_amdgcn_sched_barrier(0);  // one channel tile at a time: this path is rare, its registers are not
          }
        }
      }
    }
  };

  int page, i, buf;
  auto step = [&](auto masked_c, auto careful_c) {
    // The buffer is complete in every wave, and the other one has been read.
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    int page1 = 0;
    const int i1 = next_tile(i + 1, page1);
    if (i1 < tiles) issue(page1, buf ^ 1);
    const int p0 = page_pos(i) * kPage;
    if (!decltype(masked_c)::value || any_seen(p0)) compute(masked_c, careful_c, p0, buf);
    if (i1 < tiles) settle(buf ^ 1);
    i = i1, buf ^= 1;
  };
  auto run = [&](auto careful_c) {
    page = 0, i = next_tile(tile0, page), buf = 0;
    if (i < tiles) {
      issue(page, 0);
      settle(0);
    }
    // Loops of their own for the pages without and with a mask: joined in one,
    // the accumulators were copied at each join (128 moves a page).
    while (i < tiles) {
      while (i < tiles && all_seen(page_pos(i) * kPage)) step(std::false_type(), careful_c);
      while (i < tiles && !all_seen(page_pos(i) * kPage)) step(std::true_type(), careful_c);
    }
  };
  run(std::false_type());
  // A masked weight is 0, and 0 times an infinity or a NaN of V is NaN in rows
  // that do not see it.  Such values show in the result: if a wave's is not
  // finite, the workgroup starts over with masked pages done carefully.  (Care
  // from the start made a masked page cost 2.8 times an unmasked one.)  So it
  // does, with weights of rounded products on all pages, where maxima are huge.
  {
    float top = l.x;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int k = 0; k < 16; k += 2) top = max_nan(max_nan(top, fabsf(acc[d][k])), fabsf(acc[d][k + 1]));
    __shared__ uint32_t not_finite[NW];
    const bool bad = ballot(!(top < INFINITY) || fabsf(finite_max(m)) > kHugeScore) != 0;
    if (lane == 0) not_finite[wave] = bad;
    __syncthreads();
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < NW; ++k) any |= not_finite[k];
    if (any) {
      m = -INFINITY, l = Sums{0.f, 0.f};
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[d][k] = 0.f;
      run(std::true_type());
    }
  }

#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint32_t u = __float_as_uint(l[e]);
    auto x = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    l[e] = __uint_as_float(x[0]) + __uint_as_float(x[1]);
  }
  if (a.nsplit > 1) {
    constexpr int COLS = 32 * NW;
    float* part = a.partial + ((uint64_t)group * a.nsplit + split) * (COLS * (D + 4));
    if (ok) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<f32x4_t*>(part + col * D + 32 * d + 8 * g + 4 * half) =
              f32x4_t{acc[d][4 * g], acc[d][4 * g + 1], acc[d][4 * g + 2], acc[d][4 * g + 3]};
      if (half == 0) *reinterpret_cast<f32x4_t*>(part + COLS * D + 4 * col) = f32x4_t{m, l.x, l.y, 0.f};
    }
    return;
  }
  const float inv = l.y == 0.f ? 0.f : 1.f / l.y;
  typename T::elem* dst = static_cast<typename T::elem*>(a.out) + (int64_t)(row0 + rr) * a.ld_out + (h0 + hh) * D;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
      // Channels 8g + 4*half + 0..3 of the tile and the same of g + 1: the
      // halves exchange so that each stores 8 channels at once.
      uint32_t w[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          w[e][k] = T::pack(acc[d][4 * (g + e) + 2 * k] * inv, acc[d][4 * (g + e) + 2 * k + 1] * inv);
      auto x = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
      auto y = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
      if (ok) *reinterpret_cast<u32x4_t*>(dst + 32 * d + 8 * (g + half)) = u32x4_t{x[0], y[0], x[1], y[1]};
    }
  if (ok && half == 0 && a.lse != nullptr)
    a.lse[(int64_t)(row0 + rr) * a.hq + h0 + hh] = row_lse<T>(m, l.x);
}

// Joins the parts of every group, in their order: a lane takes 4 channels of a
// column.  A launch of its own: one workgroup a group, the last of its parts
// to arrive, would read its 66 KiB a part alone (50 rows over 64 pages in 16
// parts: 40 us in place of 22).
template <class T, int D, int COLS>
__global__ __launch_bounds__(256) void attn_join_kernel(const PrefillArgs a) {
  constexpr int PIECES = COLS * D / 4 / 256;
  const uint32_t group = blockIdx.x / PIECES, u = blockIdx.x % PIECES * 256 + threadIdx.x;
  PrefillGroup w;
  if (!w.locate(a, group)) return;
  const int col = u / (D / 4), d = u % (D / 4) * 4, rr = col / a.gb, hh = col % a.gb;
  if (rr >= w.nrows || hh >= w.heads) return;
  const float* part = a.partial + (uint64_t)group * a.nsplit * (COLS * (D + 4));
  float m = -INFINITY;
  Sums l = {0.f, 0.f};
  f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (uint32_t i = 0; i < a.nsplit; ++i, part += COLS * (D + 4)) {
    const f32x4_t x = *reinterpret_cast<const f32x4_t*>(part + COLS * D + 4 * col);
    const f32x4_t y = *reinterpret_cast<const f32x4_t*>(part + col * D + d);
    const float nm = fmaxf(m, x.x), nf = finite_max(nm), f = exp2_fast(m - nf), g = exp2_fast(x.x - nf);
    l = l * f + x.yz * g, o = o * f + y * g, m = nm;
  }
  write_joined<T>(static_cast<typename T::elem*>(a.out) + (int64_t)(w.row0 + rr) * a.ld_out + (w.h0 + hh) * D, d, o, m, l,
                  a.lse == nullptr ? nullptr : a.lse + (int64_t)(w.row0 + rr) * a.hq + w.h0 + hh);
}

template <class T, int FORM>
int launch_attn_prefill(const PrefillArgs& a, int d, int waves, uint32_t grid, hipStream_t stream) {
  auto go = [&](auto dim, auto nw) {
    constexpr int NW = decltype(nw)::value;
    constexpr int D = decltype(dim)::value, COLS = 32 * NW;
    hipLaunchKernelGGL((attn_prefill_kernel<T, FORM, D, NW>), dim3(grid), dim3(64 * NW), 0, stream, a);
    if (a.nsplit > 1)
      hipLaunchKernelGGL((attn_join_kernel<T, D, COLS>), dim3(a.groups * (COLS * D / 4 / 256)), dim3(256), 0, stream, a);
  };
  auto by_waves = [&](auto dim) {
    if (waves == 8)
      go(dim, std::integral_constant<int, 8>());
    else
      go(dim, std::integral_constant<int, 4>());
  };
  if (d == 64)
    by_waves(std::integral_constant<int, 64>());
  else if (d == 128)
    by_waves(std::integral_constant<int, 128>());
  else if constexpr (FORM != kForm4)  // the registers hold one wave a SIMD; the 4-bit cache is gathered at this size
    go(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
  return hipGetLastError() == hipSuccess ? BS_OK : BS_ERR_LAUNCH;
}

}  // namespace bs
