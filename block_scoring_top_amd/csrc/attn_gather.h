// attn_gather.h - attention over gathered KV slots, for few query rows a key:
// the rows of a selection (attn_slots), and decode or verify rows of a
// sliding window (attn_window).
//
// Per query row r and head h (kv head h / G): x_i = scale * <q, K_i> over the
// row's keys, o = sum_i softmax(x)_i V_i, lse = log sum_i exp(x_i).  One pass
// over the keys with a running maximum and sum in FP32.
//
// What bounds it is the gather: a key is read once for the G (times rows)
// query vectors that share it, 4*G*D flops for 17/16*D bytes (4-bit) or 4*D
// bytes (16-bit).  So the kernel keeps loads in flight and the rest small:
//   * a wave works alone on 32-key chunks, the next chunk's K and V in flight
//     while it computes; no workgroup barrier in the loop;
//   * S^T = K q^T with v_mfma_f32_16x16x32: the A operand's lane is a key and
//     a quarter of its row (16 bytes of codes hold one group of 32 channels at
//     D = 128: one scale a lane).  The order of channels inside the product is
//     free as long as q has the same;
//   * O^T += V^T P^T: in S^T's accumulator a lane already holds the P of one
//     query vector and of keys 4*(lane/16)+0..3 of each 16-key tile, which is
//     the B operand of a 32-key product whose key order is chosen to match.
//     The A operand needs 8 keys of one channel: a lane loads D/16 channels
//     of 8 keys, converts, and transposes pairs of keys with byte permutes;
//   * the running maximum moves only when a score exceeds it by more than
//     kSlack (in log2): the accumulators are hardly ever rescaled, and P stays
//     below 2^(kSlack + kRaise), inside FP32 and both 16-bit types (fp16's are
//     raised by 2^kRaise = 2^7, which keeps small weights out of its subnormals);
//   * P is rounded to the 16-bit operand type for the product (relative
//     2^-8 in bf16, as the output's own rounding); the output is divided by the
//     FP32 sum of the rounded values, lse is of the FP32 values' own.
// The 4 waves of a workgroup interleave chunks and join through LDS.  With
// few rows the keys are split over workgroups too: partial results go to the
// workspace and the last workgroup of a group to arrive joins them in split
// order (so the result does not depend on the arrival order).
//
// Measured (calls back to back, the cache in the Infinity Cache where it fits):
// 64 x 6 rows of 2,051 slots, 16 query / 2 kv heads of 128, 4-bit cache: 43 us, 225
// MB fetched at 5.1 TB/s (a large copy from HBM: 4.8), the vector units busy for
// 54% of it.  16 rows of 2,048 slots, 4 kv heads: 10.3 us; one row: 7.9 us.  777
// rows of 2,051 slots over a 25 MB 16-bit pool, 3 kv heads of 64: 111 to 116 us,
// 1.2 GB gathered, of which the L2s let 732 MB through at 6.4 TB/s.
#pragma once

#include "attn.h"

namespace bs {

constexpr int kGaWaves = 4;
constexpr int kGaKeys = 32;  // keys per wave and step

struct GatherArgs {
  const void* q;
  int64_t ld_q;
  const uint8_t *a, *b;  // 4-bit and 8-bit: codes, scales; 16-bit: K and V pools
  int64_t ld_kv;         // 16-bit pools: elements from one slot to the next
  int32_t num_slots, num_rows, hq, hkv;
  int32_t gb, hblocks;   // heads per block and blocks of one kv head's query heads
  // a selection's slot lists
  const int32_t* slots;
  int32_t ld_slots;
  const int32_t* count;
  // a window
  const int32_t *page_table, *req_row_ptr, *row_pos;
  int32_t pt_stride, max_rows, rows_per_tile, tiles_per_req, window, sinks;
  float scale_log2;  // of the scores, above 0
  uint32_t flip;     // sign bits to turn in q: the scale was negative
  void* out;
  int64_t ld_out;
  float* lse;
  uint32_t* counters;  // one per group of splits, zero between calls
  float* partial;
  int32_t nsplit;
  int32_t tiles;     // row tiles; xcd_rows: eight consecutive ones on one XCD
  bool xcd_rows;
};

template <int FORM, int D>
struct GatherRaw {
  static constexpr int kKDwords = FORM == kForm4 ? D / 32 : FORM == kForm8 ? D / 16 : D / 8;  // a quarter of a key's row
  // D/16 channels of a key
  static constexpr int kVDwords = FORM == kForm4 ? (D < 128 ? 1 : D / 128) : FORM == kForm8 ? D / 64 : D / 32;
  uint32_t k[2][kKDwords];
  uint32_t v[8][kVDwords];
};

__device__ __forceinline__ void load_4dwords(uint32_t* dst, const uint8_t* p) {
  const u32x4_t x = *reinterpret_cast<const u32x4_t*>(p);
  dst[0] = x.x, dst[1] = x.y, dst[2] = x.z, dst[3] = x.w;
}

template <int N>
__device__ __forceinline__ void load_dwords(uint32_t (&dst)[N], const uint8_t* p) {
  if constexpr (N == 1) {
    dst[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const u32x2_t x = *reinterpret_cast<const u32x2_t*>(p);
    dst[0] = x.x, dst[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) load_4dwords(dst + i, p + 4 * i);
  }
}

// How a chunk of 32 keys travels to the lanes.  A wave's 16-byte loads are
// served four neighbouring lanes at a time; neighbours in an operand are
// different keys, so loading operands directly takes an access of the vector
// cache for each 16 bytes (777 rows over the 16-bit pool, D = 64: 59 million).
// Staged chunks are copied by neighbours along a key's row (20 million)
// straight into a buffer of the wave's own in LDS, two chunks in flight, and
// the operands read from there: 122 -> 117 us there, 22.4 -> 21.6 (19.6 now) for 64 decode
// rows of a 4,096 window (4-bit, D = 128), and 40 registers fewer.  The 16-bit
// pools are staged at D = 64 only: larger chunks would leave LDS for too few
// waves.  The 8-bit cache leaves two a SIMD at D = 128: 64 x 6 rows of 2,051 slots
// 75 us, 79 unstaged; with one buffer and three waves 67, but then 512 rows take 66
// for 53, and 64 x 6 windows of 4,000 130 for 68 (they spill).
//
// A buffer holds the rows of the 32 keys (4-bit and 8-bit: K and V codes, which
// lie together, then the scales; 16-bit: K, then V), their 16-byte pieces XOR-ed
// with a function of the key that spreads the operands' reads over the banks.
template <int FORM, int D>
struct Staging {
  static constexpr bool kUsed = FORM != kForm16 || D == 64;
  static constexpr int kRow = FORM == kForm4 ? D : 2 * D, kArrays = FORM == kForm16 ? 2 : 1;
  static constexpr int kLanes = kRow / 16, kKeysPerCopy = 64 / kLanes, kCopies = kGaKeys / kKeysPerCopy;
  static constexpr int kScaleBytes = FORM == kForm4 ? D / 16 : FORM == kForm8 ? 8 : 0;  // of a key
  static constexpr int kScales = kArrays * kGaKeys * kRow, kBytes = kScales + kGaKeys * kScaleBytes;
  static constexpr int kInFlight = kArrays * kCopies + (FORM != kForm16 ? 1 : 0);  // copy instructions a chunk
  static __device__ __forceinline__ int swizzle(int key) {
    if (FORM == kForm8 && kRow >= 256) return key & 15;
    return kRow == 64 ? key >> 2 & 3 : kRow == 128 ? (key >> 1 & 3) | (key & 4) : key & 7;
  }
  static __device__ __forceinline__ const uint8_t* at(const uint8_t* buf, int key, int byte) {
    return buf + key * kRow + (((byte >> 4) ^ swizzle(key)) << 4) + (byte & 15);
  }
};

// Copies 16 (4) bytes a lane from p to LDS address lds + 16 (4) * lane, counted
// by vmcnt.  Written as assembly so that the compiler does not wait for every
// copy in flight before the next LDS read; the kernel waits by count.
__device__ __forceinline__ void copy_to_lds16(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void copy_to_lds4(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(p), "s"(lds) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Waves a SIMD must hold.  One where the registers of two would spill in the
// loop (the 16-bit loads of two chunks take 256 at D = 256; one such wave keeps
// 64 KiB in flight): 64 decode rows of 2,051 slots, D = 256, 16-bit pool 60 us,
// 131 with two.  Four where two registers decide between three and four: 1,024
// rows of 2,051 slots, 4-bit, D = 128: 71 us, 75 with three.
constexpr int gather_waves(int form, int d, int nt, bool window) {
  return nt * d == 256 && form != kForm4 ? 1 : form == kForm4 && nt * d == 128 && !window ? 4 : 2;
}

template <class T, int FORM, int D, int NT, bool WINDOW>
__global__ __launch_bounds__(64 * kGaWaves, gather_waves(FORM, D, NT, WINDOW)) void attn_gather_kernel(const GatherArgs a) {
  constexpr bool FP4 = FORM == kForm4, FP8 = FORM == kForm8;
  typedef GatherRaw<FORM, D> Raw;
  typedef Staging<FORM, D> Stage;
  constexpr int KS = D / 32;       // 32-channel steps of the score product
  constexpr int VD = D / 16;       // channels of the output per lane and accumulator row
  constexpr int COLS = 16 * NT;    // (row, head) pairs of a tile
  constexpr int OLD = D + 4;       // LDS row of the join, in floats
  __shared__ union {
    struct {
      __attribute__((aligned(16))) uint64_t at[kGaWaves][kGaKeys];  // byte offsets of a chunk's keys
      __attribute__((aligned(16))) uint8_t buf[kGaWaves][2][Stage::kUsed ? Stage::kBytes : 16];
      __attribute__((aligned(16))) int32_t id[kGaWaves][kGaKeys];   // slots or pages of the chunk after
    } st;
    struct {
      __attribute__((aligned(16))) float o[kGaWaves][16][OLD];
      float m[kGaWaves][16];
      Sums l[kGaWaves][16];
    } jn;
  } sh;
  __shared__ uint32_t arrived;

  const int tid = threadIdx.x, lane = tid & 63, n16 = lane & 15, qd = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Grid: row tiles, head blocks, splits; so the chip works on one kv head at a
  // time, whose keys then come from a cache more often.
  const int split = blockIdx.z, hb = blockIdx.y, bx = blockIdx.x;
  const int tile = a.xcd_rows ? bx / 64 * 64 + bx % 8 * 8 + bx / 8 % 8 : bx;
  if (tile >= a.tiles) return;
  const uint32_t group = (uint32_t)hb * a.tiles + tile;
  const int kvh = hb / a.hblocks, G = a.hq / a.hkv, hin = (hb % a.hblocks) * a.gb;
  const int heads = min(a.gb, G - hin), h0 = kvh * G + hin;

  // The tile's rows, and its key list: n keys.
  int row0, nrows, n;
  // Window: positions of the rows that have one, first keys, where the window
  // starts, and the last position that every row of the tile sees.
  int tmin = 0, tmax = 0, ns = 0, start = 0, seen_by_all = 0;
  const int32_t* ptab = nullptr;
  if constexpr (WINDOW) {
    const int b = tile / a.tiles_per_req, i = tile % a.tiles_per_req;
    const int ra = max(a.req_row_ptr[b], 0);
    const int rb = (int)min((int64_t)min(a.req_row_ptr[b + 1], a.num_rows), (int64_t)ra + a.max_rows);
    const int64_t first = (int64_t)ra + (int64_t)i * a.rows_per_tile;
    if (first >= rb) return;
    row0 = (int)first;
    nrows = min(a.rows_per_tile, rb - row0);
    ptab = a.page_table + (int64_t)b * a.pt_stride;
    const int t = a.row_pos[row0 + min(lane, nrows - 1)];
    int lo = t < 0 ? 0x7FFFFFFF : t, hi = t;
    for (int o = 32; o > 0; o >>= 1) lo = min(lo, __shfl_xor(lo, o)), hi = max(hi, __shfl_xor(hi, o));
    tmin = __builtin_amdgcn_readfirstlane(lo), tmax = __builtin_amdgcn_readfirstlane(hi);
    seen_by_all = ballot(t < 0) ? -1 : tmin;  // a row without a position sees nothing
    // last addressable position (and its chunk's keys stay below 2^31)
    const int last = (int)min((int64_t)min(tmax, 0x7FFFFF00), (int64_t)a.pt_stride * kPage - 1);
    ns = max(0, min(a.sinks, last + 1));
    start = max(max(0, tmin - a.window + 1), ns);
    n = last < 0 ? 0 : ns + max(0, last + 1 - start);
  } else {
    row0 = tile, nrows = 1;
    n = a.ld_slots;
  }
  const uint32_t chunks = ((uint32_t)n + kGaKeys - 1) / kGaKeys;
  const int c0 = part_start(chunks, a.nsplit, split);
  int c1 = part_start(chunks, a.nsplit, split + 1);
  const int n_listed = n;

  // The 8 channels of step ks of the score product in this lane's quarter of
  // the wave (their order is free): those that its 16-byte loads of a key hold,
  // which four quarters make 64 contiguous bytes.
  auto channel = [&](int ks) {
    if constexpr (FP8) return 64 * (ks / 2) + 16 * qd + 8 * (ks % 2);
    return !FP4 ? 32 * ks + 8 * qd : D == 64 ? 16 * qd + 8 * ks : 128 * (ks / 4) + 32 * qd + 8 * (ks % 4);
  };
  // This lane's query vectors (column 16*nt + n16 of the tile).
  u32x4_t qf[NT][KS];
  int tcol[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int col = nt * 16 + n16, rr = col / a.gb, hh = col % a.gb;
    const bool ok = rr < nrows && hh < heads;
    const typename T::elem* src =
        static_cast<const typename T::elem*>(a.q) + (int64_t)(row0 + (ok ? rr : 0)) * a.ld_q + (h0 + (ok ? hh : 0)) * D;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const u32x4_t x = *reinterpret_cast<const u32x4_t*>(src + channel(ks));
      qf[nt][ks] = ok ? x ^ a.flip : u32x4_t{0, 0, 0, 0};
    }
    tcol[nt] = WINDOW && ok ? a.row_pos[row0 + rr] : -1;
  }

  f32x4_t acc[NT][VD];
  float m[NT];
  Sums l[NT];
  uint64_t huge = 0;  // of lanes with a maximum past kHugeScore
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = -INFINITY, l[nt] = Sums{0.f, 0.f};
#pragma unroll
    for (int d = 0; d < VD; ++d) acc[nt][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }

  auto key_pos = [&](int i) { return i < ns ? i : start + (i - ns); };
  // The slot of this lane's key (lane mod 32) of chunk c; -1: none.
  auto load_slot = [&](int c) -> int {
    const uint32_t i = (uint32_t)c * kGaKeys + (lane & 31);  // unsigned: up to two steps past a list of almost 2^31
    if (c >= c1 || i >= (uint32_t)n) return -1;
    if constexpr (WINDOW) {
      const int p = key_pos((int)i);
      const int page = ptab[p >> 6];
      return page < 0 || page > (0x7FFFFFFF >> 6) ? -1 : page * kPage + (p & (kPage - 1));
    } else {
      return a.slots[(int64_t)row0 * a.ld_slots + i];
    }
  };
  // A key's byte offset is computed by one lane and read by those that load from
  // it; mask: the keys whose slot is one.
  auto put_offsets = [&](int sl, uint32_t& mask) {
    const bool ok = sl >= 0 && sl < a.num_slots;
    mask = (uint32_t)ballot(ok);
    const uint32_t rec = FP4 ? (uint32_t)a.hkv * D : FP8 ? (uint32_t)a.hkv * 2 * D : (uint32_t)a.ld_kv * 2;
    wave_fence();
    if (lane < kGaKeys) sh.st.at[wave][lane] = (uint64_t)(uint32_t)(ok ? sl : 0) * rec;
    wave_fence();
  };
  // Not staged (16-bit): issues the loads of a chunk.
  auto fetch = [&](int sl, Raw& r, uint32_t& mask) {
    put_offsets(sl, mask);
    const uint64_t* ls = sh.st.at[wave];
    uint64_t va[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const ulonglong2 x = reinterpret_cast<const ulonglong2*>(ls)[(j >> 2) * 8 + 2 * qd + (j >> 1 & 1)];
      va[j] = x.x, va[j + 1] = x.y;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint8_t* p = a.a + kvh * 2 * D + qd * 16 + ls[16 * j + n16];
#pragma unroll
      for (int i = 0; i < Raw::kKDwords; i += 4) load_4dwords(&r.k[j][i], p + 16 * i);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) load_dwords(r.v[j], a.b + kvh * 2 * D + n16 * (D / 8) + va[j]);
  };

  // Staged chunks: the copies of a chunk's slot (window: page) numbers, which
  // are clamped to the list; its keys' slots once they are there; the copies of
  // its rows; the operands out of the buffer.
  const uint32_t lds_buf = lds_address(sh.st.buf[wave][0]), lds_id = lds_address(sh.st.id[wave]);
  auto copy_ids = [&](int c) {
    // Unsigned: two steps past a list of almost 2^31 entries.
    const int i = (int)min((uint32_t)c * kGaKeys + lane, (uint32_t)n_listed - 1);
    const int32_t* p = WINDOW ? ptab + (key_pos(i) >> 6) : a.slots + (int64_t)row0 * a.ld_slots + i;
    if (lane < kGaKeys) copy_to_lds4(p, lds_id);
  };
  auto staged_slot = [&](int c) -> int {
    const uint32_t i = (uint32_t)c * kGaKeys + (lane & 31);
    const int x = sh.st.id[wave][lane & 31];
    if (c >= c1 || i >= (uint32_t)n) return -1;
    if constexpr (WINDOW) return x < 0 || x > (0x7FFFFFFF >> 6) ? -1 : x * kPage + (key_pos((int)i) & (kPage - 1));
    return x;
  };
  auto copy_rows = [&](int sl, int buf, uint32_t& mask) {
    put_offsets(sl, mask);
    uint32_t page_of = 0;
    if constexpr (FP8) {
      const uint32_t x = __shfl(sl, lane >> 1);
      page_of = x < (uint32_t)a.num_slots ? x : 0;
    }
    const uint64_t* ls = sh.st.at[wave];
    const uint32_t dst = lds_buf + buf * Stage::kBytes;
    // The buffer's last operands have been read, and so have the slot numbers.
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < Stage::kCopies; ++i) {
      const int key = i * Stage::kKeysPerCopy + lane / Stage::kLanes;
      const uint64_t at = ls[key] + kvh * Stage::kRow + ((lane % Stage::kLanes) ^ Stage::swizzle(key)) * 16;
      copy_to_lds16(a.a + at, dst + i * 1024);
      if constexpr (FORM == kForm16) copy_to_lds16(a.b + at, dst + kGaKeys * Stage::kRow + i * 1024);
    }
    if constexpr (FP8)  // the scales of each key's page: a lane's is K's or V's
      copy_to_lds4(a.b + ((uint64_t)(page_of >> 6) * a.hkv + kvh) * 8 + (lane & 1) * 4, dst + Stage::kScales);
    if constexpr (FP4) {
      const uint8_t* sc = a.b + kvh * (D / 16);
      if constexpr (D == 64) {
        const uint8_t* p = sc + (ls[lane & 31] >> 4);
        if (lane < kGaKeys) copy_to_lds4(p, dst + Stage::kScales);
      } else if constexpr (D == 128) {
        copy_to_lds4(sc + (ls[lane >> 1] >> 4) + (lane & 1) * 4, dst + Stage::kScales);
      } else {
        const uint8_t* p = sc + (ls[lane & 31] >> 4);
        if (lane < kGaKeys) copy_to_lds16(p, dst + Stage::kScales);
      }
    }
  };
  auto read_rows = [&](int buf, Raw& r) {
    const uint8_t* rows = sh.st.buf[wave][buf];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int key = 16 * j + n16;
      if constexpr (FP4 && D == 64) {
        load_dwords(r.k[j], Stage::at(rows, key, qd * 8));
      } else {
#pragma unroll
        for (int i = 0; i < Raw::kKDwords; i += 4) load_4dwords(&r.k[j][i], Stage::at(rows, key, 16 * i + qd * 16));
      }
    }
    const uint8_t* v = FORM != kForm16 ? rows : rows + kGaKeys * Stage::kRow;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint8_t* p = Stage::at(v, (j >> 2) * 16 + 4 * qd + (j & 3),
                                   FP4 ? D / 2 + n16 * (D / 32) : FP8 ? D + n16 * (D / 16) : n16 * (D / 8));
      if constexpr (FP4 && D == 64)
        r.v[j][0] = *reinterpret_cast<const uint16_t*>(p);
      else
        load_dwords(r.v[j], p);
    }
  };

  auto compute = [&](Raw& r, uint32_t mask, int c, int buf) {
    float vscale[8];
    float kscale[2][FP4 && D == 256 ? 2 : 1];
    bool full = mask == 0xFFFFFFFFu;
    if constexpr (FP4) {
      const uint8_t* sc = sh.st.buf[wave][buf] + Stage::kScales;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint8_t* p = sc + (16 * j + n16) * (D / 16);
        if constexpr (D == 256) {
          kscale[j][0] = kv4_scale(p[qd]), kscale[j][1] = kv4_scale(p[4 + qd]);
        } else {
          kscale[j][0] = kv4_scale(p[qd * D / 128]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        vscale[j] = kv4_scale(sc[((j >> 2) * 16 + 4 * qd + (j & 3)) * (D / 16) + D / 32 + n16 * D / 512]);
    }
    if constexpr (FP8) {
      const float* sc = reinterpret_cast<const float*>(sh.st.buf[wave][buf] + Stage::kScales);
#pragma unroll
      for (int j = 0; j < 2; ++j) kscale[j][0] = sc[2 * (16 * j + n16)];
#pragma unroll
      for (int j = 0; j < 8; ++j) vscale[j] = sc[2 * ((j >> 2) * 16 + 4 * qd + (j & 3)) + 1];
    }
    // Keys without a slot: their K is read from slot 0 and masked below,
    // their V must be zeros (0 * NaN is not 0).
    // Bit j: is there a key of v[j]?  (Opaque, or its eight tests move in front
    // of the branches that need them.)
    auto have = [&] {
      uint32_t b = ((mask >> (4 * qd)) & 0xFu) | (((mask >> (16 + 4 * qd)) & 0xFu) << 4);
      asm volatile("" : "+v"(b));
      return b;
    };
    if (!full) {
      const uint32_t there = have();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool ok = (there >> j) & 1u;
#pragma unroll
        for (int i = 0; i < Raw::kVDwords; ++i) r.v[j][i] = ok ? r.v[j][i] : 0u;
        if constexpr (FP4 || FP8) vscale[j] = ok ? vscale[j] : 1.f;
      }
    }

    f32x4_t s[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    static_for<KS>([&](auto ksc) {
      constexpr int ks = decltype(ksc)::value;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        u32x4_t kf;
        if constexpr (FP4) {
          const float sc = kscale[j][D == 256 ? ks / 4 : 0];
          const uint32_t w = r.k[j][ks];
          kf = u32x4_t{T::template from_fp4<0>(w, sc), T::template from_fp4<1>(w, sc), T::template from_fp4<2>(w, sc),
                       T::template from_fp4<3>(w, sc)};
        } else if constexpr (FP8) {
          const float sc = kscale[j][0];
          const uint32_t w0 = r.k[j][2 * ks], w1 = r.k[j][2 * ks + 1];
          kf = u32x4_t{T::template from_fp8<0>(w0, sc), T::template from_fp8<1>(w0, sc), T::template from_fp8<0>(w1, sc),
                       T::template from_fp8<1>(w1, sc)};
        } else {
          kf = u32x4_t{r.k[j][4 * ks], r.k[j][4 * ks + 1], r.k[j][4 * ks + 2], r.k[j][4 * ks + 3]};
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][j] = T::mfma16(kf, qf[nt][ks], s[nt][j]);
      }
    });

    // Which of the lane's 8 keys each query vector sees.
    uint32_t vis[NT];
    int pk[8];
    bool masked = !full;
    if constexpr (WINDOW) {
      const int pf = key_pos(c * kGaKeys), pl = key_pos(min(c * kGaKeys + kGaKeys - 1, n - 1));
      masked = masked || pl > seen_by_all || !(pf > tmax - a.window || pl < a.sinks);
      if (masked) {
#pragma unroll
        for (int j = 0; j < 8; ++j) pk[j] = key_pos(c * kGaKeys + (j >> 2) * 16 + 4 * qd + (j & 3));
      }
    }
    u32x4_t pfr[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = s[nt][j >> 2][j & 3];
      if (masked) {
        vis[nt] = have();
        if constexpr (WINDOW) {
          const int t = tcol[nt];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (!(pk[j] <= t && (pk[j] > t - a.window || pk[j] < a.sinks))) vis[nt] &= ~(1u << j);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[j] = __uint_as_float(bit_select(bit_mask(vis[nt], j), __float_as_uint(x[j]), 0xFF800000u));
      }
      float mx = x[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) mx = max_nan(mx, x[j]);
      mx = rounded_product(rows_max(mx), a.scale_log2);
      if (ballot(mx - m[nt] > kSlack)) {
        mx = fmaxf(m[nt], mx);
        const float f = exp2_fast(m[nt] - finite_max(mx));
        l[nt] *= f;
#pragma unroll
        for (int d = 0; d < VD; ++d) acc[nt][d] *= f;
        m[nt] = mx;
        huge |= ballot(fabsf(finite_max(mx)) > kHugeScore);
      }
      float scale = a.scale_log2, base = finite_max(m[nt]);  // of the weights
      if (huge) {  // apart from the branch above, which then copied the accumulators (3 to 5% at D = 256)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = rounded_product(x[j], scale) - base;
        scale = 1.f, base = 0.f;
      }
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = exp2_fast(__builtin_fmaf(x[j], scale, T::kRaise - base));
      l[nt].x += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
      pfr[nt] = u32x4_t{T::pack(p[0], p[1]), T::pack(p[2], p[3]), T::pack(p[4], p[5]), T::pack(p[6], p[7])};
      l[nt].y = add_rounded<T>(pfr[nt], l[nt].y);
    }

    // A key that some rows of the tile see and others do not may hold
    // infinities or NaN: 0 * inf is NaN, so those go a way of their own.
    bool fix = false;
    if constexpr (WINDOW) {
      if (masked) {
        uint32_t bad = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (FP4) {
            bad |= vscale[j] > T::kTopScale;
          } else if constexpr (FP8) {
            bad |= vscale[j] > T::kTopScale8;
#pragma unroll
            for (int i = 0; i < Raw::kVDwords; ++i) bad |= kv8_nan_codes(r.v[j][i]);
          } else {
#pragma unroll
            for (int i = 0; i < Raw::kVDwords; ++i) bad |= nonfinite_pair<T>(r.v[j][i]);
          }
        }
        fix = ballot(bad != 0) != 0;
      }
    }
    auto v_pair = [&](auto pic, u32x4_t& f0, u32x4_t& f1) {
      constexpr int pi = decltype(pic)::value;
      uint32_t two[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (FP4)
          two[j] = T::template from_fp4<pi % 4>(r.v[j][pi / 4], vscale[j]);
        else if constexpr (FP8)
          two[j] = T::template from_fp8<pi % 2>(r.v[j][pi / 2], vscale[j]);
        else
          two[j] = r.v[j][pi];
      }
      f0 = u32x4_t{pair_lo(two[0], two[1]), pair_lo(two[2], two[3]), pair_lo(two[4], two[5]), pair_lo(two[6], two[7])};
      f1 = u32x4_t{pair_hi(two[0], two[1]), pair_hi(two[2], two[3]), pair_hi(two[4], two[5]), pair_hi(two[6], two[7])};
    };
    if (!fix) {
      static_for<VD / 2>([&](auto pic) {
        constexpr int pi = decltype(pic)::value;
        u32x4_t f0, f1;
        v_pair(pic, f0, f1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[nt][2 * pi] = T::mfma16(f0, pfr[nt], acc[nt][2 * pi]);
          acc[nt][2 * pi + 1] = T::mfma16(f1, pfr[nt], acc[nt][2 * pi + 1]);
        }
      });
    } else {
      static_for<VD / 2>([&](auto pic) {
        constexpr int pi = decltype(pic)::value;
        u32x4_t f[2];
        v_pair(pic, f[0], f[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          u32x4_t clean, marks;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            clean[i] = f[e][i] & ~spread_halves(nonfinite_pair<T>(f[e][i]));
            marks[i] = nonfinite_marks<T>(f[e][i]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            u32x4_t see;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              see[i] = (bit_mask(vis[nt], 2 * i) & T::kOne) | (bit_mask(vis[nt], 2 * i + 1) & (T::kOne << 16));
            const f32x4_t cnt = T::mfma16(marks, see, f32x4_t{0.f, 0.f, 0.f, 0.f});
            f32x4_t o = T::mfma16(clean, pfr[nt], acc[nt][2 * pi + e]);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] += nonfinite_term(cnt[i]);
            acc[nt][2 * pi + e] = o;
            __builtin_amdgcn_sched_barrier(0);  // one channel at a time: this path is rare, its registers are not
          }
        }
      });
    }
  };

  // Chunks c0 + wave, + 4, ...  A list's splits go by its storage, so that its
  // first entries are on their way before its count is known.
  int c = c0 + wave;
  auto count = [&] {
    if constexpr (!WINDOW)
      if (a.count != nullptr) n = max(min(n, a.count[row0]), 0), c1 = min(c1, (int)(((uint32_t)n + kGaKeys - 1) / kGaKeys));
  };
  if constexpr (Stage::kUsed) {
    if (c < c1) {
      copy_ids(c);
      count();
      wait_vmcnt<0>();  // the builtin: it also tells the compiler that q is there
      asm volatile("" ::: "memory");
      if (c < c1) {
        uint32_t kc, kn = 0;
        int buf = 0;
        const int sl = staged_slot(c);
        wave_fence();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        copy_ids(c + kGaWaves);
        copy_rows(sl, 0, kc);
        for (;;) {
          const bool more = c + kGaWaves < c1;
          if (more) {
            wait_copies<Stage::kInFlight>();  // the next chunk's slot numbers
            const int sn = staged_slot(c + kGaWaves);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            copy_ids(c + 2 * kGaWaves);
            copy_rows(sn, buf ^ 1, kn);
            wait_copies<Stage::kInFlight + 1>();  // this chunk's rows
          } else {
            wait_copies<0>();
          }
          Raw r;
          read_rows(buf, r);
          compute(r, kc, c, buf);
          if (!more) break;
          c += kGaWaves, kc = kn, buf ^= 1;
        }
      }
    }
  } else {
    // The loads of the next chunk are issued before this one's products, its
    // slots one chunk earlier still.
    int sl0 = load_slot(c), sl = load_slot(c + kGaWaves);
    count();
    const uint32_t i = (uint32_t)c * kGaKeys + (lane & 31);
    sl0 = i < (uint32_t)n ? sl0 : -1;
    sl = i + kGaWaves * kGaKeys < (uint32_t)n ? sl : -1;
    if (c < c1) {
      Raw r0, r1;
      uint32_t k0, k1;
      fetch(sl0, r0, k0);
      auto step = [&](Raw& cur, uint32_t& kc, Raw& nxt, uint32_t& kn) {
        if (c + kGaWaves < c1) {
          fetch(sl, nxt, kn);
          sl = load_slot(c + 2 * kGaWaves);
        }
        compute(cur, kc, c, 0);
        c += kGaWaves;
        return c < c1;
      };
      while (step(r0, k0, r1, k1) && step(r1, k1, r0, k0)) {
      }
    }
  }

  // Join the waves, 16 columns at a time.  Thread (col, part) owns channels
  // part*VD .. +VD of its column.
  const int col = tid >> 4, part = tid & 15;
  const uint32_t slot_floats = COLS * (D + 4);
  const SplitBuffer sb(a.partial, a.nsplit > 1 ? (uint32_t)((uint32_t)a.tiles * gridDim.y * a.nsplit * slot_floats * 4u) : 0u);
  auto finish = [&](int nt, const float (&o)[VD], float mm, const Sums& ll) {
    const int cc = nt * 16 + col, rr = cc / a.gb, hh = cc % a.gb;
    if (rr >= nrows || hh >= heads) return;
    const float inv = ll.y == 0.f ? 0.f : 1.f / ll.y;
    typename T::elem* dst = static_cast<typename T::elem*>(a.out) + (int64_t)(row0 + rr) * a.ld_out + (h0 + hh) * D + part * VD;
    uint32_t w[VD / 2];
#pragma unroll
    for (int i = 0; i < VD / 2; ++i) w[i] = T::pack(o[2 * i] * inv, o[2 * i + 1] * inv);
    if constexpr (VD == 4) {
      *reinterpret_cast<u32x2_t*>(dst) = u32x2_t{w[0], w[1]};
    } else {
#pragma unroll
      for (int i = 0; i < VD / 2; i += 4) *reinterpret_cast<u32x4_t*>(dst + 2 * i) = u32x4_t{w[i], w[i + 1], w[i + 2], w[i + 3]};
    }
    if (a.lse != nullptr && part == 0)
      a.lse[(int64_t)(row0 + rr) * a.hq + h0 + hh] = row_lse<T>(mm, ll.x);
  };
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const Sums ls = {rows_sum(l[nt].x), rows_sum(l[nt].y)};
    __syncthreads();
    if (qd == 0) sh.jn.m[wave][n16] = m[nt], sh.jn.l[wave][n16] = ls;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int d = 0; d < VD; d += 4)
        *reinterpret_cast<f32x4_t*>(&sh.jn.o[wave][n16][VD * (4 * qd + i) + d]) =
            f32x4_t{acc[nt][d][i], acc[nt][d + 1][i], acc[nt][d + 2][i], acc[nt][d + 3][i]};
    __syncthreads();
    float mm = -INFINITY, o[VD];
    Sums ll = {0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kGaWaves; ++w) mm = fmaxf(mm, sh.jn.m[w][col]);
#pragma unroll
    for (int d = 0; d < VD; ++d) o[d] = 0.f;
#pragma unroll
    for (int w = 0; w < kGaWaves; ++w) {
      const float f = exp2_fast(sh.jn.m[w][col] - finite_max(mm));
      ll += sh.jn.l[w][col] * f;
#pragma unroll
      for (int d = 0; d < VD; ++d) o[d] += sh.jn.o[w][col][part * VD + d] * f;
    }
    if (a.nsplit == 1) {
      finish(nt, o, mm, ll);
    } else {
      if (nt * 16 + col >= nrows * a.gb) continue;  // no such column
      const uint32_t base = (group * a.nsplit + split) * slot_floats * 4;
#pragma unroll
      for (int d = 0; d < VD; d += 4)
        sb.store4(base + ((nt * 16 + col) * D + part * VD + d) * 4, f32x4_t{o[d], o[d + 1], o[d + 2], o[d + 3]});
      if (part == 0) sb.store4(base + (COLS * D + 4 * (nt * 16 + col)) * 4, f32x4_t{mm, ll.x, ll.y, 0.f});
    }
  }
  if (a.nsplit == 1) return;

  if (!last_of_group(a.counters, group, a.nsplit, tid, arrived)) return;
  join_splits<D, 64 * kGaWaves, COLS>(sb, group * a.nsplit * slot_floats * 4, slot_floats * 4, min(nrows * a.gb, COLS),
                                      a.nsplit, tid, [&](int cc, int d, const f32x4_t& o, float mm, const Sums& ll) {
    const int rr = cc / a.gb, hh = cc % a.gb;
    if (hh < heads)
      write_joined<T>(static_cast<typename T::elem*>(a.out) + (int64_t)(row0 + rr) * a.ld_out + (h0 + hh) * D, d, o, mm, ll,
                      a.lse == nullptr ? nullptr : a.lse + (int64_t)(row0 + rr) * a.hq + h0 + hh);
  });
}

// nt: column tiles of a workgroup, 1 or (head_dim up to 128: registers) 2.
template <class T, int FORM>
int launch_attn_gather(const GatherArgs& a, int d, int nt, bool window, hipStream_t stream) {
  const dim3 grid(a.xcd_rows ? (a.tiles + 63) / 64 * 64 : a.tiles, a.hkv * a.hblocks, a.nsplit);
  auto go = [&](auto dim, auto tiles, auto win) {
    hipLaunchKernelGGL((attn_gather_kernel<T, FORM, decltype(dim)::value, decltype(tiles)::value, decltype(win)::value>),
                       grid, dim3(64 * kGaWaves), 0, stream, a);
  };
  auto by_window = [&](auto dim, auto tiles) {
    if (window)
      go(dim, tiles, std::true_type());
    else
      go(dim, tiles, std::false_type());
  };
  auto by_tiles = [&](auto dim) {
    if constexpr (decltype(dim)::value <= 128)
      if (nt == 2) return by_window(dim, std::integral_constant<int, 2>());
    by_window(dim, std::integral_constant<int, 1>());
  };
  if (d == 64)
    by_tiles(std::integral_constant<int, 64>());
  else if (d == 128)
    by_tiles(std::integral_constant<int, 128>());
  else
    by_tiles(std::integral_constant<int, 256>());
  return hipGetLastError() == hipSuccess ? BS_OK : BS_ERR_LAUNCH;
}

}  // namespace bs
