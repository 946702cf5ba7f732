// score4.hip - block scores over the 4-bit index keys, on the scaled matrix
// instructions.
//
// The same equation as the 16-bit scorers (page "Qwen3.8-Flash-Next Day-0 in
// SGLang", QSA section), with both operands microscaled: query heads are
// quantised by the call, 32 channels a scale, as the keys were when they were
// stored, and v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 head-rows by 16
// keys over all 128 channels in one instruction.  Codes, exponents and the
// products of a group of 32 are exact; sums are FP32.
//
// Operands as stored: lane l holds 32 channels (16 bytes), group l/16, of
// head-row or key l mod 16, and one exponent byte for them, which is the layout
// of a key's 64 bytes of codes and 4 of exponents.  The A operand holds 4 query
// rows, their 4 heads on adjacent rows, so a lane's 4 accumulators are the heads
// of one (query row, key) pair: ReLU, head sum and scale stay in the lane.
//
// Few rows a request (decode, verify): a stream of 68 bytes a key, bound by HBM.
// A wave takes TILES tiles of 64 keys, all of their loads in flight at once, and
// runs the request's rows over them.  Many rows (prefill): 1,024 flop and 4
// bytes written a (row, key) pair, bound by the writes.  A workgroup copies a
// chunk of keys into LDS, each of its waves holds its own rows' operands, and
// the chunk is gone through without waiting for anything but LDS.
#include <algorithm>

#include "idx4.h"
#include "kernels.h"

namespace bs {

namespace {

typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
typedef f32x4_t f32x4_unaligned_t __attribute__((aligned(4)));

constexpr int kTile = 64;       // keys
constexpr int kScoreWaves = 4;  // of a workgroup
constexpr int kChunkTiles = 8;  // prefill: keys in LDS

struct ScoreArgs {
  const uint16_t* q;
  const uint8_t *codes, *scales;
  int32_t num_pages;
  const int32_t* page_table;
  int32_t pt_stride;
  const int32_t *req_row_ptr, *row_pos;
  int32_t num_rows, max_vis;
  float* scores;
  int64_t ld;
  int32_t* row_len;
};

// 4 query rows as an operand.
struct Query {
  u32x4_t codes;
  uint32_t exponent;
  // Lane l: 32 channels of head l mod 4 of row `first` + l/4 mod 4 (at most `last`).
  __device__ __forceinline__ void load(const uint16_t* q, int first, int last, int lane) {
    const int m = lane & 15, row = min(first + (m >> 2), last);
    const uint16_t* p = q + ((int64_t)row * kHeads + (m & 3)) * kDim + (lane >> 4) * kGroup;
    Chunk<Bf16> x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i].load(p + 8 * i);
    bool bad;
    exponent = group_exponent(max(max(x[0].top(), x[1].top()), max(x[2].top(), x[3].top())), bad);
    const float s = kv4_scale(exponent);
#pragma unroll
    for (int i = 0; i < 4; ++i) codes[i] = bad ? 0u : x[i].codes(s);
    exponent = bad ? kExpNan : exponent;
  }
};

// The scores of one row with 16 keys: lane l has those of row l/16 and key l mod 16.  J: which byte of
// `exponents` is the keys'.
template <int J>
__device__ __forceinline__ float pair_score(const Query& q, const u32x4_t& k, uint32_t exponents) {
  // 4-bit operands are the first 4 registers of 8.
  auto wide = [](const u32x4_t& x) { return (i32x8_t)__builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1); };
  const f32x4_t x = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      wide(q.codes), wide(k), f32x4_t{0.f, 0.f, 0.f, 0.f}, 4, 4, 0, (int)q.exponent, J, (int)exponents);
  return ((fmaxf(x.x, 0.f) + fmaxf(x.y, 0.f)) + (fmaxf(x.z, 0.f) + fmaxf(x.w, 0.f))) * kScale;
}

// The rows of request b.
__device__ __forceinline__ void request_rows(const ScoreArgs& a, int b, int& r0, int& r1) {
  r0 = max(a.req_row_ptr[b], 0), r1 = min(a.req_row_ptr[b + 1], a.num_rows);
}

// Physical page of logical page i (page 0 where there is none: such scores are
// unspecified, and the read stays inside the cache).
__device__ __forceinline__ int page_at(const ScoreArgs& a, const int32_t* table, int i) {
  const int p = table[min(i, a.pt_stride - 1)];
  return p < 0 || p >= a.num_pages ? 0 : p;
}

// Byte g of four dwords, as the bytes of one.
__device__ __forceinline__ uint32_t gather_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t g) {
  const uint32_t sel = 0x0C0C0400u + g * 0x0101u;  // 0C: a zero
  return __builtin_amdgcn_perm(b, a, sel) | __builtin_amdgcn_perm(d, c, sel) << 16;
}

}  // namespace

// Few rows: RG groups of 4 rows at a time.
template <int C, int RG, int TILES>
__global__ __launch_bounds__(64 * kScoreWaves) void score4_decode_kernel(const ScoreArgs a) {
  constexpr int PAGE_KEYS = kPage / C;
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), b = blockIdx.y;
  int r0, r1;
  request_rows(a, b, r0, r1);
  if (blockIdx.x == 0 && a.row_len != nullptr)
    for (int r = r0 + tid; r < r1; r += 64 * kScoreWaves) a.row_len[r] = visible_blocks(a.row_pos[r], C, a.max_vis);
  const int64_t k0 = ((int64_t)blockIdx.x * kScoreWaves + wave) * (TILES * kTile);
  int most = 0;
  for (int r = r0 + lane; r < r1; r += 64) most = max(most, visible_blocks(a.row_pos[r], C, a.max_vis));
  for (int o = 32; o > 0; o >>= 1) most = max(most, __shfl_xor(most, o));
  most = __builtin_amdgcn_readfirstlane(most);
  if (k0 >= most) return;
  const int key0 = (int)k0;

  const int32_t* table = a.page_table + (int64_t)b * a.pt_stride;
  u32x4_t k[TILES][4];
  uint32_t sc[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    int page[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      page[j] = C == 4 ? page_at(a, table, key0 / PAGE_KEYS + t * 4 + j)
                       : j == 0 ? page_at(a, table, key0 / PAGE_KEYS + t) : page[0];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* p = a.codes + ((int64_t)page[j] * PAGE_KEYS + (C == 4 ? 0 : 16 * j)) * kIdxCodes;
      k[t][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + (n * kIdxCodes + g * 16)));
    }
    // Lane l: the exponents of key l of the tile.
    const int mine = C == 4 ? (g < 2 ? (g == 0 ? page[0] : page[1]) : (g == 2 ? page[2] : page[3])) : page[0];
    sc[t] = __builtin_nontemporal_load(
        reinterpret_cast<const uint32_t*>(a.scales + ((int64_t)mine * PAGE_KEYS + (C == 4 ? n : lane)) * kIdxScales));
  }
  for (int r = r0; r < r1; r += 4 * RG) {
    Query q[RG];
#pragma unroll
    for (int i = 0; i < RG; ++i) q[i].load(a.q, r + 4 * i, r1 - 1, lane);
    int vis[RG];
#pragma unroll
    for (int i = 0; i < RG; ++i) {
      const int row = r + 4 * i + g;
      vis[i] = row < r1 ? visible_blocks(a.row_pos[row], C, a.max_vis) : 0;
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      // Byte j: the exponent of this lane's group of key 16 * j + n.
      auto half = __builtin_amdgcn_permlane32_swap(sc[t], sc[t], false, false);
      auto lo = __builtin_amdgcn_permlane16_swap(half[0], half[0], false, false);
      auto hi = __builtin_amdgcn_permlane16_swap(half[1], half[1], false, false);
      const uint32_t e = gather_bytes(lo[0], lo[1], hi[0], hi[1], g);
#pragma unroll
      for (int i = 0; i < RG; ++i) {
        const float s[4] = {pair_score<0>(q[i], k[t][0], e), pair_score<1>(q[i], k[t][1], e),
                            pair_score<2>(q[i], k[t][2], e), pair_score<3>(q[i], k[t][3], e)};
        float* dst = a.scores + (int64_t)(r + 4 * i + g) * a.ld + key0 + t * kTile + n;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (key0 + t * kTile + 16 * j + n < vis[i]) dst[16 * j] = s[j];
      }
    }
  }
}

// Many rows: RG groups of 4 rows a wave, kChunkTiles tiles of keys a workgroup.
// In LDS the 16-byte pieces of 4 consecutive keys (256 bytes) are XOR-ed with
// their number, which spreads the operands' reads over the banks.
template <int C, int RG>
__global__ __launch_bounds__(64 * kScoreWaves) void score4_prefill_kernel(const ScoreArgs a) {
  constexpr int PAGE_KEYS = kPage / C, ROWS = 4 * RG * kScoreWaves;
  __shared__ __attribute__((aligned(16))) uint8_t codes[kChunkTiles][kTile * kIdxCodes];
  __shared__ __attribute__((aligned(16))) uint32_t exps[kChunkTiles * kTile];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), b = blockIdx.z;
  int r0, r1;
  request_rows(a, b, r0, r1);
  const int64_t k0 = (int64_t)blockIdx.x * (kChunkTiles * kTile);
  const int32_t* table = a.page_table + (int64_t)b * a.pt_stride;
  bool loaded = false;
  for (int64_t rb = r0 + (int64_t)blockIdx.y * ROWS; rb < r1; rb += (int64_t)gridDim.y * ROWS) {
    const int first = (int)rb, end = (int)min((int64_t)r1, rb + ROWS);
    if (blockIdx.x == 0 && a.row_len != nullptr)
      for (int r = first + tid; r < end; r += 64 * kScoreWaves) a.row_len[r] = visible_blocks(a.row_pos[r], C, a.max_vis);
    int most = 0;
    for (int r = first + lane; r < end; r += 64) most = max(most, visible_blocks(a.row_pos[r], C, a.max_vis));
    for (int o = 32; o > 0; o >>= 1) most = max(most, __shfl_xor(most, o));
    most = __builtin_amdgcn_readfirstlane(most);
    if (k0 >= most) continue;
    const int key0 = (int)k0;
    if (!loaded) {  // the same for every wave
      loaded = true;
#pragma unroll
      for (int t = 0; t < kChunkTiles; ++t) {
        // This wave's 16 keys of the tile, all in one page.
        const int page = page_at(a, table, C == 4 ? key0 / PAGE_KEYS + t * 4 + wave : key0 / PAGE_KEYS + t);
        const uint8_t* p = a.codes + ((int64_t)page * PAGE_KEYS + (C == 4 ? 0 : 16 * wave)) * kIdxCodes;
        const int row = lane >> 4, piece = (lane & 15) ^ (4 * wave + row);
        *reinterpret_cast<u32x4_t*>(&codes[t][wave * 1024 + lane * 16]) =
            *reinterpret_cast<const u32x4_t*>(p + (4 * row) * kIdxCodes + piece * 16);
      }
      for (int i = tid; i < kChunkTiles * kTile; i += 64 * kScoreWaves) {
        const int page = page_at(a, table, (key0 + i) / PAGE_KEYS);
        exps[i] = *reinterpret_cast<const uint32_t*>(a.scales + ((int64_t)page * PAGE_KEYS + (i & (PAGE_KEYS - 1))) * kIdxScales);
      }
      __syncthreads();
    }
    const int wr = first + wave * 4 * RG;
    if (wr >= end) continue;
    Query q[RG];
    int vis[RG];
    int all = 0x7FFFFFFF, any = 0;
#pragma unroll
    for (int i = 0; i < RG; ++i) {
      q[i].load(a.q, wr + 4 * i, end - 1, lane);
      const int row = wr + 4 * i + g;
      vis[i] = row < end ? visible_blocks(a.row_pos[row], C, a.max_vis) : 0;
      any = max(any, vis[i]), all = min(all, vis[i]);
    }
    for (int o = 32; o >= 16; o >>= 1) any = max(any, __shfl_xor(any, o)), all = min(all, __shfl_xor(all, o));
    any = __builtin_amdgcn_readfirstlane(any), all = __builtin_amdgcn_readfirstlane(all);
    float* const dst0 = a.scores + (int64_t)(wr + g) * a.ld + key0 + 4 * n;
    for (int t = 0; t < kChunkTiles && key0 + t * kTile < any; ++t) {
      u32x4_t k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const u32x4_t*>(&codes[t][n * 256 + (((4 * j + g) ^ n) * 16)]);
      const u32x4_t ex = *reinterpret_cast<const u32x4_t*>(&exps[t * kTile + 4 * n]);
      const uint32_t e = gather_bytes(ex.x, ex.y, ex.z, ex.w, g);
      auto rows = [&](auto masked_c) {
#pragma unroll
        for (int i = 0; i < RG; ++i) {
          const f32x4_t s = {pair_score<0>(q[i], k[0], e), pair_score<1>(q[i], k[1], e), pair_score<2>(q[i], k[2], e),
                             pair_score<3>(q[i], k[3], e)};
          float* dst = dst0 + (int64_t)(4 * i) * a.ld + t * kTile;
          const int left = decltype(masked_c)::value ? vis[i] - (key0 + t * kTile + 4 * n) : 4;
          if (left >= 4) {
            __builtin_nontemporal_store(s, reinterpret_cast<f32x4_unaligned_t*>(dst));
          } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
              if (j < left) dst[j] = s[j];
          }
        }
      };
      if (key0 + (t + 1) * kTile <= all)
        rows(std::false_type());
      else
        rows(std::true_type());
    }
  }
}

int launch_idx4_score(const uint16_t* q, const uint8_t* codes, const uint8_t* scales, int64_t num_pages,
                      const int32_t* page_table, int32_t pt_stride, const int32_t* req_row_ptr, int32_t num_req,
                      const int32_t* row_pos, int32_t num_rows, int32_t c, int32_t max_vis, float* scores, int64_t ld,
                      int32_t* row_len, hipStream_t stream) {
  const ScoreArgs a = {q,       codes,    scales,  (int32_t)num_pages, page_table, pt_stride, req_row_ptr,
                       row_pos, num_rows, max_vis, scores,             ld,         row_len};
  const int64_t keys = std::max(max_vis, 1), rows = (num_rows + (int64_t)num_req - 1) / num_req;  // of a request
  auto decode = [&](auto cc, auto rg, auto tiles) {
    constexpr int TILES = decltype(tiles)::value, CHUNK = kScoreWaves * TILES * kTile;
    hipLaunchKernelGGL((score4_decode_kernel<decltype(cc)::value, decltype(rg)::value, TILES>),
                       dim3((uint32_t)((keys + CHUNK - 1) / CHUNK), num_req), dim3(64 * kScoreWaves), 0, stream, a);
  };
  auto run = [&](auto cc) {
    if (rows > 8) {
      constexpr int RG = 8, ROWS = 4 * RG * kScoreWaves, CHUNK = kChunkTiles * kTile;
      const int64_t slices = std::min<int64_t>((rows + ROWS - 1) / ROWS, 65535);
      hipLaunchKernelGGL((score4_prefill_kernel<decltype(cc)::value, RG>),
                         dim3((uint32_t)((keys + CHUNK - 1) / CHUNK), (uint32_t)slices, num_req), dim3(64 * kScoreWaves), 0,
                         stream, a);
      return;
    }
    auto by_tiles = [&](auto rg) {
      if (num_req * keys >= 1024 * 256)
        decode(cc, rg, std::integral_constant<int, 4>());
      else
        decode(cc, rg, std::integral_constant<int, 1>());
    };
    if (rows <= 4)
      by_tiles(std::integral_constant<int, 1>());
    else
      by_tiles(std::integral_constant<int, 2>());
  };
  if (c == 4)
    run(std::integral_constant<int, 4>());
  else
    run(std::integral_constant<int, 1>());
  return hipGetLastError() == hipSuccess ? BS_OK : BS_ERR_LAUNCH;
}

}  // namespace bs
