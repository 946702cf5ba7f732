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
// Few rows a request (decode, verify): a stream of 68 bytes a key, bound by the
// latency of memory (16 rows x 81,920 keys, 94 MB: 18.1 us out of the Infinity Cache,
// 23.4 from HBM, 2 to 3 of them the timing's own).  A wave takes TILES tiles of 64
// keys, all of their loads in flight at once, and runs the request's rows over them.
// The grid is of max_vis keys for every request: 64 x 6 rows over 586,000 keys 15.2
// us, 22.2 with max_vis four times the longest request.  Many rows (prefill): 1,024 flop and 4
// bytes written a (row, key) pair, bound by the writes.  A workgroup copies a
// chunk of keys into LDS, each of its waves holds its own rows' operands, and
// the chunk is gone through without waiting for anything but LDS.
#include <algorithm>

#include "idx4.h"
#include "kernels.h"

namespace bs {

namespace {

typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
typedef f32x4_t f32x4_unaligned_t __attribute__((aligned(4)));

constexpr int kTile = 64;       // keys
constexpr int kScoreWaves = 4;  // of a workgroup

struct ScoreArgs {
  const uint16_t* q;
  const uint8_t *codes, *scales;
  int32_t num_pages;
  const int32_t* page_table;
  int32_t pt_stride;
  const int32_t *req_row_ptr, *row_pos;
  int32_t num_req, num_rows, max_vis;
  float* scores;
  int64_t ld;
  int32_t* row_len;
  int32_t more;  // blocks past the requests' first ones (few rows)
};

// 4 query rows as they are loaded: lane l has 32 channels of head l mod 4 of row
// `first` + l/4 mod 4 (at most `last`), and the length of row `first` + l/16.
struct Rows {
  Chunk<Bf16> x[4];
  int vis;
  template <int C>
  __device__ __forceinline__ void load(const ScoreArgs& a, int first, int last, int lane) {
    const int m = lane & 15, row = min(first + (m >> 2), last), mine = first + (lane >> 4);
    const uint16_t* p = a.q + ((int64_t)row * kHeads + (m & 3)) * kDim + (lane >> 4) * kGroup;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i].load(p + 8 * i);
    const int t = a.row_pos[min(mine, last)];
    vis = mine > last ? 0 : visible_blocks(t, C, a.max_vis);
  }
};

// 4 query rows as an operand.
struct Query {
  u32x4_t codes = {0, 0, 0, 0};
  uint32_t exponent = 0;
  Query() = default;
  __device__ __forceinline__ Query(const u32x4_t& c, uint32_t e) : codes(c), exponent(e) {}
  __device__ __forceinline__ explicit Query(const Rows& r) {
    // Bit patterns of |x| order like the values, two to a register.
    u16x2_t top = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2_t, r.x[i].v[j] & 0x7FFF7FFFu));
    bool bad;
    exponent = group_exponent((uint32_t)max(top.x, top.y) << 16, bad);
    const float s = kv4_scale(exponent);
    const uint32_t keep = bad ? 0u : ~0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) codes[i] = r.x[i].codes(s) & keep;
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
  // The median with 0 and infinity: ReLU, 0 for NaN, one instruction (a maximum,
  // which the compiler makes of it unless infinity is hidden, would first
  // quieten its operand).
  float top = INFINITY;
  asm("" : "+s"(top));
  auto relu = [&](float v) { return __builtin_amdgcn_fmed3f(v, 0.f, top); };
  float s = ((relu(x.x) + relu(x.y)) + (relu(x.z) + relu(x.w))) * kScale;
  // Matrix instructions take all lanes, whatever the lane mask, but what
  // prepares their operands does not: neither may move into a branch that only
  // some lanes take (the one around a store of the result, say).
  asm volatile("" : "+v"(s));
  return s;
}

// The rows of request b.
__device__ __forceinline__ void request_rows(const ScoreArgs& a, int b, int& r0, int& r1) {
  r0 = max(a.req_row_ptr[b], 0), r1 = min(a.req_row_ptr[b + 1], a.num_rows);
}

// Block `block` of up to ROWS rows of one request, the requests' blocks (from their FROM-th on) numbered one after the
// other: false if there is none.  Lane i looks at every 64th request.
template <int ROWS, int FROM>
__device__ __forceinline__ bool locate_rows(const ScoreArgs& a, uint32_t block, int lane, int& b, int& first, int& end) {
  for (int base = 0; base < a.num_req; base += 64) {
    int r0 = 0, r1 = 0;
    if (base + lane < a.num_req) request_rows(a, base + lane, r0, r1);
    const uint32_t blocks = r1 > r0 ? ((uint32_t)(r1 - r0) + ROWS - 1) / ROWS : 0u;
    const uint32_t upto = wave_incl_scan(blocks > FROM ? blocks - FROM : 0u), all = readlane(upto, 63);
    if (block < all) {
      const int i = __builtin_ctzll(ballot(upto > block));
      b = base + i, r0 = (int)readlane(r0, i), r1 = (int)readlane(r1, i);
      first = r0 + (int)(block - (i > 0 ? readlane(upto, i - 1) : 0u) + FROM) * ROWS;
      end = r1 - first < ROWS ? r1 : first + ROWS;
      return true;
    }
    block -= all;
  }
  return false;
}

// Physical page of logical page i >= 0 (page 0 where there is none: such scores are
// unspecified, and the read stays inside the cache).
__device__ __forceinline__ int page_at(const ScoreArgs& a, const int32_t* table, int i) {
  const int p = table[min(i, a.pt_stride - 1)];
  return p < 0 || p >= a.num_pages ? 0 : p;
}

// Byte g of four dwords, as the bytes of one.
__device__ __forceinline__ uint32_t gather_bytes(const u32x4_t& x, uint32_t g) {
  const uint32_t sel = 0x0C0C0400u + g * 0x0101u;  // 0C: a zero
  return __builtin_amdgcn_perm(x.y, x.x, sel) | __builtin_amdgcn_perm(x.w, x.z, sel) << 16;
}

// The largest of a wave's values, not below 0.
__device__ __forceinline__ int wave_most(int x) {
  for (int o = 32; o > 0; o >>= 1) x = max(x, __shfl_xor(x, o));
  return __builtin_amdgcn_readfirstlane(x);
}

// The scores of 4 rows with TILES tiles of keys from `key` on: lane l has those of row l/16 (which sees vis keys) with
// keys 4n .. 4n + 3 of each tile, n = l mod 16, and stores them at dst.  e, byte j: the exponents of k[..][j].
// Non-temporal: the selection reads the scores after the whole launch (8,192 rows: 96 us, 118 with cached stores).
template <int TILES>
__device__ __forceinline__ void store_scores(const Query& q, const u32x4_t (&k)[TILES][4], const uint32_t (&e)[TILES], float* dst,
                                             int vis, int key, int n) {
  auto tiles = [&](auto masked_c) {
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const f32x4_t s = {pair_score<0>(q, k[t][0], e[t]), pair_score<1>(q, k[t][1], e[t]), pair_score<2>(q, k[t][2], e[t]),
                         pair_score<3>(q, k[t][3], e[t])};
      float* p = dst + t * kTile;
      const int left = decltype(masked_c)::value ? vis - (key + t * kTile + 4 * n) : 4;
      if (left >= 4) {
        __builtin_nontemporal_store(s, reinterpret_cast<f32x4_unaligned_t*>(p));
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (j < left) p[j] = s[j];
      }
    }
  };
  if (ballot(vis >= key + TILES * kTile) == ~0ull)
    tiles(std::false_type());
  else
    tiles(std::true_type());
}

}  // namespace

// Rows of a block in the kernel for few rows: one block is of the first rows of each request, others of the rest of
// those that have more (63 requests of one row beside one of 1,000, 30,000 tokens each, c = 4: 20 to 22 us, 172 with a
// request's rows in one block).
constexpr int kRowsOnce = 64;

// Few rows a request: TILES tiles a wave, up to 64 rows.
//
// What a wave does before its first product takes about as long as the products:
// so page ids are one load (a lane a page: loads of one id for all lanes were
// scalar, waited for one by one), and the waves prepare the rows' operands for
// each other (64 requests x 6 rows over 586,000 keys of c = 4: 46 us with neither,
// 15.5 now).  With MFMA j of a tile taking keys 4n + j a lane stores 4 scores at
// once.
template <int C, int TILES>
__global__ __launch_bounds__(64 * kScoreWaves) void score4_decode_kernel(const ScoreArgs a) {
  constexpr int PAGE_KEYS = kPage / C, BATCH = kScoreWaves;
  __shared__ u32x4_t q_codes[BATCH][64];
  __shared__ uint32_t q_exponent[BATCH][64];
  __shared__ int q_vis[BATCH][4];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int b = (int)blockIdx.y - a.more, r0, r1;  // the rest of the long requests first: the search takes its time
  if (b >= 0) {
    request_rows(a, b, r0, r1);
    r1 = r1 > r0 ? r0 + min(r1 - r0, kRowsOnce) : r0;
  } else if (!locate_rows<kRowsOnce, 1>(a, blockIdx.y, lane, b, r0, r1)) {
    return;
  }
  const int64_t block0 = (int64_t)blockIdx.x * (kScoreWaves * TILES * kTile), k0 = block0 + wave * (TILES * kTile);
  const int key0 = (int)min(k0, (int64_t)0x7FFFFF00);
  // The pages of the wave's keys, on their way while the rows' lengths are found.
  const int my_page = page_at(a, a.page_table + (int64_t)b * a.pt_stride, key0 / PAGE_KEYS + min(lane, TILES * C - 1));
  const int row = lane < r1 - r0 ? visible_blocks(a.row_pos[r0 + lane], C, a.max_vis) : 0;
  static_assert(kRowsOnce <= 64, "a lane a row");
  if (blockIdx.x == 0 && a.row_len != nullptr) {
    if (wave == 0 && lane < r1 - r0) a.row_len[r0 + lane] = row;
    if ((int)blockIdx.y >= a.more)
      clear_padding(a.row_len, a.req_row_ptr, a.num_req, a.num_rows, (int64_t)b * blockDim.x + tid, (int64_t)a.num_req * blockDim.x);
  }
  const int most = wave_most(row);
  if (block0 >= most) return;

  u32x4_t k[TILES][4], ex[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    const int page = C == 4 ? __shfl(my_page, 4 * t + (n >> 2)) : (int)readlane(my_page, t);
    const int64_t at = (int64_t)page * PAGE_KEYS + (C == 4 ? 4 * (n & 3) : 4 * n);
#pragma unroll
    for (int j = 0; j < 4; ++j) k[t][j] = *reinterpret_cast<const u32x4_t*>(a.codes + (at + j) * kIdxCodes + g * 16);
    ex[t] = *reinterpret_cast<const u32x4_t*>(a.scales + at * kIdxScales);
  }
  uint32_t e[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t) e[t] = gather_bytes(ex[t], g);

  for (int first = r0; first < r1; first += 4 * BATCH) {
    const int groups = min(BATCH, (r1 - first + 3) / 4);
    if (first > r0) __syncthreads();
    if (wave < groups) {
      Rows x;
      x.load<C>(a, first + 4 * wave, r1 - 1, lane);
      const Query q(x);
      q_codes[wave][lane] = q.codes, q_exponent[wave][lane] = q.exponent;
      if (n == 0) q_vis[wave][g] = x.vis;
    }
    __syncthreads();
    if (k0 >= most) continue;
#pragma unroll 1
    for (int i = 0; i < groups; ++i) {
      const Query q(q_codes[i][lane], q_exponent[i][lane]);
      store_scores<TILES>(q, k, e, a.scores + (int64_t)(first + 4 * i + g) * a.ld + key0 + 4 * n, q_vis[i][g], key0, n);
    }
  }
}

// Many rows a request: 8 rows a wave, STAGES times 256 keys a workgroup.
//
// Bound by the scores' writes, and how fast those go depends on their order.
// Stores alone, 8,192 rows of 16,384, us: 102 with each wave writing 4 rows x 256
// bytes of 8 row groups in turn, 84 with one row group's 2 KiB first, 119 with
// four times as many rows between neighbours in time; workgroups of few rows,
// consecutive ones along the keys, 80 to 86.  So a stage is one row group's 4 tiles,
// then the other's.  A stage's keys are copied into LDS for all 4 waves while the
// stage before is computed (as operands straight from memory each wave's loads
// would take an access of the vector cache for every 16 bytes); the 16-byte pieces
// of 4 consecutive keys (256 bytes) are XOR-ed with their number, which spreads the
// operands' reads over the banks.
constexpr int kStage = 4;      // tiles in LDS at a time
constexpr int kRowGroups = 2;  // of 4 rows, a wave
template <int C, int STAGES>
__global__ __launch_bounds__(64 * kScoreWaves, 3) void score4_prefill_kernel(const ScoreArgs a) {
  constexpr int RG = kRowGroups;
  constexpr int PAGE_KEYS = kPage / C, ROWS = 4 * RG * kScoreWaves, KEYS = kStage * kTile, PAGES = KEYS / PAGE_KEYS;
  static_assert(kScoreWaves == 4, "a wave copies a quarter of a tile, 16 keys of one page");
  static_assert(PAGES * STAGES <= 64, "a lane a page");
  __shared__ __attribute__((aligned(16))) uint8_t codes[2][kStage][kTile * kIdxCodes];
  __shared__ __attribute__((aligned(16))) uint32_t exps[2][KEYS];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t k0 = (int64_t)blockIdx.x * (STAGES * KEYS);
  if (blockIdx.x == 0 && a.row_len != nullptr)
    clear_padding(a.row_len, a.req_row_ptr, a.num_req, a.num_rows, (int64_t)blockIdx.y * blockDim.x + tid,
                  (int64_t)gridDim.y * blockDim.x);
  const uint32_t blocks = a.num_rows / ROWS + a.num_req;  // at least as many as there are
  int b, first, end;
  for (uint32_t block = blockIdx.y; block < blocks && locate_rows<ROWS, 0>(a, block, lane, b, first, end); block += gridDim.y) {
    const int my_page = page_at(a, a.page_table + (int64_t)b * a.pt_stride,
                                (int)min(k0 / PAGE_KEYS, (int64_t)0x7FFFFF00) + min(lane, PAGES * STAGES - 1));
    const int row = first + lane < end ? visible_blocks(a.row_pos[first + lane], C, a.max_vis) : 0;
    static_assert(ROWS <= 64, "a lane a row");
    if (blockIdx.x == 0 && wave == 0 && a.row_len != nullptr && first + lane < end) a.row_len[first + lane] = row;
    const int most = wave_most(row);
    if (k0 >= most) continue;  // the same for every wave
    const int key0 = (int)k0, stages = min(STAGES, (most - key0 + KEYS - 1) / KEYS);

    u32x4_t stage_codes[kStage];
    uint32_t stage_exp;
    auto fetch = [&](int s) {
#pragma unroll
      for (int t = 0; t < kStage; ++t) {
        const int page = (int)readlane(my_page, C == 4 ? s * PAGES + t * 4 + wave : s * PAGES + t);
        const uint8_t* p = a.codes + ((int64_t)page * PAGE_KEYS + (C == 4 ? 0 : 16 * wave)) * kIdxCodes;
        stage_codes[t] = *reinterpret_cast<const u32x4_t*>(p + (4 * g) * kIdxCodes + (n ^ (4 * wave + g)) * 16);
      }
      const int page = C == 4 ? __shfl(my_page, s * PAGES + wave * 4 + g) : (int)readlane(my_page, s * PAGES + wave);
      stage_exp = *reinterpret_cast<const uint32_t*>(a.scales + ((int64_t)page * PAGE_KEYS + (C == 4 ? n : lane)) * kIdxScales);
    };
    auto put = [&](int buf) {
#pragma unroll
      for (int t = 0; t < kStage; ++t) *reinterpret_cast<u32x4_t*>(&codes[buf][t][wave * 1024 + lane * 16]) = stage_codes[t];
      exps[buf][tid] = stage_exp;
    };
    fetch(0);
    const int wr = first + wave * 4 * RG;
    const bool some = wr < end;
    Query q[RG] = {};
    int vis[RG];
    if (some) {
#pragma unroll
      for (int i = 0; i < RG; ++i) {
        Rows x;
        x.load<C>(a, wr + 4 * i, end - 1, lane);
        q[i] = Query(x), vis[i] = x.vis;
      }
    }
    __syncthreads();  // the buffers have been read
    put(0);
    __syncthreads();
    for (int s = 0; s < stages; ++s) {
      const int buf = s & 1, at = key0 + s * KEYS;
      if (s + 1 < stages) fetch(s + 1);
      if (some) {
        u32x4_t k[kStage][4];
        uint32_t e[kStage];
#pragma unroll
        for (int t = 0; t < kStage; ++t) {
#pragma unroll
          for (int j = 0; j < 4; ++j) k[t][j] = *reinterpret_cast<const u32x4_t*>(&codes[buf][t][n * 256 + (((4 * j + g) ^ n) * 16)]);
          e[t] = gather_bytes(*reinterpret_cast<const u32x4_t*>(&exps[buf][t * kTile + 4 * n]), g);
        }
#pragma unroll
        for (int i = 0; i < RG; ++i)
          store_scores<kStage>(q[i], k, e, a.scores + (int64_t)(wr + 4 * i + g) * a.ld + at + 4 * n, vis[i], at, n);
      }
      if (s + 1 < stages) {
        put(buf ^ 1);
        __syncthreads();
      }
    }
  }
}

namespace {

// The kernel for few rows goes through up to 64 rows of a request in each workgroup,
// the other is at its best with many; over 575 calls (1 to 256 requests of 6 to
// 8,192 rows, 1,000 to 65,536 tokens, c = 1 and 4) this rule costs 1.5% more than the
// best of the three (at most 27%: 16 requests of 8,000 with 256 rows 15.4 for 12.1).
// us, few rows / many with one stage / with four: 64 requests of 8,000 tokens (c = 4)
// with 12 rows 5.9 / 7.0 / 11.3, 20 7.5 / 7.7 / 12.0, 32 9.1 / 8.6 / 11.5; 16 of
// 65,536 (c = 1) with 16 rows 25.1 / 31.1 / 28.0.  num_rows counts padding: 64
// requests of 8,000 tokens with one row each 4.3 us, 10.9 in a call of 8,192 rows.
constexpr int64_t kFewRows = 20;
// Below so many workgroups of four stages: one stage each, four times as many.  1
// request of 65,536 tokens (c = 4) with 64 rows (48 workgroups) 6.5 us with one
// stage, 10.8 with four, 512 (272) 13.4 and 12.6, 2,000 (1,008) 36.3 and 33.2.
constexpr int64_t kFewGroups = 320;
// From so many keys in all on, two tiles a wave: 16 x 81,920 keys 18.1 us, 19.1 with
// one, 19.1 with four.
constexpr int64_t kManyKeys = 1 << 18;

}  // namespace

int launch_idx4_score(const uint16_t* q, const uint8_t* codes, const uint8_t* scales, int64_t num_pages,
                      const int32_t* page_table, int32_t pt_stride, const int32_t* req_row_ptr, int32_t num_req,
                      const int32_t* row_pos, int32_t num_rows, int32_t c, int32_t max_vis, float* scores, int64_t ld,
                      int32_t* row_len, hipStream_t stream) {
  const ScoreArgs a = {q,       codes,   scales,   (int32_t)num_pages, page_table, pt_stride, req_row_ptr,
                       row_pos, num_req, num_rows, max_vis,            scores,     ld,        row_len,     num_rows / kRowsOnce};
  const int64_t keys = std::max(max_vis, 1);
  const uint32_t few_blocks = num_req + a.more;  // at least as many as there are
  const bool few = num_rows <= kFewRows * (int64_t)num_req && few_blocks <= 65535;
  auto decode = [&](auto cc, auto tiles) {
    constexpr int TILES = decltype(tiles)::value, CHUNK = kScoreWaves * TILES * kTile;
    hipLaunchKernelGGL((score4_decode_kernel<decltype(cc)::value, TILES>), dim3((uint32_t)((keys + CHUNK - 1) / CHUNK), few_blocks),
                       dim3(64 * kScoreWaves), 0, stream, a);
  };
  auto run = [&](auto cc) {
    if (!few) {
      constexpr int ROWS = 4 * kRowGroups * kScoreWaves;
      const int64_t blocks = std::min<int64_t>(num_rows / ROWS + num_req, 65535);  // at least as many as there are
      auto prefill = [&](auto stages) {
        constexpr int STAGES = decltype(stages)::value, CHUNK = STAGES * kStage * kTile;
        hipLaunchKernelGGL((score4_prefill_kernel<decltype(cc)::value, STAGES>),
                           dim3((uint32_t)((keys + CHUNK - 1) / CHUNK), (uint32_t)blocks), dim3(64 * kScoreWaves), 0, stream, a);
      };
      if ((keys + 4 * kStage * kTile - 1) / (4 * kStage * kTile) * blocks < kFewGroups)
        prefill(std::integral_constant<int, 1>());
      else
        prefill(std::integral_constant<int, 4>());
    } else if (num_req * keys >= kManyKeys) {
      decode(cc, std::integral_constant<int, 2>());
    } else {
      decode(cc, std::integral_constant<int, 1>());
    }
  };
  if (c == 4)
    run(std::integral_constant<int, 4>());
  else
    run(std::integral_constant<int, 1>());
  return hipGetLastError() == hipSuccess ? BS_OK : BS_ERR_LAUNCH;
}

}  // namespace bs
