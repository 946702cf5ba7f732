// attn.hip - host side of the attention calls: which kernel, its tiles, and
// over how many workgroups a row's keys are split.
#include <algorithm>
#include <cmath>
#include <limits>

#include "attn_gather.h"
#include "attn_prefill.h"

namespace bs {

#define BS_FORM(T, FORM)                                                                                       \
  extern template int launch_attn_prefill<T, FORM>(const PrefillArgs&, int, int, uint32_t, hipStream_t);       \
  extern template int launch_attn_gather<T, FORM>(const GatherArgs&, int, int, bool, hipStream_t);
BS_FORM(Bf16, kForm16)
BS_FORM(Bf16, kForm4)
BS_FORM(Bf16, kForm8)
BS_FORM(F16, kForm16)
BS_FORM(F16, kForm4)
BS_FORM(F16, kForm8)
#undef BS_FORM

namespace {

constexpr int64_t kCounterBytes = 64 << 10;  // first part of the workspace: arrival counters
constexpr int64_t kPartialBytes = (int64_t)BS_ATTN_WORKSPACE_BYTES - kCounterBytes;
// Does the gathering kernel take an attn_window call, or the prefill kernel?  The
// first is quicker to start and splits the keys of few rows well; it reads them
// once for 16 or 32 (row, head) pairs where the other reads them for 128.  It takes
//   * calls of at most `most` row tiles times keys, which latency bounds.  us,
//     gathered and not: 4-bit, D = 128, 6 rows x 8 heads, window 700 12.0 and 13.1,
//     36 requests of them 14.8 and 21.2; 700 rows, 700,000 tiles times keys, 40.5
//     and 43.3, 1.4 million 65.2 and 50.6.  16-bit, D = 128, 100 rows, window 1,200
//     (60,000) 16.0 and 17.3, 4,000 29.2 and 23.8;
//   * requests whose pairs are one tile, or (`ratio`) whose tiles read the keys no
//     more than that many times for the other's once: half of its pairs would
//     be padding.  64 requests, window 4,000: 1 row, 16-bit 46 and 59; 6 rows,
//     4-bit 40 and 60;
//   * the 4-bit cache at D = 256, where one wave a SIMD is all that the other's
//     registers allow.  16 query / 2 kv heads, window 4,000: 8,192 rows from position 0
//     820 and 925, at the end of a 64K context 1,026 and 1,015 (window 500: 207 and
//     186); 64 x 6 rows 78 and 271.
// The 8-bit cache: 16 query / 2 kv heads, gathered and not, D = 128: 100 rows, window
// 1,200 (60,000 tiles times keys) 16 and 19 us, 300, 1,000 (150,000) 21 and 22, 700,
// 1,000 (350,000) 41 and 27; 36 x 6 rows, window 700 18 and 22, 64 x 6, window 4,000
// 65 and 60.  D = 64: 1,000 rows, window 1,000 (500,000) 19 and 23, but 2,000, 500 (the
// same number) 23 and 16.  D = 256, where its codes take the other's registers only
// for a page at a time: 100 rows, window 1,000 (100,000) 23 and 36, 300, 1,000 (300,000) 43
// and 49, 700, 500 (350,000) 41 and 51, 200, 2,000 (400,000) 39 and 49, 300, 1,500 (450,000)
// 60 and 53, 300, 2,000 (600,000) 74 and 54, 2,000 rows 293 and 151; 64 x 6 rows, window
// 4,000 140 and 324.  Over 42 such calls (60 to 2,000 rows, windows of 500 to 2,000) the
// kernel chosen is 3% slower than the better one; at most 25% at D = 256, 10% at 128,
// 42% at 64.
bool gathers(const AttnCall& c, int64_t tiles, int64_t keys, int64_t pairs, int64_t num_req) {
  const bool kv4 = c.form == BS_KV_4, kv8 = c.form == BS_KV_8;
  if (pairs <= 16 || (kv4 && c.d == 256)) return true;
  const double most = kv8 ? (c.d == 64 ? 550e3 : c.d == 128 ? 150e3 : 350e3)
                      : kv4 ? (c.d == 64 ? 550e3 : 700e3) : c.d == 64 ? 500e3 : c.d == 128 ? 60e3 : 80e3;
  const int64_t ratio = kv8 ? (c.d == 64 ? 2 : c.d == 128 ? 1 : 4) : kv4 || c.d == 64 ? 2 : 0;
  return (double)tiles * keys <= most || tiles <= ratio * num_req * c.hkv * ((pairs + 127) / 128);
}
// Keys are split over up to kFillBlocks workgroups in all.  us, 512 / 768 / 1,024:
// 64 decode rows x 2 kv heads of a 4,096 window (4-bit, D = 128) 20.9 / 23.0 / 25.9,
// of 2,051 slots (D = 256) 23.7 / 28.9 / 28.4.
constexpr int64_t kFillBlocks = 512;
// What splitting the prefill kernel's pages costs, in the time of a page (1.27
// us at D = 128, D to that): kJoinPages for the launch that joins, a page for
// every kPartsPerPage parts written and read again, kPartPages for each part
// that a joining lane goes through.  us, D = 128, 8 heads a group of 4: a window
// of 800 in 1 / 2 / 3 / 4 / 8 parts, 8 blocks 25.6 / 20.3 / 16.9 / 15.9 / 14.7, 100
// blocks 26.3 / 27.7 / 27.4 / 28.0 / 28.0; 4,096, 28 blocks 91.8 / 52.6 / 40.2 /
// 34.6 / 27.4 (16 parts: 30.5).
constexpr double kJoinPages = 2.5, kPartsPerPage = 42, kPartPages = 1. / 6;
// Its workgroups have 8 waves if there are this many of them, else 4: 4 fill
// the chip with less work, 8 read a page of K and V for twice the rows.  us,
// 8 and 4 waves: 512 workgroups (8,192 rows, window 4,096) 279 and 293; 360 (5
// ragged requests) 87 and 51; 256 (1,024 rows, 8 kv heads) 40 and 32.
constexpr int64_t kEightWaves = 512;
// Row tiles times head blocks of a launch: 2^30 lanes.
constexpr int64_t kMaxGroups = (int64_t)1 << 21;

template <class F>
int by_type_and_form(const AttnCall& c, F f) {
  auto form = [&](auto t) {
    if (c.form == BS_KV_4) return f(t, std::integral_constant<int, kForm4>());
    if (c.form == BS_KV_8) return f(t, std::integral_constant<int, kForm8>());
    return f(t, std::integral_constant<int, kForm16>());
  };
  return c.dtype == BS_BF16 ? form(Bf16()) : form(F16());
}

// The running maximum is of unscaled scores times the scale, which then must
// not be negative (q changes sign instead) nor 0 (a masked -inf times 0): the
// least positive number stands for that, under which the largest score that
// FP32 holds is 5e-7.  (The kernels compute with subnormal numbers.)
void set_scale(const AttnCall& c, float& scale_log2, uint32_t& flip) {
  const float s = c.scale * kLog2e;
  scale_log2 = std::max(std::fabs(s), std::numeric_limits<float>::denorm_min());
  flip = s < 0.f ? 0x80008000u : 0u;
}

GatherArgs common_args(const AttnCall& c) {
  GatherArgs a = {};
  a.q = c.q, a.ld_q = c.ld_q;
  a.a = static_cast<const uint8_t*>(c.cache0), a.b = static_cast<const uint8_t*>(c.cache1);
  a.ld_kv = c.ld_cache;
  a.num_slots = c.num_slots, a.num_rows = c.num_rows, a.hq = c.hq, a.hkv = c.hkv;
  set_scale(c, a.scale_log2, a.flip);
  a.out = c.out, a.ld_out = c.ld_out, a.lse = c.lse;
  a.nsplit = 1;
  return a;
}

// Heads of one kv head's group in blocks of at most 16*nt, as even as possible.
void split_heads(GatherArgs& a, int nt) {
  const int g = a.hq / a.hkv;
  a.hblocks = (g + 16 * nt - 1) / (16 * nt);
  a.gb = (g + a.hblocks - 1) / a.hblocks;
}

// Over how many workgroups a group of the gathering kernel has its keys split:
// of 1, 2, 4 .. `most` the number whose estimated time is least.  In us: a chunk of
// each of the 4 waves after the other (workgroups past one a compute unit slow each
// other down), but no less than the keys' bytes take; a join of 4 us, the parts
// that are written and read again (1.3 MB a us), and 3 for each round of loads that
// a joining lane waits for after the first.  (`cols`: columns in use.)  Over 106
// sweeps of 1 to 128 parts (1 to 240 groups of 250 to 64,000 keys, both caches, all
// head dims) the number chosen is 1.6% slower than the best one; as many as 512
// workgroups and 256 keys a part allow, 11%: 1 row of 256 slots 5.5 and 8.0 us, 30
// requests x 2 rows x 8 heads of D = 256 over 4,096 keys 24 and 42.  Those were the
// 16-bit pools and the 4-bit cache; the 8-bit one has the latter's constants, with
// which its number is 3.9, 1.0 and 2.1% slower than the best at D = 64, 128 and 256
// (38 calls each: 1 to 120 rows of 256 to 32,768 slots, 2 and 8 kv heads; at most
// 17, 10 and 20%).
int gather_splits(const AttnCall& c, int nt, int cols, int64_t groups, int64_t keys, int64_t most) {
  const bool codes = c.form != BS_KV_16;
  const double chunk = 0.6 + 0.7 * nt * c.d / 128 + (codes || c.d == 64 ? 0. : c.d == 256 ? 3. : 1.1);
  const double read = groups * keys * c.d * (c.form == BS_KV_4 ? 17. / 16 : codes ? 2. : 4.) / 4.5e6;
  const double part = cols * (c.d + 4) * 4e-6 * groups, rounds = cols * c.d / 16384.;
  int64_t best = 1;
  double least = 0;
  for (int64_t n = 1; n <= most; n *= 2) {
    const int64_t chunks = ((keys + kGaKeys - 1) / kGaKeys + kGaWaves * n - 1) / (kGaWaves * n);
    const int64_t layers = (groups * n + 255) / 256;
    double t = std::max(chunks * chunk * (layers == 1 ? 1. : 0.6 * layers), read) + (layers - 1);
    if (n > 1) t += 4 + 0.75 * n * part + 3 * std::max(0., n * rounds - 1);
    if (n == 1 || t < least) best = n, least = t;
    if (chunks <= 1) break;
  }
  return (int)best;
}

int run_gather(GatherArgs& a, const AttnCall& c, int nt, bool window, int64_t tiles, int64_t max_keys,
               hipStream_t stream) {
  const int64_t groups = tiles * a.hkv * a.hblocks;
  if (c.workspace != nullptr && groups < kFillBlocks) {
    const int64_t per = (int64_t)16 * nt * (c.d + 4) * 4;
    const int64_t most = std::min(kFillBlocks / groups, kPartialBytes / per / groups);
    a.nsplit = gather_splits(c, nt, window ? std::min(16 * nt, a.rows_per_tile * a.gb) : a.gb, groups, max_keys, most);
    a.counters = static_cast<uint32_t*>(c.workspace);
    a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(c.workspace) + kCounterBytes);
  }
  if (groups > kMaxGroups) return BS_ERR_ARG;
  a.tiles = (int32_t)tiles;
  // Rows of a request read many of the same keys: 64 x 6 verify rows of 2,051
  // slots (4-bit) 42.0 us with eight neighbours on an XCD, 44.8 without.
  a.xcd_rows = tiles >= 64;
  return by_type_and_form(c, [&](auto t, auto form) {
    return launch_attn_gather<decltype(t), decltype(form)::value>(a, c.d, nt, window, stream);
  });
}

int run_prefill(const AttnCall& c, const int32_t* page_table, int32_t pt_stride, const int32_t* req_row_ptr,
                int32_t num_req, const int32_t* row_pos, int32_t max_rows, int32_t window, int32_t sinks,
                hipStream_t stream) {
  PrefillArgs a = {};
  a.q = c.q, a.ld_q = c.ld_q;
  a.a = static_cast<const uint8_t*>(c.cache0), a.b = static_cast<const uint8_t*>(c.cache1);
  a.ld_kv = c.ld_cache;
  a.num_pages = c.num_slots / kPage, a.num_rows = c.num_rows, a.hq = c.hq, a.hkv = c.hkv;
  const int g = c.hq / c.hkv;
  int waves = 8;
  int64_t blocks = 0;
  auto tile = [&]() {  // for `waves`: 32 (row, head) pairs a wave
    const int cols = 32 * waves;
    a.hblocks = (g + cols - 1) / cols;
    a.gb = (g + a.hblocks - 1) / a.hblocks;
    a.rows_per_tile = cols / a.gb;
    a.tiles_per_req = (int)(((int64_t)max_rows + a.rows_per_tile - 1) / a.rows_per_tile);
    blocks = (int64_t)num_req * a.tiles_per_req * a.hkv * a.hblocks;
  };
  tile();
  if (c.d == 256 || blocks < kEightWaves) {
    waves = 4;
    tile();
  }
  a.page_table = page_table, a.req_row_ptr = req_row_ptr, a.row_pos = row_pos, a.pt_stride = pt_stride;
  a.max_rows = max_rows, a.window = window, a.sinks = sinks;
  // Without a window a request's later rows see more keys, and workgroups that
  // start last should not be the longest: 8,192 rows from position 0, 16 query / 2
  // kv heads of 128, 16-bit 312 us so, 401 in order; 4,096 rows of 256 237 and 323,
  // of 128 126 and 125.  Under a window all are about as long, and in order is up
  // to 6% quicker.
  a.latest_first = window >= (int64_t)pt_stride * kPage;
  set_scale(c, a.scale_log2, a.flip);
  a.out = c.out, a.ld_out = c.ld_out, a.lse = c.lse;
  a.nsplit = 1;
  if (c.workspace != nullptr && blocks < kFillBlocks) {
    const int64_t pages = std::min<int64_t>(pt_stride, ((int64_t)window + a.rows_per_tile) / kPage + sinks / kPage + 2);
    const int64_t per = (int64_t)32 * waves * (c.d + 4) * 4;
    const double part = blocks / kPartsPerPage + kPartPages;
    const int64_t best = (int64_t)std::sqrt(pages / part);
    const int64_t n = std::min(std::min(kFillBlocks / blocks, best), kPartialBytes / per / blocks);
    if (n > 1 && pages - pages / (double)n > kJoinPages + n * part) a.nsplit = (uint32_t)n;
    a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(c.workspace) + kCounterBytes);
  }
  if (blocks > kMaxGroups) return BS_ERR_ARG;
  a.groups = (uint32_t)blocks;
  const uint32_t grid = (a.groups * a.nsplit + 63) / 64 * 64;
  return by_type_and_form(c, [&](auto t, auto form) {
    return launch_attn_prefill<decltype(t), decltype(form)::value>(a, c.d, waves, grid, stream);
  });
}

}  // namespace

int launch_attn_slots(const AttnCall& c, const int32_t* slots, int32_t ld_slots, const int32_t* count,
                      hipStream_t stream) {
  GatherArgs a = common_args(c);
  const int nt = c.hq / c.hkv <= 16 || c.d == 256 ? 1 : 2;
  split_heads(a, nt);
  a.slots = slots, a.ld_slots = ld_slots, a.count = count;
  return run_gather(a, c, nt, false, c.num_rows, ld_slots, stream);
}

int launch_attn_window(const AttnCall& c, const int32_t* page_table, int32_t pt_stride, const int32_t* req_row_ptr,
                       int32_t num_req, const int32_t* row_pos, int32_t max_rows, int32_t window, int32_t sinks,
                       hipStream_t stream) {
  const int g = c.hq / c.hkv, nt = (int64_t)g * max_rows <= 16 || c.d == 256 ? 1 : 2;
  GatherArgs a = common_args(c);
  split_heads(a, nt);
  a.rows_per_tile = std::max(1, 16 * nt / a.gb);
  a.tiles_per_req = (int)(((int64_t)max_rows + a.rows_per_tile - 1) / a.rows_per_tile);
  const int64_t keys = std::min<int64_t>((int64_t)pt_stride * kPage, (int64_t)window + sinks + a.rows_per_tile - 1);
  const int64_t tiles = (int64_t)num_req * a.tiles_per_req;
  // The other kernel's tiles are at most 256 times as many rows: too many for
  // both, and for the products with heads below.
  if (tiles > kMaxGroups * 256) return BS_ERR_ARG;
  if (!gathers(c, tiles * c.hkv * a.hblocks, keys, (int64_t)g * max_rows, num_req))
    return run_prefill(c, page_table, pt_stride, req_row_ptr, num_req, row_pos, max_rows, window, sinks, stream);
  a.page_table = page_table, a.pt_stride = pt_stride, a.req_row_ptr = req_row_ptr, a.row_pos = row_pos;
  a.max_rows = max_rows, a.window = window, a.sinks = sinks;
  return run_gather(a, c, nt, true, tiles, keys, stream);
}

}  // namespace bs
