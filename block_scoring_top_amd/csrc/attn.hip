// attn.hip - host side of the attention calls: which kernel, its tiles, and
// over how many workgroups a row's keys are split.
#include <algorithm>
#include <cmath>
#include "attn_gather.h"
#include "attn_prefill.h"

namespace bs {

extern template int launch_attn_prefill<Bf16, true>(const PrefillArgs&, int, int, uint32_t, hipStream_t);
extern template int launch_attn_prefill<Bf16, false>(const PrefillArgs&, int, int, uint32_t, hipStream_t);
extern template int launch_attn_prefill<F16, true>(const PrefillArgs&, int, int, uint32_t, hipStream_t);
extern template int launch_attn_prefill<F16, false>(const PrefillArgs&, int, int, uint32_t, hipStream_t);

extern template int launch_attn_gather<Bf16, true>(const GatherArgs&, int, int, bool, hipStream_t);
extern template int launch_attn_gather<Bf16, false>(const GatherArgs&, int, int, bool, hipStream_t);
extern template int launch_attn_gather<F16, true>(const GatherArgs&, int, int, bool, hipStream_t);
extern template int launch_attn_gather<F16, false>(const GatherArgs&, int, int, bool, hipStream_t);

namespace {

constexpr int64_t kCounterBytes = 64 << 10;  // first part of the workspace: arrival counters
constexpr int64_t kPartialBytes = (int64_t)BS_ATTN_WORKSPACE_BYTES - kCounterBytes;
// (row, head) pairs that a request may have for the gathering kernel to take
// an attn_window call; the prefill kernel takes those with more.  64 requests,
// window 4,096, D = 128, 48 pairs: 4-bit 46 us gathered, 61 otherwise; 16-bit
// 102 and 68 (two gathered tiles read each key twice, four times the bytes).  8
// pairs: 4-bit 21 and 59 us, 16-bit 49 and 64.
int gather_cols(const AttnCall& c) { return c.form == BS_KV_4 && c.d <= 128 ? 64 : 32; }
// Keys are split over workgroups up to kFillBlocks in all, with at least
// kSplitKeys keys each (two chunks a wave).  us, 512 / 768 / 1,024 workgroups:
// 64 decode rows x 2 kv heads of a 4,096 window (4-bit, D = 128) 20.9 / 23.0 /
// 25.9, of 2,051 slots (D = 256) 23.7 / 28.9 / 28.4.  One row of 2,050 slots with
// at least 128 / 256 / 512 keys a split: 8.8 / 8.1 / 9.8.
constexpr int64_t kFillBlocks = 512, kSplitKeys = 256;
// The prefill kernel's pages: 50 rows x 2 kv heads of 8 over 65 pages, with at
// least 2 / 4 / 8 pages a part: 28.0 / 21.5 / 23.4 us (93 unsplit).
constexpr int64_t kSplitPages = 4;
// Its workgroups have 8 waves if there are this many of them, else 4: 4 fill
// the chip with less work, 8 read a page of K and V for twice the rows.  us,
// 8 and 4 waves: 512 workgroups (8,192 rows, window 4,096) 279 and 293; 360 (5
// ragged requests) 87 and 51; 256 (1,024 rows, 8 kv heads) 40 and 32.
constexpr int64_t kEightWaves = 512;
// Row tiles times head blocks of a launch: 2^30 lanes.
constexpr int64_t kMaxGroups = (int64_t)1 << 21;

// The running maximum is of unscaled scores times the scale, which then must
// not be negative (q changes sign instead) nor 0 (a masked -inf times 0).
void set_scale(const AttnCall& c, float& scale_log2, uint32_t& flip) {
  const float s = c.scale * kLog2e;
  scale_log2 = std::max(std::fabs(s), 1.1754944e-38f);
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

int run_gather(GatherArgs& a, const AttnCall& c, int nt, bool window, int64_t tiles, int64_t max_keys,
               hipStream_t stream) {
  const int64_t groups = tiles * a.hkv * a.hblocks;
  if (c.workspace != nullptr && groups < kFillBlocks) {
    const int64_t per = (int64_t)16 * nt * (c.d + 4) * 4;
    int64_t n = std::min((kFillBlocks + groups - 1) / groups, (max_keys + kSplitKeys - 1) / kSplitKeys);
    n = std::min(n, kPartialBytes / per / groups);
    a.nsplit = (int)std::max<int64_t>(n, 1);
    a.counters = static_cast<uint32_t*>(c.workspace);
    a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(c.workspace) + kCounterBytes);
  }
  if (groups > kMaxGroups) return BS_ERR_ARG;
  a.tiles = (int32_t)tiles;
  // Rows of a request read many of the same keys: 64 x 6 verify rows of 2,051
  // slots (4-bit) 42.0 us with eight neighbours on an XCD, 44.8 without.
  a.xcd_rows = tiles >= 64;
  if (c.dtype == BS_BF16)
    return c.form == BS_KV_4 ? launch_attn_gather<Bf16, true>(a, c.d, nt, window, stream)
                             : launch_attn_gather<Bf16, false>(a, c.d, nt, window, stream);
  return c.form == BS_KV_4 ? launch_attn_gather<F16, true>(a, c.d, nt, window, stream)
                           : launch_attn_gather<F16, false>(a, c.d, nt, window, stream);
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
  set_scale(c, a.scale_log2, a.flip);
  a.out = c.out, a.ld_out = c.ld_out, a.lse = c.lse;
  a.nsplit = 1;
  if (c.workspace != nullptr && blocks < kFillBlocks) {
    const int64_t pages = std::min<int64_t>(pt_stride, ((int64_t)window + a.rows_per_tile) / kPage + sinks / kPage + 2);
    const int64_t per = (int64_t)32 * waves * (c.d + 4) * 4;
    const int64_t n = std::min(std::min(kFillBlocks / blocks, pages / kSplitPages), kPartialBytes / per / blocks);
    a.nsplit = (uint32_t)std::max<int64_t>(n, 1);
    a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(c.workspace) + kCounterBytes);
  }
  if (blocks > kMaxGroups) return BS_ERR_ARG;
  a.groups = (uint32_t)blocks;
  const uint32_t grid = (a.groups * a.nsplit + 63) / 64 * 64;
  if (c.dtype == BS_BF16)
    return c.form == BS_KV_4 ? launch_attn_prefill<Bf16, true>(a, c.d, waves, grid, stream)
                             : launch_attn_prefill<Bf16, false>(a, c.d, waves, grid, stream);
  return c.form == BS_KV_4 ? launch_attn_prefill<F16, true>(a, c.d, waves, grid, stream)
                           : launch_attn_prefill<F16, false>(a, c.d, waves, grid, stream);
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
  if ((int64_t)g * max_rows > gather_cols(c))
    return run_prefill(c, page_table, pt_stride, req_row_ptr, num_req, row_pos, max_rows, window, sinks, stream);
  GatherArgs a = common_args(c);
  split_heads(a, nt);
  a.page_table = page_table, a.pt_stride = pt_stride, a.req_row_ptr = req_row_ptr, a.row_pos = row_pos;
  a.max_rows = max_rows, a.window = window, a.sinks = sinks;
  a.rows_per_tile = std::max(1, 16 * nt / a.gb);
  a.tiles_per_req = (int)(((int64_t)max_rows + a.rows_per_tile - 1) / a.rows_per_tile);
  const int64_t keys = std::min<int64_t>((int64_t)pt_stride * kPage, (int64_t)window + sinks + a.rows_per_tile - 1);
  return run_gather(a, c, nt, true, (int64_t)num_req * a.tiles_per_req, keys, stream);
}

}  // namespace bs
