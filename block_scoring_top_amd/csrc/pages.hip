// pages.hip - the page tables of a batch, kept on the GPU: pages for new
// tokens with each new token's position and slot (extend), and pages given
// back (release).
//
// Both are prefix sums over the requests followed by writes that the sums
// place: request b's rows start at the sum of the earlier requests' new tokens,
// its pages at the sum of their needs, in the ring of free page ids.  A few
// kilobytes move, so what bounds them is latency: the launch, the lengths'
// load, the scans, a search, a load of the page id, the store.  Hence one
// launch: every workgroup scans all requests by itself (they fit in LDS) and
// writes its share of the rows and pages.  The lengths, where a caller has them
// updated in place, are written by the last workgroup to have read them, which a
// counter in the pool's state tells; into buffers of their own the first one writes.
#include <algorithm>
#include <type_traits>

#include "device.h"
#include "kernels.h"

namespace bs {

namespace {

constexpr uint32_t kMost = 0x7FFFFFFFu;  // sums saturate here

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kMost); }  // of two at most kMost

// Inclusive saturating prefix sum over a wave (saturating sums of numbers not
// below 0 associate).
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x = sat_add(x, dpp_u32<kDppRowShr1>(x));
  x = sat_add(x, dpp_u32<kDppRowShr2>(x));
  x = sat_add(x, dpp_u32<kDppRowShr4>(x));
  x = sat_add(x, dpp_u32<kDppRowShr8>(x));
  x = sat_add(x, dpp_u32<kDppRowBcast15, 0xA, false>(x));
  x = sat_add(x, dpp_u32<kDppRowBcast31, 0xC, false>(x));
  return x;
}

template <int THREADS, int BATCH>
struct Shared {
  int32_t len[BATCH], held[BATCH], change[BATCH];
  uint32_t row_end[THREADS], page_end[THREADS];  // of the chunk's requests
  uint32_t sums[2][THREADS / 64];
  uint32_t head, count, arrived;
};

// The same over the workgroup, on top of `carry`; `carry` becomes the total.
template <int WAVES>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t (&sums)[WAVES], uint32_t& carry) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  x = wave_scan(x);
  if (lane == 63) sums[wave] = x;
  __syncthreads();
  uint32_t before = carry;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const uint32_t s = sums[w];
    before = w < wave ? sat_add(before, s) : before;
    carry = sat_add(carry, s);
  }
  return sat_add(before, x);
}

// The first entry of an increasing list that is above x (there is one).
__device__ __forceinline__ int find_above(const uint32_t* ends, int n, uint32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ uint32_t ring_at(uint32_t head, uint32_t i, uint32_t size) {  // head, i <= size < 2^31
  const uint32_t x = head + i;
  return x >= size ? x - size : x;
}

}  // namespace

// BATCH requests in LDS at a time, of which THREADS are scanned together.
template <bool RELEASE, int THREADS, int BATCH>
__global__ __launch_bounds__(THREADS) void pages_kernel(const PagesCall a) {
  __shared__ Shared<THREADS, BATCH> sh;
  const int tid = threadIdx.x;
  const uint32_t share = gridDim.x * THREADS, mine = blockIdx.x * THREADS + tid;
  const uint32_t size = a.ring_size, cap = (uint32_t)min((int64_t)a.pt_stride * kPage, (int64_t)kMost);
  if (tid == 0) {
    sh.head = min(max(a.pool[0], 0), a.ring_size - 1);
    sh.count = min(max(a.pool[1], 0), a.ring_size);
    if (!RELEASE && blockIdx.x == 0) a.req_row_ptr[0] = 0;
  }
  uint32_t rows = 0, pages = 0;  // of the requests so far
  bool last = gridDim.x == 1 || (!a.in_place && blockIdx.x == 0);  // this workgroup writes the lengths
  const bool counts = gridDim.x > 1 && a.in_place;
  for (int b0 = 0; b0 < a.num_req; b0 += BATCH) {  // one turn, unless one workgroup does everything
    const int nb = min(BATCH, a.num_req - b0);
    for (int i = tid; i < nb; i += THREADS) {
      sh.len[i] = min((uint32_t)max(a.kv_len[b0 + i], 0), cap);
      sh.held[i] = min(max(a.held[b0 + i], 0), a.pt_stride);
      sh.change[i] = a.change[b0 + i];
      if (!RELEASE && blockIdx.x == 0 && a.tok_start != nullptr) a.tok_start[b0 + i] = sh.len[i];
    }
    __syncthreads();
    const uint32_t head = sh.head, count = sh.count;
    if (counts && tid == 0)
      sh.arrived = __hip_atomic_fetch_add(reinterpret_cast<uint32_t*>(a.pool_out + 3), 1u, __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT);
    for (int c0 = 0; c0 < nb; c0 += THREADS) {
      const int nc = min(THREADS, nb - c0), i = c0 + tid;
      const bool there = tid < nc;
      const uint32_t len = there ? sh.len[i] : 0, held = there ? sh.held[i] : 0;
      const int change = there ? sh.change[i] : 0;
      const uint32_t row0 = rows, page0 = pages;
      uint32_t len1 = len, held1 = held, want = 0;
      if constexpr (RELEASE) {
        len1 = change < 0 ? len : min((uint32_t)change, len);
        held1 = min(held, (len1 + kPage - 1) / kPage);
        want = held - held1;
      } else {
        const uint32_t n = change < 0 ? 0 : min((uint32_t)change, cap - len);
        const uint32_t end = min(block_scan(n, sh.sums[0], rows), (uint32_t)a.num_rows);
        rows = min(rows, (uint32_t)a.num_rows);
        sh.row_end[tid] = end;
        __syncthreads();
        // New tokens past the last row are not taken.
        len1 = len + (end - (tid == 0 ? row0 : sh.row_end[tid - 1]));
        const uint32_t need = (len1 + kPage - 1) / kPage;
        want = there && need > held ? need - held : 0;
      }
      const uint32_t page_end = block_scan(want, sh.sums[1], pages), first = page_end - min(want, page_end);
      sh.page_end[tid] = page_end;
      if constexpr (!RELEASE) {
        held1 = held + (first < count ? min(want, count - first) : 0);
        if (there && blockIdx.x == 0) a.req_row_ptr[b0 + i + 1] = (int32_t)sh.row_end[tid];
      }
      if (there) sh.change[i] = first;  // from here on: where the request's pages start
      __syncthreads();

      // The chunk's pages.
      const uint32_t page1 = RELEASE ? min(pages, size - count) : min(pages, count);
      for (uint32_t x = page0 / share * share + mine; x < page1; x += share) {
        if (x < page0) continue;
        const int r = find_above(sh.page_end, nc, x), b = c0 + r;
        const uint32_t at = x - (uint32_t)sh.change[b];
        if constexpr (RELEASE) {
          const uint32_t h = sh.held[b], gone = sh.page_end[r] - (uint32_t)sh.change[b];
          int32_t* p = a.page_table + (int64_t)(b0 + b) * a.pt_stride + (h - gone + at);
          a.ring[ring_at(ring_at(head, count, size), x, size)] = *p;
          *p = -1;
        } else {
          a.page_table[(int64_t)(b0 + b) * a.pt_stride + sh.held[b] + at] = a.ring[ring_at(head, x, size)];
        }
      }
      if constexpr (!RELEASE) {  // and its rows
        for (uint32_t x = row0 / share * share + mine; x < rows; x += share) {
          if (x < row0) continue;
          const int r = find_above(sh.row_end, nc, x), b = c0 + r;
          const uint32_t p = sh.len[b] + (x - (r == 0 ? row0 : sh.row_end[r - 1])), pi = p / kPage, h = sh.held[b];
          int page = -1;
          if (pi < h) {
            page = a.page_table[(int64_t)(b0 + b) * a.pt_stride + pi];
          } else {
            const uint32_t at = sat_add(sh.change[b], pi - h);
            if (at < count) page = a.ring[ring_at(head, at, size)];
          }
          a.row_pos[x] = (int32_t)p;
          a.slots[x] = page < 0 || page > (int)(kMost / kPage) ? -1 : page * kPage + (int)(p % kPage);
        }
      }
      __syncthreads();
      if (there) sh.len[i] = len1, sh.held[i] = held1;
    }
    // Everything that this workgroup reads of the caller's lengths has been
    // read; the last one to say so may write them.
    __syncthreads();
    if (counts) last = sh.arrived == gridDim.x - 1;
    if (last)
      for (int i = tid; i < nb; i += THREADS) a.kv_len_out[b0 + i] = sh.len[i], a.held_out[b0 + i] = sh.held[i];
    __syncthreads();
  }
  if constexpr (!RELEASE)
    for (uint32_t x = rows + mine; x < (uint32_t)a.num_rows; x += share) a.row_pos[x] = a.slots[x] = -1;
  __syncthreads();
  if (last && tid == 0) {
    const uint32_t head = sh.head, count = sh.count;
    if constexpr (RELEASE) {
      a.pool_out[0] = head, a.pool_out[1] = count + min(pages, size - count), a.pool_out[2] = 0;
    } else {
      const uint32_t taken = min(pages, count);
      a.pool_out[0] = taken == size ? head : ring_at(head, taken, size);
      a.pool_out[1] = count - taken, a.pool_out[2] = pages - taken;
    }
    a.pool_out[3] = 0;
  }
}

// Whether several workgroups can take a call: its state is updated in place, with the
// counter that the state has, or no workgroup reads what another writes.
static bool can_share(const PagesCall& a) {
  if (a.in_place) return true;
  const int64_t n = a.num_req;
  auto meet = [](const int32_t* x, int64_t nx, const int32_t* y, int64_t ny) { return x < y + ny && y < x + nx; };
  auto read = [&](const int32_t* x, int64_t nx) {
    return meet(x, nx, a.kv_len, n) || meet(x, nx, a.held, n) || meet(x, nx, a.change, n) || meet(x, nx, a.pool, 4);
  };
  return !read(a.kv_len_out, n) && !read(a.held_out, n) && !read(a.pool_out, 4);
}

// There is a workgroup for every kItems rows (extend) or 16 times as many page
// table entries (release: few of them are given back).  us, both calls of 1,003
// requests with 56,000 new tokens, kItems 512 / 1,024 / 2,048: 10.6 / 10.6 / 12.5.
// Up to 256 requests: workgroups of 256, whose barriers and scans are shorter
// (64 requests x 6 rows: 7.6 us, 8.8 with 1,024; 7.1 of them on the GPU).
int launch_pages(const PagesCall& a, bool release, hipStream_t stream) {
  constexpr int64_t kItems = 1024;
  auto go = [&](auto rel, auto threads, auto batch) {
    constexpr int THREADS = decltype(threads)::value, BATCH = decltype(batch)::value;
    const int64_t items = release ? (int64_t)a.num_req * a.pt_stride / 16 : a.num_rows;
    const bool once = a.num_req > 0 && a.num_req <= BATCH && can_share(a);  // else one workgroup does everything, in turns
    const uint32_t grid = once ? (uint32_t)std::min<int64_t>(128, std::max<int64_t>(1, items / kItems)) : 1;
    hipLaunchKernelGGL((pages_kernel<decltype(rel)::value, THREADS, BATCH>), dim3(grid), dim3(THREADS), 0, stream, a);
  };
  auto by_size = [&](auto rel) {
    if (a.num_req <= 256)
      go(rel, std::integral_constant<int, 256>(), std::integral_constant<int, 256>());
    else
      go(rel, std::integral_constant<int, 1024>(), std::integral_constant<int, 4096>());
  };
  if (release)
    by_size(std::true_type());
  else
    by_size(std::false_type());
  return hipGetLastError() == hipSuccess ? BS_OK : BS_ERR_LAUNCH;
}

}  // namespace bs
