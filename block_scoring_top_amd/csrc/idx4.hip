// idx4.hip - index keys in 4 bits: rows quantised as they are written, and
// read back.
//
// Per group of 32 channels: e = floor(log2(max |x|)) - 2, clamped to -120 ..
// 125; code = x * 2^-e rounded to the nearest E2M1 value, ties to the even code,
// saturating at 6; an infinity or a NaN makes the group NaN.  Streams without
// reuse, bound by the launch at the sizes of decode and by HBM beyond: a lane
// takes 8 channels of a key, the 4 lanes of a group agree on the scale with two
// DPP moves, and a wave writes 4 whole keys.
#include <algorithm>

#include "idx4.h"
#include "kernels.h"

namespace bs {

namespace {
constexpr int kLanes = kDim / 8;  // of a key
}

template <class T>
__global__ __launch_bounds__(256) void idx4_store_kernel(const typename T::elem* __restrict__ keys, int64_t ld,
                                                         const int32_t* __restrict__ slots, int32_t n,
                                                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                         int32_t num_slots) {
  const uint32_t id = blockIdx.x * 256 + threadIdx.x, t = id / kLanes, j = id % kLanes;
  if (t >= (uint32_t)n) return;
  const int32_t slot = slots[t];
  Chunk<T> x;
  x.load(keys + (int64_t)t * ld + j * 8);
  if (slot < 0 || slot >= num_slots) return;  // whole keys are left out, so a group's 4 lanes stay together
  bool bad;
  const uint32_t e = group_exponent(quad_max(x.top()), bad);
  *reinterpret_cast<uint32_t*>(codes + (int64_t)slot * kIdxCodes + j * 4) = bad ? 0u : x.codes(kv4_scale(e));
  if ((j & 3) == 0) scales[(int64_t)slot * kIdxScales + j / 4] = (uint8_t)(bad ? kExpNan : e);
}

template <class T>
__global__ __launch_bounds__(256) void idx4_load_kernel(const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales, int32_t num_slots,
                                                        const int32_t* __restrict__ slots, int32_t n,
                                                        typename T::elem* __restrict__ out, int64_t ld) {
  const uint32_t id = blockIdx.x * 256 + threadIdx.x, t = id / kLanes, j = id % kLanes;
  if (t >= (uint32_t)n) return;
  const int32_t slot = slots[t];
  uint32_t c = 0, b = 127;
  if (slot >= 0 && slot < num_slots) {
    c = *reinterpret_cast<const uint32_t*>(codes + (int64_t)slot * kIdxCodes + j * 4);
    b = scales[(int64_t)slot * kIdxScales + j / 4];
  }
  Chunk<T> x;
  x.values(c, kv4_scale(b));
  x.store(out + (int64_t)t * ld + j * 8);
}

namespace {

// Calls f(type, first row, rows) for launches of at most 2^31 lanes.
template <class F>
int by_type_and_rows(int32_t dtype, int32_t rows, F f) {
  auto go = [&](auto t) {
    constexpr int64_t most = ((int64_t)1 << 31) / kLanes;
    for (int64_t r = 0; r < rows; r += most) {
      f(t, r, (int32_t)std::min<int64_t>(most, rows - r));
      if (hipGetLastError() != hipSuccess) return (int)BS_ERR_LAUNCH;
    }
    return (int)BS_OK;
  };
  if (dtype == BS_BF16) return go(Bf16());
  if (dtype == BS_F16) return go(F16());
  return go(F32());
}

}  // namespace

int launch_idx4_store(const void* keys, int32_t dtype, int64_t ld, const int32_t* slots, int32_t num_keys,
                      uint8_t* codes, uint8_t* scales, int32_t num_slots, hipStream_t stream) {
  return by_type_and_rows(dtype, num_keys, [&](auto t, int64_t r, int32_t n) {
    typedef decltype(t) T;
    hipLaunchKernelGGL(idx4_store_kernel<T>, dim3(((int64_t)n * kLanes + 255) / 256), dim3(256), 0, stream,
                       static_cast<const typename T::elem*>(keys) + r * ld, ld, slots + r, n, codes, scales, num_slots);
  });
}

int launch_idx4_load(const uint8_t* codes, const uint8_t* scales, int32_t num_slots, const int32_t* slots,
                     int32_t num_slot_ids, void* out, int32_t dtype, int64_t ld, hipStream_t stream) {
  return by_type_and_rows(dtype, num_slot_ids, [&](auto t, int64_t r, int32_t n) {
    typedef decltype(t) T;
    hipLaunchKernelGGL(idx4_load_kernel<T>, dim3(((int64_t)n * kLanes + 255) / 256), dim3(256), 0, stream, codes, scales,
                       num_slots, slots + r, n, static_cast<typename T::elem*>(out) + r * ld, ld);
  });
}

}  // namespace bs
