// kv4.hip - the 4-bit KV cache: rows quantised as they are written, and read
// back.
//
// Store, per group of 32 channels: e = floor(log2(max |x|)) - 2, clamped to
// -120 .. 125, read off the exponent field of the largest bit pattern (as
// unsigned integers, bit patterns of |x| order like the values, with
// infinities and NaN on top, so one integer maximum serves both purposes);
// code = x * 2^-e rounded to the nearest E2M1 value, ties to the even code,
// saturating at 6.  Load: code * 2^e.
//
// Both are streams without reuse: what bounds them is HBM at the prefill
// sizes and the launch at the decode ones.  A lane takes 8 channels: its
// 16-byte read (or write) of the 16-bit side and its 4-byte write (or read)
// of the codes are both contiguous over the wave, and the 4 lanes of a group
// agree on the scale with two DPP moves, with no LDS.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "kv4.h"

namespace bs {

namespace {

__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kDppQuadXor1, 0xF, 0xF, true));
  return max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kDppQuadXor2, 0xF, 0xF, true));
}

// 8 channels as loaded: 4 pairs of 16-bit values, or 8 floats.
template <class T>
struct Chunk {
  u32x4_t v;
  __device__ __forceinline__ void load(const void* p) { v = *reinterpret_cast<const u32x4_t*>(p); }
  __device__ __forceinline__ uint32_t top() const {
    return max(max(T::abs_bits(v.x), T::abs_bits(v.y)), max(T::abs_bits(v.z), T::abs_bits(v.w)));
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    uint32_t c = T::template to_fp4<0>(0u, v.x, s);
    c = T::template to_fp4<1>(c, v.y, s);
    c = T::template to_fp4<2>(c, v.z, s);
    return T::template to_fp4<3>(c, v.w, s);
  }
  __device__ __forceinline__ void values(uint32_t c, float s) {
    v = u32x4_t{T::template from_fp4<0>(c, s), T::template from_fp4<1>(c, s), T::template from_fp4<2>(c, s),
                T::template from_fp4<3>(c, s)};
  }
  __device__ __forceinline__ void store(void* p) const { __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(p)); }
};

template <>
struct Chunk<F32> {
  float v[8];
  __device__ __forceinline__ void load(const void* p) {
    const f32x4_t a = reinterpret_cast<const f32x4_t*>(p)[0], b = reinterpret_cast<const f32x4_t*>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  }
  __device__ __forceinline__ void values(uint32_t c, float s) {
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
    const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = d.x, v[5] = d.y, v[6] = e.x, v[7] = e.y;
  }
  __device__ __forceinline__ void store(void* p) const {
    __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4_t*>(p));
    __builtin_nontemporal_store(f32x4_t{v[4], v[5], v[6], v[7]}, reinterpret_cast<f32x4_t*>(p) + 1);
  }
};

}  // namespace

// Lane `id` of a call: 8 channels of a row; a row's lanes go through its
// heads, K then V of each, so that a wave writes whole lines of codes.
template <int D>
struct Piece {
  uint32_t t, h, which, j;
  __device__ __forceinline__ Piece(uint32_t id, uint32_t hkv) {
    constexpr uint32_t kLanes = D / 8;
    const uint32_t per_row = hkv * 2 * kLanes, u = id % per_row;
    t = id / per_row, h = u / (2 * kLanes), which = u / kLanes & 1, j = u % kLanes;
  }
  __device__ __forceinline__ int64_t row(int64_t ld) const { return (int64_t)t * ld + h * D + j * 8; }
  __device__ __forceinline__ uint64_t code(int32_t slot, int32_t hkv) const {
    return ((uint64_t)slot * hkv + h) * kv4_code_bytes(D) + which * (D / 2) + j * 4;
  }
  __device__ __forceinline__ uint64_t scale(int32_t slot, int32_t hkv) const {
    return ((uint64_t)slot * hkv + h) * kv4_scale_bytes(D) + which * (D / 32) + j / 4;
  }
};

// R pieces a lane, 256 ids apart, their loads all in flight: with one, a large
// call is bound by how many waves the chip holds (their whole life is two
// memory latencies).
template <class T, int D, int R>
__global__ __launch_bounds__(256) void kv4_store_kernel(const typename T::elem* __restrict__ k,
                                                        const typename T::elem* __restrict__ v, int64_t ld_k,
                                                        int64_t ld_v, const int32_t* __restrict__ slots,
                                                        int32_t num_tok, int32_t hkv, int32_t num_slots,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const uint32_t first = blockIdx.x * (256 * R) + threadIdx.x;  // a launch has at most 2^31 pieces
  Chunk<T> x[R];
  int32_t slot[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const Piece<D> p(first + 256 * i, hkv);
    slot[i] = -1;
    if (p.t < (uint32_t)num_tok) {
      slot[i] = slots[p.t];
      x[i].load(p.which ? v + p.row(ld_v) : k + p.row(ld_k));
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    // Whole rows are left out, so a group's 4 lanes stay together.
    if (slot[i] < 0 || slot[i] >= num_slots) continue;
    const Piece<D> p(first + 256 * i, hkv);
    const uint32_t top = quad_max(x[i].top());
    const int e = min(max((int)(top >> 23) - 2, kExpMin), kExpMax);
    const bool bad = top >= 0x7F800000u;
    *reinterpret_cast<uint32_t*>(codes + p.code(slot[i], hkv)) = bad ? 0u : x[i].codes(kv4_scale(e));
    if ((p.j & 3) == 0) scales[p.scale(slot[i], hkv)] = (uint8_t)(bad ? kExpNan : (uint32_t)e);
  }
}

// The rows' stores are non-temporal: they are a stream that the call itself
// does not read (131,264 slots x 4 heads, fp16: 52 us, 6.6 TB/s; 93 with cached
// stores).  Several pieces a lane gained nothing here.
template <class T, int D>
__global__ __launch_bounds__(256) void kv4_load_kernel(const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales, int32_t num_slots,
                                                       const int32_t* __restrict__ slots, int32_t n, int32_t hkv,
                                                       typename T::elem* __restrict__ k,
                                                       typename T::elem* __restrict__ v, int64_t ld_k, int64_t ld_v) {
  const Piece<D> p(blockIdx.x * 256 + threadIdx.x, hkv);
  if (p.t >= (uint32_t)n) return;
  const int32_t slot = slots[p.t];
  uint32_t c = 0, b = 127;
  if (slot >= 0 && slot < num_slots)
    c = *reinterpret_cast<const uint32_t*>(codes + p.code(slot, hkv)), b = scales[p.scale(slot, hkv)];
  Chunk<T> x;
  x.values(c, kv4_scale(b));
  x.store(p.which ? v + p.row(ld_v) : k + p.row(ld_k));
}

namespace {

// From here on a storing lane takes 4 pieces: 8,192 / 65,536 tokens x 8 heads of
// 128 (2^21 / 2^24 pieces) 8.7 / 68 us in place of 10.0 / 78; 4,096 tokens would
// lose (5.5 for 5.2).
constexpr int64_t kManyPieces = 1 << 21;

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

// Calls f(first row, rows, pieces) for launches of at most 2^31 pieces.
template <class F>
int by_rows(int32_t rows, int32_t hkv, int32_t d, F f) {
  const int64_t lanes = (int64_t)2 * hkv * (d / 8), most = std::max<int64_t>(1, ((int64_t)1 << 31) / lanes);
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = std::min<int64_t>(most, rows - r), pieces = n * lanes;
    f(r, (int32_t)n, pieces);
    if (hipGetLastError() != hipSuccess) return BS_ERR_LAUNCH;
  }
  return BS_OK;
}

}  // namespace

int launch_kv4_store(const void* k, const void* v, int32_t dtype, int64_t ld_k, int64_t ld_v, const int32_t* slots,
                     int32_t num_tok, int32_t hkv, int32_t d, uint8_t* codes, uint8_t* scales, int32_t num_slots,
                     hipStream_t stream) {
  return by_type_and_dim(dtype, d, [&](auto t, auto dim) {
    typedef decltype(t) T;
    typedef typename T::elem elem;
    return by_rows(num_tok, hkv, d, [&](int64_t r, int32_t n, int64_t pieces) {
      auto go = [&](auto each) {
        constexpr int R = decltype(each)::value;
        hipLaunchKernelGGL((kv4_store_kernel<T, decltype(dim)::value, R>), dim3((uint32_t)((pieces + 256 * R - 1) / (256 * R))),
                           dim3(256), 0, stream, static_cast<const elem*>(k) + r * ld_k, static_cast<const elem*>(v) + r * ld_v,
                           ld_k, ld_v, slots + r, n, hkv, num_slots, codes, scales);
      };
      if (pieces >= kManyPieces)
        go(std::integral_constant<int, 4>());
      else
        go(std::integral_constant<int, 1>());
    });
  });
}

int launch_kv4_load(const uint8_t* codes, const uint8_t* scales, int32_t num_slots, const int32_t* slots,
                    int32_t num_slot_ids, int32_t hkv, int32_t d, void* k, void* v, int32_t dtype, int64_t ld_k,
                    int64_t ld_v, hipStream_t stream) {
  return by_type_and_dim(dtype, d, [&](auto t, auto dim) {
    typedef decltype(t) T;
    typedef typename T::elem elem;
    return by_rows(num_slot_ids, hkv, d, [&](int64_t r, int32_t n, int64_t pieces) {
      hipLaunchKernelGGL((kv4_load_kernel<T, decltype(dim)::value>), dim3((uint32_t)((pieces + 255) / 256)), dim3(256), 0,
                         stream, codes, scales, num_slots, slots + r, n, hkv, static_cast<elem*>(k) + r * ld_k,
                         static_cast<elem*>(v) + r * ld_v, ld_k, ld_v);
    });
  });
}

}  // namespace bs
