// kv4.h - the 4-bit KV cache's number format on gfx950.
//
// A group of 32 channels of one (slot, kv head, K or V) row holds 32 E2M1
// codes (sign, 2 exponent bits, 1 mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6)
// and one biased power-of-two exponent byte b; code x stands for x * 2^(b-127).
// This is the block format CDNA4 converts in hardware, two codes an
// instruction, and every such value is a bf16 value exactly (1 mantissa bit),
// so reading the cache rounds nothing.  Layout: BLOCK comment of kv4_store in
// blockscore.h.
#pragma once

#include "device.h"

namespace bs {

constexpr int kGroup = 32;          // channels per scale
constexpr int kExpMin = 7;          // scale byte of 2^-120: all values of a group stay normal in bf16 and fp32
constexpr int kExpMax = 252;        // 2^125: 6 * 2^125 is finite in bf16 and fp32
constexpr uint32_t kExpNan = 255;   // the group held an infinity or a NaN: every value reads back as NaN

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef int16_t i16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Bytes of one (slot, kv head): K codes then V codes; K scales then V scales.
__host__ __device__ constexpr int kv4_code_bytes(int d) { return d; }
__host__ __device__ constexpr int kv4_scale_bytes(int d) { return d / 16; }

// The scale a byte stands for; 255 becomes an infinite scale, which the
// conversions turn into NaN.
__device__ __forceinline__ float kv4_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// 16-bit element types of the kernels' operands.
struct Bf16 {
  typedef __bf16 elem;
  typedef bf16x2_t vec2;
  typedef bf16x8_t vec8;
  template <int SEL>
  static __device__ __forceinline__ uint32_t from_fp4(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, SEL));
  }
  template <int SEL>
  static __device__ __forceinline__ uint32_t to_fp4(uint32_t old, uint32_t two, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(vec2, two), scale, SEL);
  }
  // Two E4M3 codes, the low (SEL 0) or the high ones of four.
  template <int SEL>
  static __device__ __forceinline__ uint32_t from_fp8(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, SEL != 0));
  }
  // And back: nearest, ties to even; for finite values of at most 448 scales.
  template <int SEL>
  static __device__ __forceinline__ i16x2_t to_fp8(i16x2_t old, uint32_t two, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(old, __builtin_bit_cast(vec2, two), scale, SEL != 0);
  }
  // Bit pattern of |x| in 32 bits, for both halves of a pair.
  static __device__ __forceinline__ uint32_t abs_bits(uint32_t two) {
    return max((two << 16) & 0x7FFF0000u, two & 0x7FFF0000u);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, vec2));
  }
  static __device__ __forceinline__ f32x4_t mfma16(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(vec8, a), __builtin_bit_cast(vec8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) { return dot2_bf16(a, b, c); }
  static constexpr uint32_t kExpMask = 0x7F807F80u, kExpLsb = 0x00800080u;  // exponent fields of a pair
  static constexpr uint32_t kOne = 0x3F80u, k64 = 0x4280u, k65 = 0x4282u;
  static constexpr float kTopScale = 0x1p125f;   // a larger scale times 6 is not finite
  static constexpr float kTopScale8 = 0x1p119f;  // nor one times 448
  static constexpr float kRaise = 0.f;          // log2 of what attention weights are multiplied by
};

struct F16 {
  typedef _Float16 elem;
  typedef f16x2_t vec2;
  typedef f16x8_t vec8;
  template <int SEL>
  static __device__ __forceinline__ uint32_t from_fp4(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, SEL));
  }
  template <int SEL>
  static __device__ __forceinline__ uint32_t to_fp4(uint32_t old, uint32_t two, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(vec2, two), scale, SEL);
  }
  // Two E4M3 codes, the low (SEL 0) or the high ones of four.
  template <int SEL>
  static __device__ __forceinline__ uint32_t from_fp8(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, SEL != 0));
  }
  // And back: nearest, ties to even; for finite values of at most 448 scales.
  template <int SEL>
  static __device__ __forceinline__ i16x2_t to_fp8(i16x2_t old, uint32_t two, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(old, __builtin_bit_cast(vec2, two), scale, SEL != 0);
  }
  static __device__ __forceinline__ uint32_t abs_bits(uint32_t two) {
    const vec2 h = __builtin_bit_cast(vec2, two);
    return max(__float_as_uint((float)h.x) & 0x7FFFFFFFu, __float_as_uint((float)h.y) & 0x7FFFFFFFu);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, vec2));
  }
  static __device__ __forceinline__ f32x4_t mfma16(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(vec8, a), __builtin_bit_cast(vec8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(vec2, a), __builtin_bit_cast(vec2, b), c, false);
  }
  static constexpr uint32_t kExpMask = 0x7C007C00u, kExpLsb = 0x04000400u;
  static constexpr uint32_t kOne = 0x3C00u, k64 = 0x5400u, k65 = 0x5410u;
  static constexpr float kTopScale = 0x1p13f, kTopScale8 = 0x1p7f;
  // A weight of 1 relative to the running maximum is held as 2^7: with weights
  // up to 2^8 (kSlack) still in range, weights keep all their bits down to
  // 2^-21 of the maximum and vanish below 2^-32.  With a 1 held as 1 these
  // would be 2^-14 and 2^-25: beside a dominating key whose values are 0, 32,768
  // others at 2^-26 then add up to nothing.
  static constexpr float kRaise = 7.f;
};

struct F32 {
  typedef float elem;
};

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

}  // namespace bs
