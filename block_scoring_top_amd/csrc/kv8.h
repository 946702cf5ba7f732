// kv8.h - the 8-bit KV cache's number format on gfx950.
//
// A (page of 64 tokens, kv head, K or V) holds E4M3 codes (sign, 4 exponent
// bits, 3 mantissa bits, largest value 448, two NaN and no infinity) and one
// scale, a power of two: code x stands for x * scale.  The codes have an
// exponent of their own, so a scale need only keep a page's largest value in
// range; as a power of two it rounds nothing, neither where codes are read (4
// significant bits are a bf16 value exactly, and the hardware's conversion takes
// the scale along) nor, but for values that become subnormal codes, where a
// page's scale is raised and its codes are written anew.
#pragma once

#include "kv4.h"

namespace bs {

constexpr float kTop8 = 448.f;               // largest E4M3 value
constexpr int kExpMin8 = 7, kExpMax8 = 246;  // biased exponents of a scale: 2^-120 .. 2^119, 448 times which is finite

// Nonzero where one of four codes is NaN.
__device__ __forceinline__ uint32_t kv8_nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// The least scale (as its biased exponent) of a page whose largest finite
// magnitude has the FP32 bit pattern `top`: top <= 448 * scale = 1.75 * 2^8 * scale.
__device__ __forceinline__ int kv8_exponent(uint32_t top) {
  const int e = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u);
  return min(max(e, kExpMin8), kExpMax8);
}

// Two values, already over their scale, as codes in the low or high half of `old`:
// nearest, ties to even, at most 448, and NaN for infinities and NaN.
template <bool HIGH>
__device__ __forceinline__ uint32_t kv8_pack(uint32_t old, float x, float y) {
  auto fit = [](float v) {
    const float t = __builtin_amdgcn_fmed3f(v, -kTop8, kTop8);
    return fabsf(v) < INFINITY ? t : __builtin_nanf("");
  };
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fit(x), fit(y), (int)old, HIGH);
}

}  // namespace bs
