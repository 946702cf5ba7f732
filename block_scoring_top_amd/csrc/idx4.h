// idx4.h - the 4-bit index keys.
//
// A key's 128 channels are E2M1 codes (channel 2i in the low nibble of byte i)
// with one biased power-of-two exponent byte per 32 channels: the number format
// of the 4-bit KV cache (kv4.h), 68 bytes a key in place of bf16's 256, and the
// operand format of the scaled matrix instructions, which take codes and
// exponents as they are stored.
#pragma once

#include "kv4.h"

namespace bs {

constexpr int kIdxCodes = kDim / 2, kIdxScales = kDim / kGroup;  // bytes of a key

// The exponent byte of a group whose largest magnitude has the bit pattern
// `top`, and whether it holds an infinity or a NaN.
__device__ __forceinline__ uint32_t group_exponent(uint32_t top, bool& bad) {
  bad = top >= 0x7F800000u;
  return (uint32_t)min(max((int)(top >> 23) - 2, kExpMin), kExpMax);
}

}  // namespace bs
