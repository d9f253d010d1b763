// Rows of a cache in 4 bits: d codes, eight a word with the lowest bits first (the affine rows of the
// quantized weights), and per group of 32, 64 or 128 values one word of two fp16 numbers, the scale in
// its low half and the bias in its high half.  A value is code * scale + bias.
#pragma once
#include "head_common.hpp"

namespace ql {

__device__ __forceinline__ f16x2_t h2(uint32_t w) { return __builtin_bit_cast(f16x2_t, w); }
__device__ __forceinline__ uint32_t w2(f16x2_t h) { return __builtin_bit_cast(uint32_t, h); }

// The values of a word as fp16 pairs (i, i + 4), i = 0 .. 3, each rounded once.  A code under the exponent bits
// of 1024 (its low bits) or of 64 (four bits further up) is 1024 + c or 64 + c, and the difference is exact.
__device__ __forceinline__ u32x4_t values4(uint32_t w, uint32_t group) {
  const f16x2_t p = h2(group), s = {p[0], p[0]}, b = {p[1], p[1]};
  const f16x2_t k1024 = h2(0x64006400u), k64 = h2(0x54005400u);
  const uint32_t v = w >> 8;
  const f16x2_t c[4] = {h2((w & 0x000f000fu) | 0x64006400u) - k1024, h2((w & 0x00f000f0u) | 0x54005400u) - k64,
                        h2((v & 0x000f000fu) | 0x64006400u) - k1024, h2((v & 0x00f000f0u) | 0x54005400u) - k64};
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = w2(__builtin_elementwise_fma(c[i], s, b));
  return r;
}

}  // namespace ql
