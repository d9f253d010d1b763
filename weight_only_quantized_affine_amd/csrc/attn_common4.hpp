// Paged attention over a cache in 4 bits: what the two kernels (attn_few4.hip, attn_tile.hip) share.
//
// Both products run in fp16 whatever the type of q and out: q enters as fp16 after an exact scaling of each
// row by a power of two that its scores take back, and the softmax weights round to fp16 (2^-12 of the value,
// where bf16 would take 2^-9).
#pragma once
#include <type_traits>

#include "attn_common.hpp"
#include "cache4.hpp"

namespace ql {

// The exponent t for which a row of largest magnitude amax has amax 2^-t in [2^14, 2^15).
__device__ __forceinline__ int q_exponent(float amax) {
  return amax == 0.f ? 0 : (int)(__float_as_uint(amax) >> 23) - 127 - 14;
}
__device__ __forceinline__ void q_values(u32x4_t w, int dt, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = dt == DT_BF16 ? bf16_bits_to_f32(w[i] & 0xffffu) : f16_bits_to_f32(w[i] & 0xffffu);
    f[2 * i + 1] = dt == DT_BF16 ? bf16_bits_to_f32(w[i] >> 16) : f16_bits_to_f32(w[i] >> 16);
  }
}
// Its scores' factor 2^t, cut where it passes fp32 (the scores then differ by more than weights can show).
__device__ __forceinline__ float q_scale(float sl, int t) { return fminf(__builtin_ldexpf(sl, t), 3.0e38f); }
// Eight bf16 or fp16 values times 2^-t as fp16 pairs (i, i + 4), the order in which a word's codes come apart.
__device__ __forceinline__ u32x4_t q_pairs(u32x4_t w, int dt, int t) {
  float f[8];
  q_values(w, dt, f);
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack2(F16{}, __builtin_ldexpf(f[i], -t), __builtin_ldexpf(f[i + 4], -t));
  return r;
}
__device__ __forceinline__ float amax8(u32x4_t w, int dt, float m) {
  float f[8];
  q_values(w, dt, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, __builtin_fabsf(f[i]));
  return m;
}

// Starts a copy of 4 bytes a lane into LDS (as copy16).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy4(const uint8_t* src, uint8_t* dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off nt"
               :
               : "s"(lds_at(dst)), "v"(src)
               : "memory", "m0");
}
// From a uniform base plus the lane's offset (as copy16_from).
__device__ __forceinline__ void copy4_from(int64_t base, uint32_t off, uint8_t* dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dword %1, %2 nt"
               :
               : "s"(lds_at(dst)), "v"(off), "s"(base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// The largest of the wave's values, uniform.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  auto step = [&](auto ctrl) {
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xf, 0xf, false));
  };
  step(std::integral_constant<int, 0xB1>{});
  step(std::integral_constant<int, 0x4E>{});
  step(std::integral_constant<int, 0x141>{});
  step(std::integral_constant<int, 0x140>{});
  const uint32_t a = max(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16));
  const uint32_t b = max(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48));
  return max(a, b);
}

}  // namespace ql
