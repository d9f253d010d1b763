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

// The exponent t for which a row of largest magnitude amax (of bf16 values) has amax 2^-t in [2^14, 2^15).
__device__ __forceinline__ int q_exponent(float amax) {
  const int e = (int)(__float_as_uint(amax) >> 23) - 127 - 14;
  return amax == 0.f ? 0 : min(100, max(-100, e));
}
// Eight bf16 or fp16 values as fp16 pairs (i, i + 4), the order in which a word's codes are decoded;
// bf16 values times 2^-t.
__device__ __forceinline__ u32x4_t q_pairs(u32x4_t w, int dt, float factor) {
  uint32_t lo[4] = {w[0] & 0xffffu, w[0] >> 16, w[1] & 0xffffu, w[1] >> 16};
  uint32_t hi[4] = {w[2] & 0xffffu, w[2] >> 16, w[3] & 0xffffu, w[3] >> 16};
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = dt == DT_BF16 ? pack2(F16{}, bf16_bits_to_f32(lo[i]) * factor, bf16_bits_to_f32(hi[i]) * factor)
                         : lo[i] | (hi[i] << 16);
  return r;
}
__device__ __forceinline__ float amax8(u32x4_t w, float m) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = fmaxf(m, fmaxf(__builtin_fabsf(__uint_as_float(w[i] << 16)), __builtin_fabsf(__uint_as_float(w[i] & 0xffff0000u))));
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
