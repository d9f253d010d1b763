// Device helpers shared by the attention-side kernels.
#pragma once
#include "attn_launch.hpp"
#include "device_common.hpp"

namespace ql {

typedef __attribute__((ext_vector_type(2))) float f32x2_t;

// Two fp32 values rounded to nearest even into one word.
__device__ __forceinline__ uint32_t pack2(BF16, float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}
__device__ __forceinline__ uint32_t pack2(F16, float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, f16x2_t));
}

}  // namespace ql
