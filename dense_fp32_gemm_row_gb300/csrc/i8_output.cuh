// i8_output.cuh -- from integer sums to the outputs of the 8-bit integer
// products.
#pragma once

#include <cuda_bf16.h>

#include "activation.cuh"

namespace gemm_f32_dev {

constexpr int kI8Float = 0;
constexpr int kI8Bfloat16 = 1;
constexpr int kI8Int32 = 2;

// The value of a sum, as a float (rounded where it is beyond 2^24), the token's
// scale first.
__device__ __forceinline__ float i8_value(float sum, float token, float channel) {
    return __fmul_rn(__fmul_rn(sum, token), channel);
}

// act(z) with the quotient of silu to 2 ulp (act_value rounds it correctly):
// the sums' own roundings are as large.
template <int ACT>
__device__ __forceinline__ float i8_act(float z) {
    return ACT == kActSilu ? __fdividef(z, 1.0f + expf(-z)) : act_value<kActGelu>(z);
}

}  // namespace gemm_f32_dev
