// i8_output.cuh -- from integer sums to the outputs of the 8-bit integer
// products.
#pragma once

#include <cuda_bf16.h>

#include "activation.cuh"

namespace gemm_f32_dev {

constexpr int kI8Float = 0;
constexpr int kI8Bfloat16 = 1;
constexpr int kI8Int32 = 2;

// The value of a sum, the token's scale first: three roundings to fp32 (the
// sum's own where it is beyond 2^24).
__device__ __forceinline__ float i8_value(int sum, float token, float channel) {
    return __fmul_rn(__fmul_rn(__int2float_rn(sum), token), channel);
}

__device__ __forceinline__ float i8_gate(int act, float g, float u) {
    return (act == kActSilu ? act_value<kActSilu>(g) : act_value<kActGelu>(g)) * u;
}

__device__ __forceinline__ void put_output(void* y, long long at, int type, float v) {
    if (type == kI8Bfloat16)
        static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(y)[at] = v;
}

}  // namespace gemm_f32_dev
