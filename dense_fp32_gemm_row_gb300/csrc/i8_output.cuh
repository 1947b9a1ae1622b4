// i8_output.cuh -- what the kernels of the 8-bit integer products share: from
// codes to fp16 numbers, and from sums to outputs.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

#include "activation.cuh"

namespace gemm_f32_dev {

constexpr int kI8Float = 0;
constexpr int kI8Bfloat16 = 1;
constexpr int kI8Int32 = 2;
constexpr int kI8NoAct = -1;  // not the gated product

// Four codes as two words of two fp16 numbers: a code's bits, offset to be positive,
// in the mantissa of 1024 are 1024 plus that number (for fp16 weights: Kim, Henry,
// Fahim and Awadalla, "Who Says Elephants Can't Run", 2022).
__device__ __forceinline__ void decode_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t bias = 0x64806480u;  // 1024 + 128, twice
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(bias));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(bias));
}

__device__ __forceinline__ void decode_f16(const uint4& w, uint32_t (&h)[8]) {
    decode_f16(w.x, h[0], h[1]);
    decode_f16(w.y, h[2], h[3]);
    decode_f16(w.z, h[4], h[5]);
    decode_f16(w.w, h[6], h[7]);
}

// The value of a sum, as a float (rounded where it is beyond 2^24), the token's
// scale first.
__device__ __forceinline__ float i8_value(float sum, float token, float channel) {
    return __fmul_rn(__fmul_rn(sum, token), channel);
}

// act(z) with the quotient of silu to 2 ulp (act_value rounds it correctly): the
// sums' own roundings are as large, and act_value would make gated 8192 x 8192 x
// 4096 736 us of 638, 1000 x 1023 x 1025 11.7 of 9.8.  Where e^-z is beyond 2^126, z
// below -87.33, the quotient is 0 instead of up to 1.1e-36.
template <int ACT>
__device__ __forceinline__ float i8_act(float z) {
    return ACT == kActSilu ? __fdividef(z, 1.0f + expf(-z)) : act_value<kActGelu>(z);
}

}  // namespace gemm_f32_dev
