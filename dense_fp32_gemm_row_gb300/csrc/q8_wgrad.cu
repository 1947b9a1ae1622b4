// q8_wgrad.cu -- the weight gradient of a linear layer from the 8-bit
// checkpoint of its input:
//
//     dW[d][n] = alpha sum_t x^[t][d] dY[t][n] + beta dW[d][n]
//
// x^ is decoded inside the kernel (codes times a power of two, exact), so
// the product reads a byte an element of X where an fp32 checkpoint reads
// four, and no decoded copy is written.
//
// The CUDA-core form: 64 x 64 tiles of dW, 256 threads with 4 x 4 outputs
// each, 16 tokens a step through shared memory; sums over 256 tokens are
// added into a second accumulator, so that the rounding error of a long sum
// grows with the number of such chunks and not with the number of tokens.
// It is for small calls (a few tokens, small outputs), which are bound by the
// launch: 16 x 512 x 512 takes 5.6 us against 6.3 on the tensor core (replayed
// from a graph 2.7 against 5.8).
#include <cstdint>

#include "device_sync.cuh"
#include "epilogue.cuh"
#include "gemm_internal.h"
#include "q8_format.cuh"

namespace gemm_f32_impl {
namespace {

using namespace gemm_f32_dev;

constexpr int kTile = 64;
constexpr int kStep = 16;
constexpr int kChunk = 256;

template <int FMT>
__global__ void __launch_bounds__(256)
q8_wgrad_ffma_kernel(Q8In x, int rows, int cols, const float* __restrict__ dy, long long lddy,
                     int N, float* __restrict__ dw, long long lddw, float alpha, float beta,
                     int mode) {
    __shared__ float xs[kStep][kTile];
    __shared__ float ys[kStep][kTile];
    const int tid = threadIdx.x;
    const int n0 = blockIdx.x * kTile;
    const int tx = tid & 15, ty = tid >> 4;
    // loads: token tid / 16 of the step, four columns from 4 (tid % 16)
    const int lt = tid >> 4, lc = 4 * (tid & 15);
    for (long long d0 = blockIdx.y * kTile; d0 < cols; d0 += gridDim.y * kTile) {
        float sum[4][4] = {}, acc[4][4];
        for (long long t0 = 0; t0 < rows; t0 += kChunk) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
            const long long t1 = min(static_cast<long long>(rows), t0 + kChunk);
            for (long long tb = t0; tb < t1; tb += kStep) {
                const long long t = tb + lt;
                const bool in = t < rows;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const long long d = d0 + lc + i;
                    const int n = n0 + lc + i;
                    float v = 0.0f;
                    if (in && d < cols)
                        v = q8_decode4<FMT>(x.codes[t * x.ldcodes + d]).x *
                            q8_scale<FMT>(x.scales[t * x.ldscales + d / kQ8Block]);
                    xs[lt][lc + i] = v;
                    ys[lt][lc + i] = in && n < N ? dy[t * lddy + n] : 0.0f;
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kStep; ++k) {
                    const float4 a = *reinterpret_cast<const float4*>(&xs[k][4 * ty]);
                    const float4 b = *reinterpret_cast<const float4*>(&ys[k][4 * tx]);
                    const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
                }
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[i][j] += acc[i][j];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long d = d0 + 4 * ty + i;
            if (d >= cols) break;
            float* row = dw + d * lddw;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + 4 * tx + j;
                if (n < N) row[n] = scale1(sum[i][j], row + n, alpha, beta, mode);
            }
        }
    }
}

}  // namespace

cudaError_t launch_q8_wgrad_ffma(const Q8WgradArgs& a, cudaStream_t s) {
    const unsigned tiles_d = (static_cast<unsigned>(a.cols) + kTile - 1) / kTile;
    const dim3 grid((static_cast<unsigned>(a.N) + kTile - 1) / kTile,
                    tiles_d < 65535u ? tiles_d : 65535u);
    if (a.format == kQ8Int8)
        q8_wgrad_ffma_kernel<kQ8Int8><<<grid, 256, 0, s>>>(a.x, a.rows, a.cols, a.dy, a.lddy, a.N,
                                                           a.dw, a.lddw, a.alpha, a.beta, a.mode);
    else
        q8_wgrad_ffma_kernel<kQ8E4m3><<<grid, 256, 0, s>>>(a.x, a.rows, a.cols, a.dy, a.lddy, a.N,
                                                           a.dw, a.lddw, a.alpha, a.beta, a.mode);
    return cudaGetLastError();
}

}  // namespace gemm_f32_impl
