// i8_dp4a.cu -- the product of 8-bit integer matrices on the CUDA cores, four
// products an instruction (dp4a), sums in 32-bit integers.
//
//   y[t][n] = (sum_k a[t][k] b[n][k]) sa[t] sb[n]
//   gated: h = act(g) u of two such products
//
// A block of 256 threads computes 64 x 64 outputs, 4 x 4 a thread, from 64-byte
// stretches of 64 rows of each operand in shared memory.
#include <cstdint>

#include "device_sync.cuh"
#include "gemm_internal.h"
#include "i8_output.cuh"

namespace gemm_f32_impl {
namespace {

using namespace gemm_f32_dev;

constexpr int kTile = 64, kWords = 16, kPitch = kWords + 1;

// 64 bytes of 64 rows from column k0; what lies outside the matrix is zero.
__device__ __forceinline__ void stage(int (*dst)[kPitch], const I8In& m, int row0, int rows,
                                      int k0, int K) {
    const int r = threadIdx.x / 4, c = threadIdx.x % 4;
    int4 w = make_int4(0, 0, 0, 0);
    const int k = k0 + 16 * c;
    if (row0 + r < rows && k < K) {
        // row strides are multiples of 16 bytes
        w = *reinterpret_cast<const int4*>(m.codes + static_cast<long long>(row0 + r) * m.ld + k);
        int* p = &w.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int left = K - k - 4 * i;  // bytes of the word that are in the row
            if (left < 4) p[i] = left <= 0 ? 0 : p[i] & static_cast<int>((1u << (8 * left)) - 1u);
        }
    }
    dst[r][4 * c] = w.x, dst[r][4 * c + 1] = w.y, dst[r][4 * c + 2] = w.z, dst[r][4 * c + 3] = w.w;
}

template <bool GATED>
__global__ void __launch_bounds__(256) i8_dp4a_kernel(I8ProductArgs p) {
    __shared__ int as[kTile][kPitch], bs[GATED ? 2 : 1][kTile][kPitch];
    const int n0 = blockIdx.x * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    pdl_wait();
    pdl_trigger();
    for (long long t0 = static_cast<long long>(blockIdx.y) * kTile; t0 < p.T;
         t0 += static_cast<long long>(gridDim.y) * kTile) {
        int acc[GATED ? 2 : 1][4][4] = {};
        for (int k0 = 0; k0 < p.K; k0 += 4 * kWords) {
            __syncthreads();
            stage(as, p.a, static_cast<int>(t0), p.T, k0, p.K);
            stage(bs[0], p.b, n0, p.N, k0, p.K);
            if (GATED) stage(bs[GATED ? 1 : 0], p.c, n0, p.N, k0, p.K);
            __syncthreads();
#pragma unroll 4
            for (int w = 0; w < kWords; ++w) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int x = as[ty + 16 * i][w];
#pragma unroll
                    for (int g = 0; g < (GATED ? 2 : 1); ++g)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[g][i][j] = __dp4a(x, bs[g][tx + 16 * j][w], acc[g][i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long t = t0 + ty + 16 * i;
            if (t >= p.T) continue;
            const float st = p.a.scales[t];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx + 16 * j;
                if (n >= p.N) continue;
                if (GATED)
                    put_output(p.y, t * p.ldy + n, p.type,
                               i8_gate(p.act, i8_value(acc[0][i][j], st, p.b.scales[n]),
                                       i8_value(acc[GATED ? 1 : 0][i][j], st, p.c.scales[n])));
                else if (p.type == kI8Int32)
                    static_cast<int*>(p.y)[t * p.ldy + n] = acc[0][i][j];
                else
                    put_output(p.y, t * p.ldy + n, p.type,
                               i8_value(acc[0][i][j], st, p.b.scales[n]));
            }
        }
    }
}

}  // namespace

cudaError_t launch_i8_dp4a(const I8ProductArgs& p, cudaStream_t stream) {
    const int tiles = (p.T - 1) / kTile + 1;
    const dim3 grid((p.N - 1) / kTile + 1, tiles < 65535 ? tiles : 65535);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, p.c.codes ? i8_dp4a_kernel<true> : i8_dp4a_kernel<false>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gemm_f32_impl
