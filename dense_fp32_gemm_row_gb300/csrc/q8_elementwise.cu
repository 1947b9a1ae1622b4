// q8_elementwise.cu -- the elementwise kernels of the 8-bit activation
// checkpoints: store, restore, and the gated unit's forward and backward
// pass, which keep and read their operands in that form.
//
//   store     codes, exponents = q8(x)
//   restore   x^ = value(codes, exponents)                 (fp32 or bf16)
//   gated     h = act(g) u; q8(g); q8(u)                   one pass
//   backward  du = dh act(g^); dg = dh u^ act'(g^); q8(act(g^) u^)
//
//   silu  act(z) = z s(z), s(z) = 1 / (1 + e^-z);  act'(z) = s (1 + z (1 - s))
//   gelu  act(z) = z P(z), P the normal distribution function;
//         act'(z) = P(z) + z e^(-z^2/2) / sqrt(2 pi)
//
// Every value is read once and written once; the kernels are bounded by HBM
// bandwidth at size and by launch latency below it.
//
// One warp takes one block of 32 columns of one row, a lane a column: the
// block's largest magnitude is one warp-wide integer maximum, loads and
// stores are coalesced whatever the strides and alignment, and a ragged last
// block is a predicate.
#include <cstdint>

#include <cuda_bf16.h>

#include "device_sync.cuh"
#include "gemm_internal.h"
#include "q8_format.cuh"

namespace gemm_f32_impl {
namespace {

using namespace gemm_f32_dev;

constexpr int kThreads = 256;
constexpr int kActSilu = 0;
constexpr int kActGelu = 1;

// act(z) and act'(z) in fp32.  erfc keeps P's relative accuracy in the
// lower tail, where 1 + erf cancels.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == kActSilu) return z * (1.0f / (1.0f + expf(-z)));
    return z * (0.5f * erfcf(-0.70710678118654752f * z));
}
template <int ACT>
__device__ __forceinline__ void act_both(float z, float* value, float* slope) {
    if (ACT == kActSilu) {
        const float s = 1.0f / (1.0f + expf(-z));
        *value = z * s;
        *slope = s * fmaf(z, 1.0f - s, 1.0f);
    } else {
        const float p = 0.5f * erfcf(-0.70710678118654752f * z);
        *value = z * p;
        *slope = fmaf(z * expf(-0.5f * z * z), 0.39894228040143268f, p);
    }
}

// One lane's column of the warp's block.
struct Place {
    long long row;
    int block, col;
    bool live;
};
__device__ __forceinline__ Place place(long long item, int nblocks, int cols, int lane) {
    Place p;
    p.row = item / nblocks;
    p.block = static_cast<int>(item - p.row * nblocks);
    p.col = p.block * kQ8Block + lane;
    p.live = p.col < cols;
    return p;
}

template <int FMT>
__device__ __forceinline__ void store_lane(float x, const Place& p, int lane,
                                           unsigned char* codes, long long ldcodes,
                                           unsigned char* scales, long long ldscales) {
    const unsigned e = q8_exponent<FMT>(__reduce_max_sync(0xFFFFFFFFu, q8_magnitude(x)));
    const unsigned w = q8_encode4<FMT>(x, 0.0f, 0.0f, 0.0f, q8_inverse_scale<FMT>(e), e);
    if (p.live) codes[p.row * ldcodes + p.col] = static_cast<unsigned char>(w);
    if (lane == 0) scales[p.row * ldscales + p.block] = static_cast<unsigned char>(e);
}

template <int FMT>
__device__ __forceinline__ float load_lane(const Place& p, const unsigned char* codes,
                                           long long ldcodes, const unsigned char* scales,
                                           long long ldscales) {
    if (!p.live) return 0.0f;
    const unsigned e = scales[p.row * ldscales + p.block];
    return q8_decode4<FMT>(codes[p.row * ldcodes + p.col]).x * q8_scale<FMT>(e);
}

#define Q8_FOR_EACH_BLOCK                                                                       \
    const int lane = threadIdx.x & 31;                                                          \
    const int nblocks = (cols + kQ8Block - 1) / kQ8Block;                                       \
    const long long items = static_cast<long long>(rows) * nblocks;                             \
    for (long long item = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;   \
         item < items; item += (static_cast<long long>(gridDim.x) * kThreads) >> 5)

template <int FMT>
__global__ void __launch_bounds__(kThreads)
q8_store_kernel(const float* x, long long ldx, int rows, int cols, Q8Out q) {
    Q8_FOR_EACH_BLOCK {
        const Place p = place(item, nblocks, cols, lane);
        const float v = p.live ? x[p.row * ldx + p.col] : 0.0f;
        store_lane<FMT>(v, p, lane, q.codes, q.ldcodes, q.scales, q.ldscales);
    }
}

template <int FMT, typename T>
__global__ void __launch_bounds__(kThreads)
q8_restore_kernel(Q8In q, int rows, int cols, T* x, long long ldx) {
    Q8_FOR_EACH_BLOCK {
        const Place p = place(item, nblocks, cols, lane);
        const float v = load_lane<FMT>(p, q.codes, q.ldcodes, q.scales, q.ldscales);
        if (p.live) x[p.row * ldx + p.col] = static_cast<T>(v);
    }
}

template <int FMT, int ACT>
__global__ void __launch_bounds__(kThreads)
q8_gated_kernel(const float* g, long long ldg, const float* u, long long ldu, int rows, int cols,
                float* h, long long ldh, Q8Out gq, Q8Out uq) {
    Q8_FOR_EACH_BLOCK {
        const Place p = place(item, nblocks, cols, lane);
        const float gv = p.live ? g[p.row * ldg + p.col] : 0.0f;
        const float uv = p.live ? u[p.row * ldu + p.col] : 0.0f;
        if (p.live) h[p.row * ldh + p.col] = act_value<ACT>(gv) * uv;
        store_lane<FMT>(gv, p, lane, gq.codes, gq.ldcodes, gq.scales, gq.ldscales);
        store_lane<FMT>(uv, p, lane, uq.codes, uq.ldcodes, uq.scales, uq.ldscales);
    }
}

template <int FMT, int ACT>
__global__ void __launch_bounds__(kThreads)
q8_gated_backward_kernel(Q8In gq, Q8In uq, const float* dh, long long lddh, int rows, int cols,
                         float* dg, long long lddg, float* du, long long lddu, Q8Out hq) {
    Q8_FOR_EACH_BLOCK {
        const Place p = place(item, nblocks, cols, lane);
        const float gv = load_lane<FMT>(p, gq.codes, gq.ldcodes, gq.scales, gq.ldscales);
        const float uv = load_lane<FMT>(p, uq.codes, uq.ldcodes, uq.scales, uq.ldscales);
        const float d = p.live ? dh[p.row * lddh + p.col] : 0.0f;
        float a, da;
        act_both<ACT>(gv, &a, &da);
        if (p.live) {
            dg[p.row * lddg + p.col] = d * uv * da;
            du[p.row * lddu + p.col] = d * a;
        }
        if (hq.codes)
            store_lane<FMT>(p.live ? a * uv : 0.0f, p, lane, hq.codes, hq.ldcodes, hq.scales,
                            hq.ldscales);
    }
}

unsigned grid_for(int rows, int cols) {
    const long long items = static_cast<long long>(rows) * ((cols + kQ8Block - 1) / kQ8Block);
    const long long blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
    return static_cast<unsigned>(blocks < 152 * 16 ? blocks : 152 * 16);
}

}  // namespace

cudaError_t launch_q8_store(const float* x, long long ldx, int rows, int cols, int format,
                            const Q8Out& q, cudaStream_t s) {
    const unsigned grid = grid_for(rows, cols);
    if (format == kQ8Int8)
        q8_store_kernel<kQ8Int8><<<grid, kThreads, 0, s>>>(x, ldx, rows, cols, q);
    else
        q8_store_kernel<kQ8E4m3><<<grid, kThreads, 0, s>>>(x, ldx, rows, cols, q);
    return cudaGetLastError();
}

cudaError_t launch_q8_restore(const Q8In& q, int rows, int cols, int format, void* x,
                              long long ldx, int bf16, cudaStream_t s) {
    const unsigned grid = grid_for(rows, cols);
    if (format == kQ8Int8) {
        if (bf16)
            q8_restore_kernel<kQ8Int8><<<grid, kThreads, 0, s>>>(
                q, rows, cols, static_cast<__nv_bfloat16*>(x), ldx);
        else
            q8_restore_kernel<kQ8Int8><<<grid, kThreads, 0, s>>>(q, rows, cols,
                                                                static_cast<float*>(x), ldx);
    } else {
        if (bf16)
            q8_restore_kernel<kQ8E4m3><<<grid, kThreads, 0, s>>>(
                q, rows, cols, static_cast<__nv_bfloat16*>(x), ldx);
        else
            q8_restore_kernel<kQ8E4m3><<<grid, kThreads, 0, s>>>(q, rows, cols,
                                                                static_cast<float*>(x), ldx);
    }
    return cudaGetLastError();
}

namespace {

template <int FMT, int ACT>
void gated(const GatedArgs& a, cudaStream_t s) {
    q8_gated_kernel<FMT, ACT><<<grid_for(a.rows, a.cols), kThreads, 0, s>>>(
        a.g, a.ldg, a.u, a.ldu, a.rows, a.cols, a.h, a.ldh, a.gq, a.uq);
}
template <int FMT, int ACT>
void gated_backward(const GatedBackwardArgs& a, cudaStream_t s) {
    q8_gated_backward_kernel<FMT, ACT><<<grid_for(a.rows, a.cols), kThreads, 0, s>>>(
        a.gq, a.uq, a.dh, a.lddh, a.rows, a.cols, a.dg, a.lddg, a.du, a.lddu, a.hq);
}

}  // namespace

cudaError_t launch_q8_gated(const GatedArgs& a, cudaStream_t s) {
    if (a.format == kQ8Int8)
        a.act == kActSilu ? gated<kQ8Int8, kActSilu>(a, s) : gated<kQ8Int8, kActGelu>(a, s);
    else
        a.act == kActSilu ? gated<kQ8E4m3, kActSilu>(a, s) : gated<kQ8E4m3, kActGelu>(a, s);
    return cudaGetLastError();
}

cudaError_t launch_q8_gated_backward(const GatedBackwardArgs& a, cudaStream_t s) {
    if (a.format == kQ8Int8)
        a.act == kActSilu ? gated_backward<kQ8Int8, kActSilu>(a, s)
                          : gated_backward<kQ8Int8, kActGelu>(a, s);
    else
        a.act == kActSilu ? gated_backward<kQ8E4m3, kActSilu>(a, s)
                          : gated_backward<kQ8E4m3, kActGelu>(a, s);
    return cudaGetLastError();
}

}  // namespace gemm_f32_impl
