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
// A warp takes a segment of 128 columns of one row, a lane four of them: a
// float4 of each matrix and a word of codes, so that every access of the warp
// is one contiguous run (512 and 128 bytes), and the 8 lanes of a block share
// its largest magnitude in three shuffles.  (A column a lane moved a quarter
// of the bytes an instruction: store and restore of 8192 x 8192 448 us, gated
// forward, backward and a restore 1086 us.)  A matrix whose base or row
// stride is not 16-byte aligned is read and written a float at a time, and so
// are the last columns of a ragged row.  Each warp keeps several segments in
// flight and walks the segments with the grid's stride, without divisions.
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

constexpr int kSegment = 128;  // columns of a warp

// The segments of a matrix, walked by the warps of the grid.
struct Walk {
    long long row, drow;
    int seg, dseg, per_row;
    __device__ __forceinline__ Walk(int cols) {
        per_row = (cols - 1) / kSegment + 1;
        const unsigned warp = (blockIdx.x * kThreads + threadIdx.x) >> 5;
        const unsigned warps = gridDim.x * (kThreads / 32);
        row = warp / static_cast<unsigned>(per_row);
        seg = static_cast<int>(warp % static_cast<unsigned>(per_row));
        drow = warps / static_cast<unsigned>(per_row);
        dseg = static_cast<int>(warps % static_cast<unsigned>(per_row));
    }
    __device__ __forceinline__ void next() {
        row += drow;
        seg += dseg;
        if (seg >= per_row) {
            seg -= per_row;
            ++row;
        }
    }
};

// One lane's place in a segment: four columns from col (those below cols).
struct Place {
    long long row;
    int col, block;
    int n;  // columns of the matrix among the four: 0 .. 4
};
__device__ __forceinline__ Place place(const Walk& w, int rows, int cols, int lane) {
    Place p;
    p.row = w.row;
    const long long col = static_cast<long long>(w.seg) * kSegment + 4 * lane;
    const long long left = w.row < rows ? cols - col : 0;
    p.n = left >= 4 ? 4 : left > 0 ? static_cast<int>(left) : 0;
    p.col = p.n ? static_cast<int>(col) : 0;
    p.block = p.col / kQ8Block;
    return p;
}

__device__ __forceinline__ float4 load4(const float* m, long long ld, bool vec, const Place& p) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float* a = m + p.row * ld + p.col;
    if (p.n == 4 && vec) {
        v = *reinterpret_cast<const float4*>(a);
    } else {
        if (p.n > 0) v.x = a[0];
        if (p.n > 1) v.y = a[1];
        if (p.n > 2) v.z = a[2];
        if (p.n > 3) v.w = a[3];
    }
    return v;
}

__device__ __forceinline__ void put4(float* m, long long ld, bool vec, const Place& p, float4 v) {
    float* a = m + p.row * ld + p.col;
    if (p.n == 4 && vec) {
        *reinterpret_cast<float4*>(a) = v;
    } else {
        if (p.n > 0) a[0] = v.x;
        if (p.n > 1) a[1] = v.y;
        if (p.n > 2) a[2] = v.z;
        if (p.n > 3) a[3] = v.w;
    }
}
// bf16, rounding nothing: the values of a checkpoint are exact in it
__device__ __forceinline__ void put4(__nv_bfloat16* m, long long ld, bool vec, const Place& p,
                                     float4 v) {
    unsigned short* a = reinterpret_cast<unsigned short*>(m) + p.row * ld + p.col;
    const uint2 w = make_uint2(__byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632),
                               __byte_perm(__float_as_uint(v.z), __float_as_uint(v.w), 0x7632));
    if (p.n == 4 && vec) {
        *reinterpret_cast<uint2*>(a) = w;
    } else {
        if (p.n > 0) a[0] = static_cast<unsigned short>(w.x);
        if (p.n > 1) a[1] = static_cast<unsigned short>(w.x >> 16);
        if (p.n > 2) a[2] = static_cast<unsigned short>(w.y);
        if (p.n > 3) a[3] = static_cast<unsigned short>(w.y >> 16);
    }
}

// Encode a lane's four values (zeros beyond the row) with its block's 8 lanes
// and write codes and exponent.
template <int FMT>
__device__ __forceinline__ void encode4(float4 v, const Place& p, int lane, const Q8Out& q) {
    unsigned m = max(max(q8_magnitude(v.x), q8_magnitude(v.y)),
                     max(q8_magnitude(v.z), q8_magnitude(v.w)));
#pragma unroll
    for (int d = 1; d < 8; d *= 2) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    const unsigned e = q8_exponent<FMT>(m);
    const unsigned w = q8_encode4<FMT>(v.x, v.y, v.z, v.w, q8_inverse_scale<FMT>(e), e);
    unsigned char* c = q.codes + p.row * q.ldcodes + p.col;
    if (p.n == 4) {
        *reinterpret_cast<unsigned*>(c) = w;
    } else {
        if (p.n > 0) c[0] = static_cast<unsigned char>(w);
        if (p.n > 1) c[1] = static_cast<unsigned char>(w >> 8);
        if (p.n > 2) c[2] = static_cast<unsigned char>(w >> 16);
    }
    if ((lane & 7) == 0 && p.n > 0)
        q.scales[p.row * q.ldscales + p.block] = static_cast<unsigned char>(e);
}

// A lane's code word (bytes beyond the row are the caller's and not used) and
// exponent byte.
struct Held {
    unsigned w, e;
};
__device__ __forceinline__ Held load_held(const Q8In& q, const Place& p) {
    Held h = {0u, 0u};
    const unsigned char* c = q.codes + p.row * q.ldcodes + p.col;
    if (p.n == 4) {
        h.w = *reinterpret_cast<const unsigned*>(c);
    } else {
        if (p.n > 0) h.w = c[0];
        if (p.n > 1) h.w |= static_cast<unsigned>(c[1]) << 8;
        if (p.n > 2) h.w |= static_cast<unsigned>(c[2]) << 16;
    }
    if (p.n > 0) h.e = q.scales[p.row * q.ldscales + p.block];
    return h;
}
template <int FMT>
__device__ __forceinline__ float4 values(const Held& h) {
    const float4 v = q8_decode4<FMT>(h.w);
    const float s = q8_scale<FMT>(h.e);
    return make_float4(v.x * s, v.y * s, v.z * s, v.w * s);
}

// Each kernel: U segments' loads first, then their arithmetic and stores.
// Lanes without columns load zeros, take part in the shuffles and store
// nothing.
#define Q8_WALK                                                         \
    const int lane = threadIdx.x & 31;                                  \
    for (Walk walk(cols); walk.row < rows;)
#define Q8_PLACES(U)                                                    \
    Place p[U];                                                         \
    _Pragma("unroll") for (int i = 0; i < U; ++i) {                     \
        p[i] = place(walk, rows, cols, lane);                           \
        walk.next();                                                    \
    }

template <int FMT, int U>
__global__ void __launch_bounds__(kThreads)
q8_store_kernel(const float* x, long long ldx, bool vec, int rows, int cols, Q8Out q) {
    Q8_WALK {
        Q8_PLACES(U)
        float4 v[U];
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] = load4(x, ldx, vec, p[i]);
#pragma unroll
        for (int i = 0; i < U; ++i) encode4<FMT>(v[i], p[i], lane, q);
    }
}

template <int FMT, typename T, int U>
__global__ void __launch_bounds__(kThreads)
q8_restore_kernel(Q8In q, int rows, int cols, T* x, long long ldx, bool vec) {
    Q8_WALK {
        Q8_PLACES(U)
        Held h[U];
#pragma unroll
        for (int i = 0; i < U; ++i) h[i] = load_held(q, p[i]);
#pragma unroll
        for (int i = 0; i < U; ++i) put4(x, ldx, vec, p[i], values<FMT>(h[i]));
    }
}

// vec: bit 0, 1, 2 for g, u, h
template <int FMT, int ACT, int U>
__global__ void __launch_bounds__(kThreads)
q8_gated_kernel(const float* g, long long ldg, const float* u, long long ldu, int rows, int cols,
                float* h, long long ldh, unsigned vec, Q8Out gq, Q8Out uq) {
    Q8_WALK {
        Q8_PLACES(U)
        float4 a[U], b[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            a[i] = load4(g, ldg, vec & 1u, p[i]);
            b[i] = load4(u, ldu, vec & 2u, p[i]);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            put4(h, ldh, vec & 4u, p[i],
                 make_float4(act_value<ACT>(a[i].x) * b[i].x, act_value<ACT>(a[i].y) * b[i].y,
                             act_value<ACT>(a[i].z) * b[i].z, act_value<ACT>(a[i].w) * b[i].w));
            encode4<FMT>(a[i], p[i], lane, gq);
            encode4<FMT>(b[i], p[i], lane, uq);
        }
    }
}

// vec: bit 0, 1, 2 for dh, dg, du
template <int FMT, int ACT, int U>
__global__ void __launch_bounds__(kThreads)
q8_gated_backward_kernel(Q8In gq, Q8In uq, const float* dh, long long lddh, int rows, int cols,
                         float* dg, long long lddg, float* du, long long lddu, unsigned vec,
                         Q8Out hq) {
    Q8_WALK {
        Q8_PLACES(U)
        Held a[U], b[U];
        float4 d[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            a[i] = load_held(gq, p[i]);
            b[i] = load_held(uq, p[i]);
            d[i] = load4(dh, lddh, vec & 1u, p[i]);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const float4 gv = values<FMT>(a[i]), uv = values<FMT>(b[i]);
            float4 v, s;
            act_both<ACT>(gv.x, &v.x, &s.x);
            act_both<ACT>(gv.y, &v.y, &s.y);
            act_both<ACT>(gv.z, &v.z, &s.z);
            act_both<ACT>(gv.w, &v.w, &s.w);
            put4(dg, lddg, vec & 2u, p[i],
                 make_float4(d[i].x * uv.x * s.x, d[i].y * uv.y * s.y, d[i].z * uv.z * s.z,
                             d[i].w * uv.w * s.w));
            put4(du, lddu, vec & 4u, p[i],
                 make_float4(d[i].x * v.x, d[i].y * v.y, d[i].z * v.z, d[i].w * v.w));
            if (hq.codes) {
                // beyond the row's end the codes read as zero, and so does this
                encode4<FMT>(make_float4(v.x * uv.x, v.y * uv.y, v.z * uv.z, v.w * uv.w), p[i],
                             lane, hq);
            }
        }
    }
}

// Blocks of 8 warps: one segment a warp, up to 8 blocks an SM and as many
// rounds as it takes.
unsigned grid_for(int rows, int cols) {
    const long long items = static_cast<long long>(rows) * ((cols - 1) / kSegment + 1);
    const long long blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
    return static_cast<unsigned>(blocks < 152 * 8 ? blocks : 152 * 8);
}

// Whether four columns of a matrix can be moved at once.
bool vectors(const void* p, long long ld, int rows, int elem) {
    return reinterpret_cast<uintptr_t>(p) % (4 * elem) == 0 && (ld % 4 == 0 || rows == 1);
}

template <int FMT, typename T>
void restore(const Q8In& q, int rows, int cols, void* x, long long ldx, cudaStream_t s) {
    q8_restore_kernel<FMT, T, 4><<<grid_for(rows, cols), kThreads, 0, s>>>(
        q, rows, cols, static_cast<T*>(x), ldx, vectors(x, ldx, rows, sizeof(T)));
}
template <int FMT, int ACT>
void gated(const GatedArgs& a, cudaStream_t s) {
    const unsigned vec = (vectors(a.g, a.ldg, a.rows, 4) ? 1u : 0u) |
                         (vectors(a.u, a.ldu, a.rows, 4) ? 2u : 0u) |
                         (vectors(a.h, a.ldh, a.rows, 4) ? 4u : 0u);
    q8_gated_kernel<FMT, ACT, 2><<<grid_for(a.rows, a.cols), kThreads, 0, s>>>(
        a.g, a.ldg, a.u, a.ldu, a.rows, a.cols, a.h, a.ldh, vec, a.gq, a.uq);
}
template <int FMT, int ACT>
void gated_backward(const GatedBackwardArgs& a, cudaStream_t s) {
    const unsigned vec = (vectors(a.dh, a.lddh, a.rows, 4) ? 1u : 0u) |
                         (vectors(a.dg, a.lddg, a.rows, 4) ? 2u : 0u) |
                         (vectors(a.du, a.lddu, a.rows, 4) ? 4u : 0u);
    q8_gated_backward_kernel<FMT, ACT, 2><<<grid_for(a.rows, a.cols), kThreads, 0, s>>>(
        a.gq, a.uq, a.dh, a.lddh, a.rows, a.cols, a.dg, a.lddg, a.du, a.lddu, vec, a.hq);
}

}  // namespace

cudaError_t launch_q8_store(const float* x, long long ldx, int rows, int cols, int format,
                            const Q8Out& q, cudaStream_t s) {
    const unsigned grid = grid_for(rows, cols);
    const bool vec = vectors(x, ldx, rows, 4);
    if (format == kQ8Int8)
        q8_store_kernel<kQ8Int8, 2><<<grid, kThreads, 0, s>>>(x, ldx, vec, rows, cols, q);
    else
        q8_store_kernel<kQ8E4m3, 2><<<grid, kThreads, 0, s>>>(x, ldx, vec, rows, cols, q);
    return cudaGetLastError();
}

cudaError_t launch_q8_restore(const Q8In& q, int rows, int cols, int format, void* x,
                              long long ldx, int bf16, cudaStream_t s) {
    if (format == kQ8Int8)
        bf16 ? restore<kQ8Int8, __nv_bfloat16>(q, rows, cols, x, ldx, s)
             : restore<kQ8Int8, float>(q, rows, cols, x, ldx, s);
    else
        bf16 ? restore<kQ8E4m3, __nv_bfloat16>(q, rows, cols, x, ldx, s)
             : restore<kQ8E4m3, float>(q, rows, cols, x, ldx, s);
    return cudaGetLastError();
}

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
