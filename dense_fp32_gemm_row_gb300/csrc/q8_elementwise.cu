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
// A warp takes a segment of 256 columns of one row, a lane eight of them: 32
// bytes of each matrix and eight codes at a time, so that every access of the
// warp is one contiguous run (1024 and 256 bytes), and the 4 lanes of a block
// share its largest magnitude in two shuffles.  (Four columns a lane spent
// some 21 instructions an element, mostly on places and exponents, and the
// instruction rate then bounds the store; a column a lane took three times
// as long.)
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

// The normal distribution function below zero, P(-a) = e^(-a^2/2) F(a), with
// F(a) = erfc(a / sqrt 2) e^(a^2/2) / 2 as a polynomial in t = 1 / (1 + 0.35 a)
// without constant term (the form of Hastings, "Approximations for Digital
// Computers", 1955).  The ten coefficients are a weighted least-squares fit
// made for 0 <= a <= 14.5, refined towards equal relative errors: at most
// 5.1e-8 with these coefficients, 3.3e-7 evaluated in fp32.  P(-a) itself has
// that error and the one of the rounded a^2 / 2, which the exponential makes a
// relative error of its own size: measured on gelu, at most 4.5e-7 for a < 2,
// 5.6e-7 to 4, 1.3e-6 to 8, and 4.2e-6 to 13, where P is below 1e-15.  The
// derivative of gelu needs the same exponential.  (erfcf and expf instead:
// 8192 x 8192 forward 164 us, backward 193, bound by instructions.)
__device__ __forceinline__ void normal(float z, float* p, float* bell) {
    const float a = fabsf(z);
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.35f, a, 1.0f)));
    const float e = expf(-0.5f * a * a);
    float f = 0.0030903539154678583f;
    f = fmaf(f, t, -0.04539582133293152f);
    f = fmaf(f, t, 0.18077702820301056f);
    f = fmaf(f, t, -0.3026995360851288f);
    f = fmaf(f, t, 0.19630774855613708f);
    f = fmaf(f, t, -0.04188587889075279f);
    f = fmaf(f, t, 0.11156046390533447f);
    f = fmaf(f, t, 0.1186375617980957f);
    f = fmaf(f, t, 0.13999271392822266f);
    f = fmaf(f, t, 0.13961537182331085f);
    const float below = f * t * e;
    *p = z < 0.0f ? below : 1.0f - below;
    *bell = e;
}

// act(z) and act'(z) in fp32.
template <int ACT>
__device__ __forceinline__ void act_both(float z, float* value, float* slope) {
    if (ACT == kActSilu) {
        const float s = 1.0f / (1.0f + expf(-z));
        *value = z * s;
        *slope = s * fmaf(z, 1.0f - s, 1.0f);
    } else {
        float p, bell;
        normal(z, &p, &bell);
        *value = z * p;
        *slope = fmaf(z * bell, 0.39894228040143268f, p);
    }
}
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    float value, slope;
    act_both<ACT>(z, &value, &slope);
    return value;
}

constexpr int kBlocksPerSm = 64;
constexpr int kLane = 8;                  // columns of a lane
constexpr int kSegment = 32 * kLane;      // of a warp
constexpr int kShare = kQ8Block / kLane;  // lanes of a block

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

// One lane's place in a segment: the columns from col (those below cols).
struct Place {
    long long row;
    int first, span;  // the segment's first column and its columns
    int col, n;       // the lane's: 0 .. 8 of them
};
__device__ __forceinline__ Place place(const Walk& w, int cols, int lane) {
    Place p;
    p.row = w.row;
    p.first = w.seg * kSegment;
    p.span = min(kSegment, cols - p.first);
    p.n = max(0, min(kLane, p.span - kLane * lane));
    p.col = p.n ? p.first + kLane * lane : 0;
    return p;
}

// How a matrix is moved: 32 or 16 bytes of a lane's columns at once, or, where
// its rows do not start on 16-byte boundaries, by columns lane, lane + 32, ...
// of the segment, which is contiguous across the warp at any alignment, and
// from or to the lanes' own columns through shared memory.
enum Vec : unsigned { kVecNone = 0, kVec16 = 1, kVec32 = 2 };

struct Lane {
    float v[kLane];
};

// The warp's buffer for that: a lane's eight floats 12 apart from the next
// lane's, so that 16-byte accesses of eight lanes cover all banks.  Each
// kernel also exists without it (ALIGNED: no matrix needs it), with a third
// fewer registers (8192 x 8192: gated forward 137 against 150 us, backward
// 151 against 166).
constexpr int kPitch = 12;
template <bool ALIGNED>
struct Staging {
    float f[kThreads / 32][32 * kPitch];
};
template <>
struct Staging<true> {};

template <bool ALIGNED>
__device__ __forceinline__ Lane load(const float* m, long long ld, unsigned vec, const Place& p) {
    Lane x;
    const float* r = m + p.row * ld;
    if (!ALIGNED && vec == kVecNone) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < kLane; ++i)
            x.v[i] = lane + 32 * i < p.span ? r[p.first + lane + 32 * i] : 0.0f;
    } else if (p.n < kLane) {
#pragma unroll
        for (int i = 0; i < kLane; ++i) x.v[i] = i < p.n ? r[p.col + i] : 0.0f;
    } else if (vec == kVec32) {
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(x.v[0]), "=f"(x.v[1]), "=f"(x.v[2]), "=f"(x.v[3]), "=f"(x.v[4]),
                       "=f"(x.v[5]), "=f"(x.v[6]), "=f"(x.v[7])
                     : "l"(r + p.col));
    } else {
        const float4 lo = reinterpret_cast<const float4*>(r + p.col)[0];
        const float4 hi = reinterpret_cast<const float4*>(r + p.col)[1];
        x.v[0] = lo.x, x.v[1] = lo.y, x.v[2] = lo.z, x.v[3] = lo.w;
        x.v[4] = hi.x, x.v[5] = hi.y, x.v[6] = hi.z, x.v[7] = hi.w;
    }
    return x;
}

// After the loads of all matrices are under way: the lane's own columns.
__device__ __forceinline__ Lane settle(Lane x, unsigned, Staging<true>&) { return x; }
__device__ __forceinline__ Lane settle(Lane x, unsigned vec, Staging<false>& st) {
    if (vec != kVecNone) return x;
    const int lane = threadIdx.x & 31;
    float* f = st.f[threadIdx.x >> 5];
#pragma unroll
    for (int i = 0; i < kLane; ++i) f[kPitch * (4 * i + (lane >> 3)) + (lane & 7)] = x.v[i];
    __syncwarp();
    const float4 lo = *reinterpret_cast<const float4*>(f + kPitch * lane);
    const float4 hi = *reinterpret_cast<const float4*>(f + kPitch * lane + 4);
    __syncwarp();
    return {{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
}

// The warp's columns as the striped stores take them: of the lane's columns x,
// value i is that of column lane + 32 i.
__device__ __forceinline__ Lane stripe(const Lane& x, Staging<true>&) { return x; }
__device__ __forceinline__ Lane stripe(const Lane& x, Staging<false>& st) {
    const int lane = threadIdx.x & 31;
    float* f = st.f[threadIdx.x >> 5];
    *reinterpret_cast<float4*>(f + kPitch * lane) = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
    *reinterpret_cast<float4*>(f + kPitch * lane + 4) = make_float4(x.v[4], x.v[5], x.v[6], x.v[7]);
    __syncwarp();
    Lane y;
#pragma unroll
    for (int i = 0; i < kLane; ++i) y.v[i] = f[kPitch * (4 * i + (lane >> 3)) + (lane & 7)];
    __syncwarp();
    return y;
}

template <bool ALIGNED>
__device__ __forceinline__ void put(float* m, long long ld, unsigned vec, const Place& p,
                                    const Lane& x, Staging<ALIGNED>& st) {
    float* r = m + p.row * ld;
    if (!ALIGNED && vec == kVecNone) {
        const int lane = threadIdx.x & 31;
        const Lane y = stripe(x, st);
#pragma unroll
        for (int i = 0; i < kLane; ++i)
            if (lane + 32 * i < p.span) r[p.first + lane + 32 * i] = y.v[i];
    } else if (p.n < kLane) {
#pragma unroll
        for (int i = 0; i < kLane; ++i)
            if (i < p.n) r[p.col + i] = x.v[i];
    } else if (vec == kVec32) {
        asm volatile("st.global.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(x.v[0]),
                     "f"(x.v[1]), "f"(x.v[2]), "f"(x.v[3]), "f"(x.v[4]), "f"(x.v[5]), "f"(x.v[6]),
                     "f"(x.v[7]), "l"(r + p.col)
                     : "memory");
    } else {
        reinterpret_cast<float4*>(r + p.col)[0] = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
        reinterpret_cast<float4*>(r + p.col)[1] = make_float4(x.v[4], x.v[5], x.v[6], x.v[7]);
    }
}
// bf16, rounding nothing: the values of a checkpoint are exact in it
template <bool ALIGNED>
__device__ __forceinline__ void put(__nv_bfloat16* m, long long ld, unsigned vec, const Place& p,
                                    const Lane& x, Staging<ALIGNED>& st) {
    unsigned short* r = reinterpret_cast<unsigned short*>(m) + p.row * ld;
    if (!ALIGNED && vec == kVecNone) {
        const int lane = threadIdx.x & 31;
        const Lane y = stripe(x, st);
#pragma unroll
        for (int i = 0; i < kLane; ++i)
            if (lane + 32 * i < p.span)
                r[p.first + lane + 32 * i] = static_cast<unsigned short>(__float_as_uint(y.v[i]) >> 16);
    } else if (p.n < kLane) {
#pragma unroll
        for (int i = 0; i < kLane; ++i)
            if (i < p.n) r[p.col + i] = static_cast<unsigned short>(__float_as_uint(x.v[i]) >> 16);
    } else {
        unsigned w[kLane / 2];
#pragma unroll
        for (int i = 0; i < kLane / 2; ++i)
            w[i] = __byte_perm(__float_as_uint(x.v[2 * i]), __float_as_uint(x.v[2 * i + 1]), 0x7632);
        *reinterpret_cast<uint4*>(r + p.col) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Encode a lane's values (zeros beyond the row) with its block's lanes and
// write codes and exponent.
template <int FMT>
__device__ __forceinline__ void encode(const Lane& x, const Place& p, int lane, const Q8Out& q) {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < kLane; ++i) m = max(m, q8_magnitude(x.v[i]));
#pragma unroll
    for (int d = 1; d < kShare; d *= 2) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    const unsigned e = q8_exponent<FMT>(m);
    const float inv = q8_inverse_scale<FMT>(e);
    const unsigned w0 = q8_encode4<FMT>(x.v[0], x.v[1], x.v[2], x.v[3], inv, e);
    const unsigned w1 = q8_encode4<FMT>(x.v[4], x.v[5], x.v[6], x.v[7], inv, e);
    unsigned char* c = q.codes + p.row * q.ldcodes + p.col;
    if (p.n == kLane) {
        *reinterpret_cast<uint2*>(c) = make_uint2(w0, w1);
    } else {
#pragma unroll
        for (int i = 0; i < kLane - 1; ++i)
            if (i < p.n) c[i] = static_cast<unsigned char>((i < 4 ? w0 : w1) >> (8 * (i & 3)));
    }
    if (lane % kShare == 0 && p.n > 0)
        q.scales[p.row * q.ldscales + p.col / kQ8Block] = static_cast<unsigned char>(e);
}

// A lane's codes (bytes beyond the row are the caller's and not used) and
// exponent byte.
struct Held {
    unsigned w0, w1, e;
};
__device__ __forceinline__ Held load_held(const Q8In& q, const Place& p) {
    Held h = {0u, 0u, 0u};
    const unsigned char* c = q.codes + p.row * q.ldcodes + p.col;
    if (p.n == kLane) {
        const uint2 w = *reinterpret_cast<const uint2*>(c);
        h.w0 = w.x;
        h.w1 = w.y;
    } else {
#pragma unroll
        for (int i = 0; i < kLane - 1; ++i) {
            const unsigned b = i < p.n ? static_cast<unsigned>(c[i]) << (8 * (i & 3)) : 0u;
            if (i < 4)
                h.w0 |= b;
            else
                h.w1 |= b;
        }
    }
    if (p.n > 0) h.e = q.scales[p.row * q.ldscales + p.col / kQ8Block];
    return h;
}
template <int FMT>
__device__ __forceinline__ Lane values(const Held& h) {
    const float4 lo = q8_decode4<FMT>(h.w0), hi = q8_decode4<FMT>(h.w1);
    const float s = q8_scale<FMT>(h.e);
    return {{lo.x * s, lo.y * s, lo.z * s, lo.w * s, hi.x * s, hi.y * s, hi.z * s, hi.w * s}};
}

// A warp's segments in turn, `p` its lane's place.  Lanes without columns load
// zeros, take part in the shuffles and store nothing.  One segment at a time:
// 64 blocks an SM's worth of short warps keep the memory busier than two or
// four segments in flight in each (8192 x 8192: store 51.5 against 55.6 us,
// gated forward 137.6 against 164.3).
#define Q8_FOR_EACH_PLACE(p)                                                       \
    const int lane = threadIdx.x & 31;                                             \
    pdl_wait();                                                                    \
    pdl_trigger();                                                                 \
    for (Walk walk(cols); walk.row < rows; walk.next())                            \
        if (const Place p = place(walk, cols, lane); true)

template <int FMT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads)
q8_store_kernel(const float* x, long long ldx, unsigned vec, int rows, int cols, Q8Out q) {
    __shared__ Staging<ALIGNED> st;
    Q8_FOR_EACH_PLACE(p) { encode<FMT>(settle(load<ALIGNED>(x, ldx, vec, p), vec, st), p, lane, q); }
}

template <int FMT, typename T, bool ALIGNED>
__global__ void __launch_bounds__(kThreads)
q8_restore_kernel(Q8In q, int rows, int cols, T* x, long long ldx, unsigned vec) {
    __shared__ Staging<ALIGNED> st;
    Q8_FOR_EACH_PLACE(p) { put<ALIGNED>(x, ldx, vec, p, values<FMT>(load_held(q, p)), st); }
}

template <int FMT, int ACT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads)
q8_gated_kernel(const float* g, long long ldg, unsigned vec_g, const float* u, long long ldu,
                unsigned vec_u, int rows, int cols, float* h, long long ldh, unsigned vec_h,
                Q8Out gq, Q8Out uq) {
    __shared__ Staging<ALIGNED> st;
    Q8_FOR_EACH_PLACE(p) {
        const Lane a0 = load<ALIGNED>(g, ldg, vec_g, p), b0 = load<ALIGNED>(u, ldu, vec_u, p);
        const Lane a = settle(a0, vec_g, st), b = settle(b0, vec_u, st);
        Lane y;
#pragma unroll
        for (int j = 0; j < kLane; ++j) y.v[j] = act_value<ACT>(a.v[j]) * b.v[j];
        put<ALIGNED>(h, ldh, vec_h, p, y, st);
        encode<FMT>(a, p, lane, gq);
        encode<FMT>(b, p, lane, uq);
    }
}

template <int FMT, int ACT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads)
q8_gated_backward_kernel(Q8In gq, Q8In uq, const float* dh, long long lddh, unsigned vec_dh,
                         int rows, int cols, float* dg, long long lddg, unsigned vec_dg,
                         float* du, long long lddu, unsigned vec_du, Q8Out hq) {
    __shared__ Staging<ALIGNED> st;
    Q8_FOR_EACH_PLACE(p) {
        const Held hg = load_held(gq, p), hu = load_held(uq, p);
        const Lane d = settle(load<ALIGNED>(dh, lddh, vec_dh, p), vec_dh, st);
        const Lane gv = values<FMT>(hg), uv = values<FMT>(hu);
        Lane y, z, h;
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            float value, slope;
            act_both<ACT>(gv.v[j], &value, &slope);
            y.v[j] = d.v[j] * uv.v[j] * slope;
            z.v[j] = d.v[j] * value;
            h.v[j] = value * uv.v[j];  // zero beyond the row's end, as the codes are read
        }
        put<ALIGNED>(dg, lddg, vec_dg, p, y, st);
        put<ALIGNED>(du, lddu, vec_du, p, z, st);
        if (hq.codes) encode<FMT>(h, p, lane, hq);
    }
}

// Blocks of 8 warps, a segment a warp, up to kBlocksPerSm blocks an SM and as
// many rounds as it takes (8192 x 8192: 64 an SM 51.5, 54.0, 137.6 and 162.3
// us for store, restore, gated forward and backward; 8 an SM 53.2, 61.7, 155.1
// and 161.5; 256 an SM 53.7, 73.9, 143.5 and 172.0).
unsigned grid_for(int rows, int cols, int sm_count) {
    const long long items = static_cast<long long>(rows) * ((cols - 1) / kSegment + 1);
    const long long blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
    const long long most = static_cast<long long>(sm_count) * kBlocksPerSm;
    return static_cast<unsigned>(blocks < most ? blocks : most);
}

unsigned vectors(const void* p, long long ld, int rows) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p) | (rows > 1 ? 4 * ld : 0);
    return a % 32 == 0 ? kVec32 : a % 16 == 0 ? kVec16 : kVecNone;
}
unsigned vectors_bf16(const void* p, long long ld, int rows) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p) | (rows > 1 ? 2 * ld : 0);
    return a % 16 == 0 ? kVec16 : kVecNone;
}

// Launched as programmatic dependents: a kernel's launch overlaps the end of
// the one before it, whose outputs it waits for.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int rows, int cols, const Q8Launch& on, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.gridDim = dim3(grid_for(rows, cols, on.sm_count));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = on.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int FMT, typename T>
cudaError_t restore(const Q8In& q, int rows, int cols, void* x, long long ldx, unsigned vec,
                    const Q8Launch& on) {
    return launch(vec ? q8_restore_kernel<FMT, T, true> : q8_restore_kernel<FMT, T, false>, rows,
                  cols, on, q, rows, cols, static_cast<T*>(x), ldx, vec);
}
template <int FMT>
cudaError_t store(const float* x, long long ldx, int rows, int cols, const Q8Out& q,
                  const Q8Launch& on) {
    const unsigned vec = vectors(x, ldx, rows);
    return launch(vec ? q8_store_kernel<FMT, true> : q8_store_kernel<FMT, false>, rows, cols, on, x,
                  ldx, vec, rows, cols, q);
}
template <int FMT, int ACT>
cudaError_t gated(const GatedArgs& a, const Q8Launch& on) {
    const unsigned vg = vectors(a.g, a.ldg, a.rows), vu = vectors(a.u, a.ldu, a.rows),
                   vh = vectors(a.h, a.ldh, a.rows);
    return launch(
        vg && vu && vh ? q8_gated_kernel<FMT, ACT, true> : q8_gated_kernel<FMT, ACT, false>, a.rows,
        a.cols, on, a.g, a.ldg, vg, a.u, a.ldu, vu, a.rows, a.cols, a.h, a.ldh, vh, a.gq, a.uq);
}
template <int FMT, int ACT>
cudaError_t gated_backward(const GatedBackwardArgs& a, const Q8Launch& on) {
    const unsigned vd = vectors(a.dh, a.lddh, a.rows), vg = vectors(a.dg, a.lddg, a.rows),
                   vu = vectors(a.du, a.lddu, a.rows);
    return launch(vd && vg && vu ? q8_gated_backward_kernel<FMT, ACT, true>
                                 : q8_gated_backward_kernel<FMT, ACT, false>,
                  a.rows, a.cols, on, a.gq, a.uq, a.dh, a.lddh, vd, a.rows, a.cols, a.dg, a.lddg,
                  vg, a.du, a.lddu, vu, a.hq);
}

}  // namespace

cudaError_t launch_q8_store(const float* x, long long ldx, int rows, int cols, int format,
                            const Q8Out& q, const Q8Launch& on) {
    return format == kQ8Int8 ? store<kQ8Int8>(x, ldx, rows, cols, q, on)
                             : store<kQ8E4m3>(x, ldx, rows, cols, q, on);
}

cudaError_t launch_q8_restore(const Q8In& q, int rows, int cols, int format, void* x,
                              long long ldx, int bf16, const Q8Launch& on) {
    const unsigned vec = bf16 ? vectors_bf16(x, ldx, rows) : vectors(x, ldx, rows);
    if (format == kQ8Int8)
        return bf16 ? restore<kQ8Int8, __nv_bfloat16>(q, rows, cols, x, ldx, vec, on)
                    : restore<kQ8Int8, float>(q, rows, cols, x, ldx, vec, on);
    return bf16 ? restore<kQ8E4m3, __nv_bfloat16>(q, rows, cols, x, ldx, vec, on)
                : restore<kQ8E4m3, float>(q, rows, cols, x, ldx, vec, on);
}

cudaError_t launch_q8_gated(const GatedArgs& a, const Q8Launch& on) {
    if (a.format == kQ8Int8)
        return a.act == kActSilu ? gated<kQ8Int8, kActSilu>(a, on) : gated<kQ8Int8, kActGelu>(a, on);
    return a.act == kActSilu ? gated<kQ8E4m3, kActSilu>(a, on) : gated<kQ8E4m3, kActGelu>(a, on);
}

cudaError_t launch_q8_gated_backward(const GatedBackwardArgs& a, const Q8Launch& on) {
    if (a.format == kQ8Int8)
        return a.act == kActSilu ? gated_backward<kQ8Int8, kActSilu>(a, on)
                                 : gated_backward<kQ8Int8, kActGelu>(a, on);
    return a.act == kActSilu ? gated_backward<kQ8E4m3, kActSilu>(a, on)
                             : gated_backward<kQ8E4m3, kActGelu>(a, on);
}

}  // namespace gemm_f32_impl
