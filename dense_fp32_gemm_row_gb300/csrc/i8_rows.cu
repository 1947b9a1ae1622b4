// i8_rows.cu -- rows to 8-bit integers with one scale a row: as they are, or
// as their root-mean-square norm after the residual's addition.
//
//   store  z = x
//   norm   s = x + r;  z = s w;  rho = 1 / sqrt(mean s^2 + eps)
//   a = max(max |z|, 2^-100);  code = rint(z (127 / a));  scale = (a / 127) [rho]
//
// The norm's factor is one number a row, so it cancels in the codes: the
// maximum and the sum of squares come from one pass over the row, and the codes
// need nothing but the maximum.  Each operation above is rounded to fp32, so
// codes do not depend on the order in which a row is summed.  A row in which z
// is not finite gets codes 0 and scale NaN.
//
// Bounded by HBM: a row is read once, held in registers (up to 32 columns a
// thread) between the two steps, and written once.  Rows beyond 16384 columns are
// read a second time, from L2.  8192 x 8192, of the measured copy rate: store
// float32 47 us, 105 %, bf16 30.5, 97 %; norm with residual float32 122, 105 %,
// bf16 75.3, 92 %.  Rows off 16-byte boundaries: norm 8191 x 8191 float32 128 us,
// 100 %, bf16, two bytes at a time, 95, 73 %, store 40, 75 %.
#include <cstdint>

#include <cuda_bf16.h>

#include "device_sync.cuh"
#include "gemm_internal.h"

namespace gemm_f32_impl {
namespace {

using namespace gemm_f32_dev;

constexpr int kLane = 8;   // consecutive columns of a thread: 8 bytes of codes
constexpr unsigned kInfinity = 0x7F800000u;
constexpr float kLeast = 7.888609052210118e-31f;  // 2^-100

enum Mode { kStore, kNorm, kNormResidual };

struct Group {
    float v[kLane];
};

// Columns of a thread: kLane consecutive ones from col, all or none of them in the
// row (VEC), or, where rows do not start on 16-byte boundaries or are no multiple
// of kLane, every stride-th from col.  No load is behind a branch, so that all
// are under way at once (a test of each vector's columns: 8192 x 8192 bf16 157
// us).
struct Columns {
    int col, n, stride;  // n of kLane are in the row
};
template <bool VEC>
__device__ __forceinline__ Columns columns(int group, int thread, int threads, int cols) {
    Columns c;
    if (VEC) {
        c.col = (group * threads + thread) * kLane;
        c.stride = 1;
        c.n = c.col < cols ? kLane : 0;
    } else {
        c.col = group * threads * kLane + thread;
        c.stride = threads;
        c.n = c.col < cols ? min(kLane, (cols - 1 - c.col) / threads + 1) : 0;
    }
    return c;
}

// An element if it is there, or 0, without a branch.  (Written in C++ a bf16 load
// waited for the one before: norm 8191 x 8191 167 us, like this 95; store 62 and
// 40.)  The asm keeps its place behind the wait for the kernel before, but not
// among this one's stores, which never go to an operand.
__device__ __forceinline__ float load_if(const float* p, bool there) {
    float v;
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t"
        "@q ld.global.f32 %0, [%1];\n\t}"
        : "=f"(v)
        : "l"(p), "r"(static_cast<int>(there)));
    return v;
}
__device__ __forceinline__ float load_if(const __nv_bfloat16* p, bool there) {
    unsigned short v;
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %2, 0;\n\tmov.u16 %0, 0;\n\t"
        "@q ld.global.u16 %0, [%1];\n\t}"
        : "=h"(v)
        : "l"(p), "r"(static_cast<int>(there)));
    return __uint_as_float(static_cast<unsigned>(v) << 16);
}

template <bool VEC>
__device__ __forceinline__ Group load(const float* p, const Columns& c) {
    Group g;
    if (VEC) {
        float4 lo = make_float4(0.0f, 0.0f, 0.0f, 0.0f), hi = lo;
        if (c.n) {
            lo = reinterpret_cast<const float4*>(p + c.col)[0];
            hi = reinterpret_cast<const float4*>(p + c.col)[1];
        }
        g.v[0] = lo.x, g.v[1] = lo.y, g.v[2] = lo.z, g.v[3] = lo.w;
        g.v[4] = hi.x, g.v[5] = hi.y, g.v[6] = hi.z, g.v[7] = hi.w;
    } else {
#pragma unroll
        for (int i = 0; i < kLane; ++i) g.v[i] = load_if(p + c.col + i * c.stride, i < c.n);
    }
    return g;
}
template <bool VEC>
__device__ __forceinline__ Group load(const __nv_bfloat16* p, const Columns& c) {
    Group g;
    if (VEC) {
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (c.n) w = *reinterpret_cast<const uint4*>(p + c.col);
        const unsigned u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            g.v[2 * i] = __uint_as_float(u[i] << 16);
            g.v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kLane; ++i) g.v[i] = load_if(p + c.col + i * c.stride, i < c.n);
    }
    return g;
}
template <bool VEC>
__device__ __forceinline__ void put(float* p, const Columns& c, const Group& g) {
    if (VEC) {
        if (!c.n) return;
        reinterpret_cast<float4*>(p + c.col)[0] = make_float4(g.v[0], g.v[1], g.v[2], g.v[3]);
        reinterpret_cast<float4*>(p + c.col)[1] = make_float4(g.v[4], g.v[5], g.v[6], g.v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < kLane; ++i)
            if (i < c.n) p[c.col + i * c.stride] = g.v[i];
    }
}
template <bool VEC>
__device__ __forceinline__ void put(__nv_bfloat16* p, const Columns& c, const Group& g) {
    if (VEC) {
        unsigned u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(g.v[2 * i], g.v[2 * i + 1]);
            u[i] = *reinterpret_cast<const unsigned*>(&two);
        }
        if (c.n) *reinterpret_cast<uint4*>(p + c.col) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kLane; ++i)
            if (i < c.n) p[c.col + i * c.stride] = __float2bfloat16_rn(g.v[i]);
    }
}

// Codes of a group.  Adding 1.5 * 2^23 leaves the integer nearest to the
// product (ties to even) in the low bits of the sum; the product is rounded
// first, as the definition has it.
template <bool VEC>
__device__ __forceinline__ void put_codes(signed char* p, const Columns& c, const Group& z,
                                          float inv, bool finite) {
    unsigned q[kLane];
#pragma unroll
    for (int i = 0; i < kLane; ++i)
        q[i] = finite ? __float_as_uint(__fadd_rn(__fmul_rn(z.v[i], inv), 12582912.0f)) : 0u;
    if (VEC) {
        uint2 w;
        w.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
        w.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
        if (c.n) *reinterpret_cast<uint2*>(p + c.col) = w;
    } else {
#pragma unroll
        for (int i = 0; i < kLane; ++i)
            if (i < c.n) p[c.col + i * c.stride] = static_cast<signed char>(q[i]);
    }
}

// One group of a row: s, and z = s w.
template <typename T, Mode MODE, bool VEC>
__device__ __forceinline__ Group sum_of(const I8RowsArgs& a, long long row, const Columns& c) {
    Group s = load<VEC>(static_cast<const T*>(a.x) + row * a.ldx, c);
    if (MODE == kNormResidual) {
        const Group r = load<VEC>(static_cast<const T*>(a.r) + row * a.ldr, c);
#pragma unroll
        for (int i = 0; i < kLane; ++i) s.v[i] = __fadd_rn(s.v[i], r.v[i]);
    }
    return s;
}
template <typename T, Mode MODE, bool VEC>
__device__ __forceinline__ Group weighted(const I8RowsArgs& a, const Columns& c, const Group& s) {
    if (MODE == kStore) return s;
    Group z = load<VEC>(static_cast<const T*>(a.w), c);
#pragma unroll
    for (int i = 0; i < kLane; ++i) z.v[i] = __fmul_rn(s.v[i], z.v[i]);
    return z;
}
template <typename T, bool VEC>
__device__ __forceinline__ void put_sum(const I8RowsArgs& a, long long row, const Columns& c,
                                        const Group& s) {
    if (a.s) put<VEC>(static_cast<T*>(a.s) + row * a.lds, c, s);
}

__device__ __forceinline__ unsigned top_of(const Group& z, unsigned top) {
#pragma unroll
    for (int i = 0; i < kLane; ++i) top = max(top, __float_as_uint(z.v[i]) & 0x7FFFFFFFu);
    return top;
}
__device__ __forceinline__ float squares_of(const Group& s, float scale, float sum) {
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
        const float v = s.v[i] * scale;
        sum = fmaf(v, v, sum);
    }
    return sum;
}

// Sum and maximum over the G threads of a row, in all of them.  The buffers
// alternate between calls, so that one barrier a call is enough.
template <int G>
struct Across {
    float* sums;
    unsigned* tops;
    __device__ __forceinline__ void operator()(float& sum, unsigned& top) const {
        top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (G == 32) return;
        constexpr int kWarps = G / 32;
        if ((threadIdx.x & 31) == 0) {
            sums[threadIdx.x >> 5] = sum;
            tops[threadIdx.x >> 5] = top;
        }
        __syncthreads();
        sum = 0.0f;
        top = 0u;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            sum += sums[i];
            top = max(top, tops[i]);
        }
    }
};

// G threads a row (a block of 256 takes eight rows where G is a warp), which hold
// E groups of columns each, or (E = 0) read the row twice.
template <typename T, Mode MODE, bool VEC, int G, int E>
__global__ void __launch_bounds__(G == 32 ? 256 : G) i8_rows_kernel(I8RowsArgs a) {
    __shared__ float sums[2][G / 32];
    __shared__ unsigned tops[2][G / 32];
    constexpr bool HELD = E > 0;
    constexpr int kHeld = HELD ? E : 1;
    const int thread = static_cast<int>(threadIdx.x) % G;
    const long long row = G == 32 ? blockIdx.x * 8LL + (threadIdx.x >> 5) : blockIdx.x;
    pdl_wait();
    pdl_trigger();
    if (G == 32 && row >= a.rows) return;
    const int groups = HELD ? kHeld : (a.cols - 1) / (G * kLane) + 1;
    Group held[kHeld];
    float sum = 0.0f;
    unsigned top = 0u;
    if (HELD) {
        // every load before the first store, which might be to where they read
        Group s[kHeld];
#pragma unroll
        for (int e = 0; e < kHeld; ++e)
            s[e] = sum_of<T, MODE, VEC>(a, row, columns<VEC>(e, thread, G, a.cols));
#pragma unroll
        for (int e = 0; e < kHeld; ++e)
            held[HELD ? e : 0] = weighted<T, MODE, VEC>(a, columns<VEC>(e, thread, G, a.cols), s[e]);
#pragma unroll
        for (int e = 0; e < kHeld; ++e) {
            if (MODE == kNormResidual)
                put_sum<T, VEC>(a, row, columns<VEC>(e, thread, G, a.cols), s[e]);
            top = top_of(held[HELD ? e : 0], top);
            if (MODE != kStore) sum = squares_of(s[e], 1.0f, sum);
        }
    } else {
        for (int e = 0; e < groups; ++e) {
            const Columns c = columns<VEC>(e, thread, G, a.cols);
            const Group s = sum_of<T, MODE, VEC>(a, row, c);
            top = top_of(weighted<T, MODE, VEC>(a, c, s), top);
            if (MODE == kNormResidual) put_sum<T, VEC>(a, row, c, s);
            if (MODE != kStore) sum = squares_of(s, 1.0f, sum);
        }
    }
    Across<G>{sums[0], tops[0]}(sum, top);
    const bool finite = top < kInfinity;
    float shrink = 1.0f;
    if (MODE != kStore && finite && __float_as_uint(__fadd_rn(sum, a.eps)) >= kInfinity) {
        // squares (or they and eps) beyond fp32, of a row that is not: again at 2^-80
        shrink = 8.271806125530277e-25f;
        sum = 0.0f;
        for (int e = 0; e < groups; ++e) {
            sum = squares_of(sum_of<T, MODE, VEC>(a, row, columns<VEC>(e, thread, G, a.cols)), shrink,
                             sum);
        }
        unsigned none = 0u;
        Across<G>{sums[1], tops[1]}(sum, none);
    }
    const float most = fmaxf(__uint_as_float(finite ? top : 0u), kLeast);
    const float inv = __fdiv_rn(127.0f, most);
    signed char* codes = a.codes + row * a.ldq;
#pragma unroll
    for (int e = 0; e < groups; ++e) {
        const Columns c = columns<VEC>(e, thread, G, a.cols);
        if (HELD)
            put_codes<VEC>(codes, c, held[HELD ? e : 0], inv, finite);
        else
            put_codes<VEC>(codes, c, weighted<T, MODE, VEC>(a, c, sum_of<T, MODE, VEC>(a, row, c)),
                           inv, finite);
    }
    if (thread == 0) {
        float scale = __fdiv_rn(most, 127.0f);
        if (MODE != kStore) {
            const float mean = __fdiv_rn(sum, static_cast<float>(a.cols));
            const float root = __fsqrt_rn(__fadd_rn(mean, a.eps * shrink * shrink));
            scale = __fmul_rn(scale, __fdiv_rn(shrink, root));
        }
        a.scales[row] = finite ? scale : __uint_as_float(0x7FFFFFFFu);
    }
}

template <typename T, Mode MODE, bool VEC, int G, int E>
cudaError_t launch(const I8RowsArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.gridDim = dim3(G == 32 ? (a.rows - 1) / 8 + 1 : a.rows);
    cfg.blockDim = dim3(G == 32 ? 256 : G);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, i8_rows_kernel<T, MODE, VEC, G, E>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Threads a row: for many rows as few as hold it, for too few to fill the GPU as
// many as have eight columns each, or hold the row (a row of 28672 bf16 stored in
// 2.5 us against 3.6; the norm's values are too many for that).  The float32 norm with its residual, which
// has most values under way, takes twice as many (8192 x 8192 122 us against
// 129, 4096 x 1000 10.5 against 14.7; the store of 50000 x 1000 51 against 36),
// but not for long rows off 16-byte boundaries (8191 x 8191 128 against 146).
template <typename T, Mode MODE, bool VEC>
cudaError_t choose(const I8RowsArgs& a, cudaStream_t stream, int sm_count) {
    if (a.rows <= 2 * sm_count) {
        if (a.cols <= 32 * kLane) return launch<T, MODE, VEC, 32, 1>(a, stream);
        if (a.cols <= 128 * kLane) return launch<T, MODE, VEC, 128, 1>(a, stream);
        if (a.cols <= 512 * kLane) return launch<T, MODE, VEC, 512, 1>(a, stream);
        if (a.cols <= 1024 * kLane) return launch<T, MODE, VEC, 1024, 1>(a, stream);
        if constexpr (MODE == kStore)
            if (a.cols > 2048 * kLane && a.cols <= 4096 * kLane)
                return launch<T, MODE, VEC, 1024, 4>(a, stream);
    }
    if constexpr (MODE == kNormResidual && sizeof(T) == 4) {
        if (a.cols > 64 * kLane && a.cols <= 128 * kLane)
            return launch<T, MODE, VEC, 128, 1>(a, stream);
        if (VEC && a.cols > 256 * kLane && a.cols <= 512 * kLane)
            return launch<T, MODE, VEC, 256, 2>(a, stream);
        if (VEC && a.cols > 512 * kLane && a.cols <= 1024 * kLane)
            return launch<T, MODE, VEC, 512, 2>(a, stream);
    }
    if (a.cols <= 32 * kLane) return launch<T, MODE, VEC, 32, 1>(a, stream);
    if (a.cols <= 64 * kLane) return launch<T, MODE, VEC, 32, 2>(a, stream);
    if (a.cols <= 128 * kLane) return launch<T, MODE, VEC, 32, 4>(a, stream);
    if (a.cols <= 256 * kLane) return launch<T, MODE, VEC, 128, 2>(a, stream);
    if (a.cols <= 512 * kLane) return launch<T, MODE, VEC, 128, 4>(a, stream);
    if (a.cols <= 1024 * kLane) return launch<T, MODE, VEC, 256, 4>(a, stream);
    if (a.cols <= 2048 * kLane) return launch<T, MODE, VEC, 512, 4>(a, stream);
    return launch<T, MODE, VEC, 512, 0>(a, stream);
}

// Whether rows can be moved 16 bytes at a time.
bool aligned(const void* p, long long ld, int rows, int elem) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * elem % 16 == 0));
}

template <typename T, Mode MODE>
cudaError_t by_alignment(const I8RowsArgs& a, cudaStream_t stream, int sm_count) {
    const int elem = static_cast<int>(sizeof(T));
    const bool vec = a.cols % kLane == 0 && aligned(a.x, a.ldx, a.rows, elem) && aligned(a.r, a.ldr, a.rows, elem) &&
                     aligned(a.s, a.lds, a.rows, elem) && aligned(a.w, 0, 1, elem);
    return vec ? choose<T, MODE, true>(a, stream, sm_count)
               : choose<T, MODE, false>(a, stream, sm_count);
}

template <typename T>
cudaError_t by_mode(const I8RowsArgs& a, cudaStream_t stream, int sm_count) {
    if (!a.w) return by_alignment<T, kStore>(a, stream, sm_count);
    return a.r ? by_alignment<T, kNormResidual>(a, stream, sm_count)
               : by_alignment<T, kNorm>(a, stream, sm_count);
}

}  // namespace

cudaError_t launch_i8_rows(const I8RowsArgs& a, cudaStream_t stream, int sm_count) {
    return a.bf16 ? by_mode<__nv_bfloat16>(a, stream, sm_count)
                  : by_mode<float>(a, stream, sm_count);
}

}  // namespace gemm_f32_impl
