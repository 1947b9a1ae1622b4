// i8_stream.cu -- the product of 8-bit integer matrices for a few tokens, where
// reading the weights is all there is to do:
//   acc[t][n] = sum_k a[t][k] b[n][k],  y = acc sa[t] sb[n]
// and the gated product of two of them, h = act(g) u.
//
// Codes stay in registers from the load to the warp's own MMAs (A the weights of
// 16 channels, B eight tokens): the weights pass through nothing else, and there
// is no pipeline to fill.  Up to eight tokens take the integer MMA, whose sums are
// exact by themselves.  On this part it runs at half the rate of the fp16 one, to
// which codes have first to be converted, but that leaves it fast enough there
// (8192 x 8192: 8 tokens 13.6 us against 13.9 through fp16, but 16 20.0 against
// 15.3, 24 28.9 against 19.0).  More tokens take the fp16 MMA as the kernel for
// many does (i8_tmem.cu): sums of up to 1024 products are exact in its fp32
// accumulators, and are then added up in 32-bit integers.
//
// A block takes 16 or 32 channels (gated: 16 of both weights) and all of K, its
// warps every W-th 64 columns each.  A lane copies 16 consecutive codes of its
// rows, and four lanes 64, to slots of its own in shared memory, several steps
// ahead, and reads them itself: no warp waits for another before the end, where
// their sums meet.  That the codes' order along K is not that of the MMA's
// fragments makes no difference, as it is the same in both operands.  A copy
// ends with K and leaves zeros behind it.
//
// Bounded by HBM and by a launch's 3 to 4 us: a token through 16384 x 16384 46
// us, 5.8 TB/s, 8192 x 8192 13.1, 4096 x 4096 5.1.  From 17 tokens on by the MMAs:
// 24 x 8192 x 8192 19.1 us, about 3 for each group of eight.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>

#include "device_sync.cuh"
#include "gemm_internal.h"
#include "i8_output.cuh"

namespace gemm_f32_impl {
namespace {

using namespace gemm_f32_dev;

constexpr int kExactSteps = 1024 / 64;  // steps of 64 columns of K
constexpr int kAhead = 4;             // steps of a warp under way
constexpr int kEarlyBytes = 512;      // of a channel, prefetched before the kernel's turn
constexpr int kSharedBytes = 233472;  // shared memory of an SM
constexpr int kBlockBytes = 232448;   // of a block, at most

// To L2; from a 16-byte boundary, a multiple of 16 bytes.
__device__ __forceinline__ void prefetch_codes(const signed char* from, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
}
// Up to 16 bytes to shared memory, zeros behind them, behind the thread's back.
__device__ __forceinline__ void copy_weights(uint32_t to, const signed char* from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy_tokens(uint32_t to, const signed char* from, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the thread's last N groups of copies have landed.
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sums of fp16 products in fp32, and of integer products in integers.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's 16 codes of a token, and 64 columns of K of 16 channels and NT groups
// of eight tokens: lo and hi are a lane's codes of channels g and g + 8.
template <int NT>
struct Whole {  // as integers
    uint4 b[NT];
    __device__ __forceinline__ void token(int i, const uint4& v) { b[i] = v; }
    __device__ __forceinline__ void add(int (&acc)[NT][4], const uint4& lo, const uint4& hi) {
#pragma unroll
        for (int i = 0; i < NT; ++i) mma(acc[i], lo.x, hi.x, lo.y, hi.y, b[i].x, b[i].y);
#pragma unroll
        for (int i = 0; i < NT; ++i) mma(acc[i], lo.z, hi.z, lo.w, hi.w, b[i].z, b[i].w);
    }
};
template <int NT>
struct Half {  // as fp16 numbers
    uint32_t b[NT][8];
    __device__ __forceinline__ void token(int i, const uint4& v) { decode_f16(v, b[i]); }
    __device__ __forceinline__ void add(float (&acc)[NT][4], const uint4& lo, const uint4& hi) {
        uint32_t l[8], h[8];
        decode_f16(lo, l);
        decode_f16(hi, h);
#pragma unroll
        for (int m = 0; m < 8; m += 2)
#pragma unroll
            for (int i = 0; i < NT; ++i)
                mma(acc[i], l[m], h[m], l[m + 1], h[m + 1], b[i][m], b[i][m + 1]);
    }
};

__device__ __forceinline__ uint4 lds_u32x4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void put_value(void* y, long long at, int type, float v) {
    if (type == kI8Bfloat16)
        static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(y)[at] = v;
}

// NT groups of eight tokens, CG groups of 16 channels; of one weight matrix, or
// gated (ACT not kI8NoAct) of two.
template <int NT, int CG, int ACT>
struct Stream {
    static constexpr bool GATED = ACT != kI8NoAct;
    static constexpr int SETS = CG * (GATED ? 2 : 1);  // of 16 channels
    static constexpr bool INTEGERS = NT == 1;          // which MMAs: see above
    using Step = std::conditional_t<INTEGERS, Whole<NT>, Half<NT>>;
    using Sum = std::conditional_t<INTEGERS, int, float>;
    static constexpr int PIECES = 2 * SETS + NT;       // 16-byte pieces of a lane and step
    static constexpr int STEP_BYTES = PIECES * 512;
    static constexpr int WARP_BYTES = kAhead * STEP_BYTES;
    static constexpr int WARPS = SETS * NT > 4 ? 8 : 16;  // at most
    static_assert(WARP_BYTES >= SETS * NT * 512, "sums fit a warp's slots");
};

template <int NT, int CG, int ACT>
__global__ void __launch_bounds__(32 * Stream<NT, CG, ACT>::WARPS)
i8_stream_kernel(I8StreamArgs p) {
    using S = Stream<NT, CG, ACT>;
    constexpr int SETS = S::SETS;
    extern __shared__ __align__(16) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int n0 = static_cast<int>(blockIdx.x) * (16 * CG);
    const uint32_t slots = smem_addr(smem) + warp * S::WARP_BYTES + 16 * lane;

    // this lane's rows (the last one again where there are no more), at its first step
    const int first = 64 * warp + 16 * c;
    const signed char* weights[SETS][2];
#pragma unroll
    for (int s = 0; s < SETS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const I8In& m = S::GATED && s >= CG ? p.c : p.b;
            const int n = min(n0 + 16 * (s % CG) + 8 * h + g, p.N - 1);
            weights[s][h] = m.codes + n * m.ld + first;
        }
    const signed char* tokens[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
        tokens[i] = p.a.codes + min(8 * i + g, p.T - 1) * p.a.ld + first;

    typename S::Sum acc[SETS][NT][4] = {};
    int total[SETS * NT * 4] = {};  // of fp32 sums

    const int stride = 64 * warps;
    // Columns in whole pieces of 16 (with copies of any size in every step 24 x 8192 x
    // 8192 took 19.8 us against 19.1, 32 tokens 22.9 against 21.4).  The rest of a row,
    // whose memory may end there, is a step before the others of the warp whose turn it is.
    const int whole = p.K & ~15;
    const bool tail = whole < p.K && warp == (whole + 63) / 64 % warps;
    // While the kernel before ends, the first codes of each channel are sent for,
    // to L2, which reads no value (a token, 4096 x 4096 5.3 to 5.1 us, 8192 x 8192
    // 13.6 to 13.2; 2048 bytes instead of 512 make gated 8192 x 2048 9.2 of 8.3).
    if (threadIdx.x < 16 * SETS) {
        const int s = threadIdx.x / 16;
        const I8In& m = S::GATED && s >= CG ? p.c : p.b;
        const int n = n0 + 16 * (s % CG) + threadIdx.x % 16;
        const int bytes = min(p.K, kEarlyBytes) & ~15;
        if (n < p.N && bytes) prefetch_codes(m.codes + n * m.ld, bytes);
    }
    pdl_wait();
    pdl_trigger();
    int ahead = first;  // the next step to copy: this lane's column
    const auto copy = [&](uint32_t slot) {
        const int there = ahead < whole ? 16 : 0;
#pragma unroll
        for (int s = 0; s < SETS; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                copy_weights(slot + 512 * (2 * s + h), weights[s][h], there);
                weights[s][h] += stride;
            }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            copy_tokens(slot + 512 * (2 * SETS + i), tokens[i], 8 * i + g < p.T ? there : 0);
            tokens[i] += stride;
        }
        ahead += stride;
        copies_commit();
    };
    if (tail) {
        // codes from `whole` on, in the place of a step's first 16
        const int there = c == 0 ? p.K - whole : 0;
        const int back = whole - 64 * warp;
#pragma unroll
        for (int s = 0; s < SETS; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                copy_weights(slots + 512 * (2 * s + h), weights[s][h] + back, there);
#pragma unroll
        for (int i = 0; i < NT; ++i)
            copy_tokens(slots + 512 * (2 * SETS + i), tokens[i] + back, 8 * i + g < p.T ? there : 0);
        copies_commit();
    } else {
        copy(slots);
    }
#pragma unroll
    for (int i = 1; i < kAhead - 1; ++i) copy(slots + i * S::STEP_BYTES);
    // the slot to read, and the one read before
    uint32_t slot = slots, last = slots + (kAhead - 1) * S::STEP_BYTES;

    int exact = 0;
    for (int k = 64 * warp - (tail ? stride : 0); k < whole; k += stride) {
        copies_wait<kAhead - 2>();
        typename S::Step now;
#pragma unroll
        for (int i = 0; i < NT; ++i) now.token(i, lds_u32x4(slot + 512 * (2 * SETS + i)));
#pragma unroll
        for (int s = 0; s < SETS; ++s)
            now.add(acc[s], lds_u32x4(slot + 512 * (2 * s)), lds_u32x4(slot + 512 * (2 * s + 1)));
        copy(last);
        last = slot;
        slot = slot == slots + (kAhead - 1) * S::STEP_BYTES ? slots : slot + S::STEP_BYTES;
        if (!S::INTEGERS && ++exact == kExactSteps) {
            exact = 0;
#pragma unroll
            for (int f = 0; f < SETS * NT * 4; ++f) {
                float& v = reinterpret_cast<float&>(acc[f / (4 * NT)][f / 4 % NT][f % 4]);
                total[f] += __float2int_rn(v);
                v = 0.0f;
            }
        }
    }
    // the warp's sums over its slots
    copies_wait<0>();
    __syncwarp();
    int4* const sums = reinterpret_cast<int4*>(smem);
    constexpr int kSums = S::WARP_BYTES / 16;  // from warp to warp
#pragma unroll
    for (int f = 0; f < SETS * NT; ++f) {
        int v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            v[x] = S::INTEGERS ? static_cast<int>(acc[f / NT][f % NT][x])
                               : total[4 * f + x] +
                                     __float2int_rn(static_cast<float>(acc[f / NT][f % NT][x]));
        sums[warp * kSums + f * 32 + lane] = make_int4(v[0], v[1], v[2], v[3]);
    }
    __syncthreads();
    // a lane's four sums of a fragment: channels g and g + 8, tokens 2 c and 2 c + 1
    for (int f = warp; f < CG * NT; f += warps) {
        const int s = f / NT, i = f % NT;
        int v[S::GATED ? 2 : 1][4] = {};
#pragma unroll
        for (int m = 0; m < (S::GATED ? 2 : 1); ++m)
            for (int x = 0; x < warps; ++x) {
                const int4 more = sums[x * kSums + ((s + m * CG) * NT + i) * 32 + lane];
                v[m][0] += more.x, v[m][1] += more.y, v[m][2] += more.z, v[m][3] += more.w;
            }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int n = n0 + 16 * s + g + 8 * (x / 2), t = 8 * i + 2 * c + x % 2;
            if (n >= p.N || t >= p.T) continue;
            const long long to = t * p.ldy + n;
            if (!S::GATED && p.type == kI8Int32) {
                static_cast<int*>(p.y)[to] = v[0][x];
                continue;
            }
            const float st = p.a.scales[t];
            float value = i8_value(__int2float_rn(v[0][x]), st, p.b.scales[n]);
            if (S::GATED)
                value = i8_act<ACT>(value) *
                        i8_value(__int2float_rn(v[S::GATED ? 1 : 0][x]), st, p.c.scales[n]);
            put_value(p.y, to, p.type, value);
        }
    }
}

// Registers of the kernel's threads, once it is set up on device `dev`.  The
// ABI's mutex is held.
template <int NT, int CG, int ACT>
cudaError_t configure(int dev, int* regs) {
    constexpr int kDevices = 64;
    static int known[kDevices] = {};
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (!known[dev]) {
        const auto kernel = i8_stream_kernel<NT, CG, ACT>;
        cudaFuncAttributes attr;
        cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBlockBytes);
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, kernel);
        if (e != cudaSuccess) return e;
        known[dev] = attr.numRegs;
    }
    *regs = known[dev];
    return cudaSuccess;
}

// Warps a block: four, or as many more as make 24 an SM, if the blocks that an SM
// gets of them find room in it side by side.  (Of a token through 8192 x 8192
// four, 13.1 us, eight 14.1; 4096 x 4096 eight 5.1, sixteen 5.7, four 6.0; 16384 x
// 16384 four 46.6, two 49.8.)  Each block then asks for its whole share of the
// SM's shared memory: a block more, on an SM that was done sooner with the kernel
// before, would take it longer than the others (gated 8192 x 2048 8.3 us against
// 9.3, 14336 x 4096 11.4 against 14.3).
template <int NT, int CG, int ACT>
cudaError_t launch(const I8StreamArgs& p, cudaStream_t stream, int dev, int sm_count) {
    using S = Stream<NT, CG, ACT>;
    int regs;
    cudaError_t e = configure<NT, CG, ACT>(dev, &regs);
    if (e != cudaSuccess) return e;
    const int blocks = (p.N - 1) / (16 * CG) + 1, steps = (p.K - 1) / 64 + 1;
    const int per = std::min((blocks - 1) / sm_count + 1, 8);
    const int share = std::min(kSharedBytes / per - 1024, kBlockBytes) & ~1023;
    const auto room = [&](int w) {
        return w * S::WARP_BYTES <= share && per * w * 32 * ((regs + 7) & ~7) <= 65536;
    };
    int warps = S::WARPS;
    while (warps > 2 &&
           (!room(warps) || steps < 2 * warps ||
            (warps > 4 && static_cast<long long>(blocks) * warps > 24LL * sm_count)))
        warps /= 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = per > 1 ? std::max(warps * S::WARP_BYTES, share) : warps * S::WARP_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, i8_stream_kernel<NT, CG, ACT>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// 32 channels a block convert the tokens' codes half as often as 16, but are
// half as many blocks: from about half a block an SM on (24 x 4096 x 4096 7.4 us
// against 8.5, 24 x 1024 x 8192 9.6 against 7.0).
bool two_groups(int N, int sm_count) { return (N - 1) / 32 + 1 > sm_count / 2; }
template <int NT, int ACT>
cudaError_t by_channels(const I8StreamArgs& p, cudaStream_t stream, int dev, int sm_count) {
    constexpr int kTwo = ACT == kI8NoAct && NT > 1 ? 2 : 1;
    if (!two_groups(p.N, sm_count)) return launch<NT, 1, ACT>(p, stream, dev, sm_count);
    return launch<NT, kTwo, ACT>(p, stream, dev, sm_count);
}

template <int ACT>
cudaError_t by_tokens(const I8StreamArgs& p, cudaStream_t stream, int dev, int sm_count) {
    if (p.T <= 8) return by_channels<1, ACT>(p, stream, dev, sm_count);
    if (p.T <= 16) return by_channels<2, ACT>(p, stream, dev, sm_count);
    if (p.T <= 24) return by_channels<3, ACT>(p, stream, dev, sm_count);
    return by_channels<4, ACT>(p, stream, dev, sm_count);
}

}  // namespace

int i8_stream_channels(int T, int N, bool gated, int sm_count) {
    const int channels = T > 8 && !gated && two_groups(N, sm_count) ? 32 : 16;
    const int blocks = (N - 1) / channels + 1;
    return ((blocks - 1) / sm_count + 1) * channels * (gated ? 2 : 1);
}

cudaError_t launch_i8_stream(const I8StreamArgs& p, cudaStream_t stream, int dev,
                             int sm_count) {
    if (p.act == kActSilu) return by_tokens<kActSilu>(p, stream, dev, sm_count);
    if (p.act == kActGelu) return by_tokens<kActGelu>(p, stream, dev, sm_count);
    return by_tokens<kI8NoAct>(p, stream, dev, sm_count);
}

}  // namespace gemm_f32_impl
