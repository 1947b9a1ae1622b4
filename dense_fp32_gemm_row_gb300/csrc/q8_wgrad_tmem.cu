// q8_wgrad_tmem.cu -- the weight gradient from an 8-bit checkpoint on the
// tensor core:  dW[d][n] = sum_t x^[t][d] dY[t][n].
//
// Arithmetic.  Every value of the checkpoint is exactly a bf16 number.  A
// float of dY (from 2^-110 up) is exactly the sum of three: b0 its upper 16
// bits, b1 the upper 16 bits of y - b0, b2 = y - b0 - b1 (8 significant bits
// each, truncated, so the differences are exact).  Three bf16 MMAs a step, x^ b2 + x^ b1 + x^ b0,
// thus form exact products of the fp32 values; what is rounded is the
// accumulation.  The tensor core truncates its running fp32 sum at each
// addition (an error of about 2^-24 * 0.7 of the sum, always towards zero),
// so a tensor-memory sum covers one chunk of tokens and is then added, with
// rounding, into fp32 registers.  (Two bf16 parts would leave 2^-17 of each
// product; TF32 parts need two MMAs at half the rate.)  The tensor core
// takes denormal parts as they are, so what is lost of dY is what lies below
// the least of them, 2^-133: nothing from 2^-110 up.  An infinity in dY leaves
// a NaN part, as in the 3xTF32 kernels, so it comes back as NaN.
//
// Shape.  Both operands have the summed index, the token, as their slow
// axis.  The MMA's A operand comes from tensor memory, one row per lane, and
// a thread writes its own lane: thread n of the splitter warpgroup reads
// column n of the dY stage (consecutive lanes, consecutive words), splits and
// stores the parts, which transposes them on the way.  x^ is the B operand in
// shared memory, which bf16 MMAs take with the features contiguous as they
// are stored, so its decoder writes rows as it reads them.  D is the
// transposed tile: lane n, column d.
//
// Two forms.  A cluster of two CTAs computes a tile of 256 features x 256
// columns with cta_group::2 MMAs (M = 256 columns n across the pair, N = 256
// features, K = 16 tokens), CTA rank r holding columns n0 + 128 r .. in its
// tensor memory and half of the features in its shared memory.  Per 16 tokens
// an SM's tensor core works 3 x 128 cycles and reads 12 KB of shared memory,
// half its share; dY in shared memory as well (both operands, three parts)
// would take more than the whole.  Or one CTA computes 256 x 128 (M = 128) and
// holds all the features: it decodes and reads twice as much of x^ for the
// same MMAs (8192 x 8192 x 8192 2.12 ms against 1.89), but wastes less of them
// on few or odd columns, is quicker to start, and has no partner to tell
// (16384 x 8192 x 32 81 us against 139, 64 x 512 x 512 6.3 against 6.8).  In a
// tile with fewer features the MMAs are as much narrower.
//
// 640 threads per CTA, registers rebalanced at start (launched at 96 each):
//   warp 0       one lane: TMA loads of a 32-token stage (dY 128 columns x 32,
//                codes 128 x 32 once or twice, exponents 16 x 32), six stages
//                deep (five in the single form);
//   warp 1       tensor-memory allocation; one lane (of a pair: the leader's)
//                issues the MMAs and commits;
//   warps 1-3 of a pair's peer  relay: one lane each tells the leader, in turn,
//                that the peer's operands of a stage are written;
//   warps 4-7    split dY into tensor memory (warp 4 + q: lanes 32 q ..);
//   warps 8-11   decode x^ to bf16 in shared memory, eight tokens each;
//   warps 12-19  per chunk add the accumulator (warp 12 + e: lanes 32 (e % 4)
//                .., columns 128 (e / 4) ..) into 128 registers a thread; at
//                the end of a unit store them: a warp writes 32 consecutive
//                columns of one row of dW.
// Tensor memory: 256 accumulator columns, then five operand stages of 48 (three
// parts of 32 tokens, two to a column).  Copies and operands are separate
// rings, so that DRAM and L2 latency is not part of the operand loop (MMA,
// commit, conversion, relay: ~1.5 us of the five stages' 2.0).
//
// What set the speed, 8192 x 8192 x 8192 (INT8), pairs: one relay lane for the
// peer, whose release at cluster scope takes ~650 ns against 400 ns of MMAs a
// stage, 2.69 ms; three relays and the separate rings 2.19; four decoder warps
// instead of two, each of whose stores fills all banks, 1.89 (2.00 to 2.04
// back to back at the power limit).  With operands that are never rewritten the same
// MMAs and copies take 1.70 ms; three bf16 products at the burst rate of the
// library's product take 1.72, at its sustained rate 1.91.  4096 x 2048 x
// 2048: 74.2 us, 64 tiles on 76 pairs, the tensor pipe busy 79 % of a CTA's
// life, a stage 0.53 us.
//
// Where the tiles do not fill the units evenly, the last of them are shared:
// their stages, end to end, are cut into equal runs, whose partial sums a
// second kernel adds in order.  (Adding them in this kernel, by CTAs that
// wait for one another, took 1000 x 1024 x 1024 20.5 us against 15.2: the
// second kernel starts as a programmatic dependent.)
// Waits are bounded and wind down as in the GEMM kernels.
#include <cstdint>

#include "device_sync.cuh"
#include "epilogue.cuh"
#include "gemm_internal.h"
#include "q8_format.cuh"
#include "tcgen05.cuh"
#include "tf32x3_common.cuh"

namespace gemm_f32_impl {
namespace {

using namespace gemm_f32_dev;

template <bool PAIR_>
struct WgradCfg {
    static constexpr bool PAIR = PAIR_;
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int TD = 256, TN = 128 * CTAS;  // features, columns of a tile
    static constexpr int CTA_D = TD / CTAS;          // per CTA: features in shared memory,
    static constexpr int CTA_N = 128;                // columns in tensor-memory lanes
    static constexpr int KT = 32;                    // tokens a stage
    static constexpr int UK = 16;                    // tokens an MMA
    static constexpr int RAW = PAIR ? 6 : 5;         // stages of copies
    static constexpr int STAGES = 5;                 // stages of MMA operands
    static constexpr int XB_BYTES = CTA_D * KT * 2;  // x^ in bf16: 64-feature groups
    static constexpr int GROUP_BYTES = 64 * KT * 2;  // rows of 128 bytes, a token each
    static constexpr int Y_BYTES = CTA_N * KT * 4;
    // dY by rows of one residue modulo 4, four columns wider (see the kernel)
    static constexpr int SHIFT_PITCH = (CTA_N + 4) * 4;
    static constexpr int SHIFT_GROUP = KT / 4 * SHIFT_PITCH;
    static constexpr int Y_SLOT = 4 * SHIFT_GROUP;
    static constexpr int C_BOX_BYTES = 128 * KT;     // codes: boxes of 128 features
    static constexpr int C_BYTES = CTA_D * KT;
    static constexpr int S_BYTES = 16 * KT;
    // the swizzled x^ stages first: each 1024-byte aligned
    static constexpr int Y_OFF = STAGES * XB_BYTES;
    static constexpr int C_OFF = Y_OFF + RAW * Y_SLOT;
    static constexpr int S_OFF = C_OFF + RAW * C_BYTES;
    static constexpr int BAR_OFF = S_OFF + RAW * S_BYTES;
    static constexpr int CONV_WARPS = 4 + 4;  // splitters, decoders
    // full, free (per copy stage), empty, ready (per operand stage), acc_full, acc_empty, drain
    static constexpr int NBARS = 2 * RAW + 2 * STAGES + 3;
    static constexpr int SMEM_BYTES = BAR_OFF + NBARS * 8 + 16 + 1024;
    static constexpr int THREADS = 640;
    static constexpr int TMEM_COLS = 512;
    static constexpr int OP_COL0 = TD;               // operand stage s at OP_COL0 + 48 s
    static constexpr int PART_COLS = KT / 2;
    static constexpr int OP_COLS = 3 * PART_COLS;
    static constexpr int RELAYS = 3;
    static constexpr int EPI_WARPS = 8;
    static constexpr int REGS_LAUNCH = 96;
    static constexpr int REGS_CONTROL = 40, REGS_SPLIT = 48, REGS_DECODE = 56, REGS_EPI = 168;
    static constexpr int DRAIN_BATCH = 2;
    // D fp32, A and B bf16, B with its N axis contiguous, M = TN; N is added
    static constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) |
                                      (static_cast<uint32_t>(TN >> 4) << 24);
    static_assert(REGS_CONTROL + REGS_SPLIT + REGS_DECODE + 2 * REGS_EPI <= 5 * REGS_LAUNCH,
                  "register shares");
    static_assert(OP_COL0 + STAGES * OP_COLS <= TMEM_COLS, "tensor-memory columns");
    static_assert(SHIFT_GROUP % 128 == 0 && Y_SLOT >= Y_BYTES, "dY stages");
    static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
};

// Shared-memory descriptor of the x^ stage: N-contiguous with 128-byte
// swizzle.  Rows of 64 features (128 bytes), one a token; eight rows make a
// 1024-byte swizzle group (stride byte offset, along K); the next 64 features
// lie GROUP_BYTES further on (leading byte offset, along N).
__device__ __forceinline__ uint64_t xhat_desc(uint32_t addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(WgradCfg<true>::GROUP_BYTES >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void lds_u32x2(uint32_t addr, uint32_t (&v)[2]) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(v[0]), "=r"(v[1])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void sts_u32x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                          uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Upper halves of two floats: bf16 truncations of a (low) and b (high).
__device__ __forceinline__ uint32_t upper_halves(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
// (a, b) minus their bf16 truncations, exact.
__device__ __forceinline__ void drop_upper(float& a, float& b) {
    const float na = __uint_as_float((__float_as_uint(a) & 0xFFFF0000u) ^ 0x80000000u);
    const float nb = __uint_as_float((__float_as_uint(b) & 0xFFFF0000u) ^ 0x80000000u);
    asm("{\n\t.reg .b64 x, n;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 n, {%2, %3};\n\t"
        "add.rn.f32x2 x, x, n;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(na), "f"(nb));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Four codes as two words of two bf16 values each, exact.  INT8: the low
// seven bits of a code below the upper byte of 128 are the bf16 number 128 +
// low, and its sign bit alone there is 128 or 256, so their difference is the
// code; five instructions for two codes against 7.5 through fp32.
template <int FMT>
__device__ __forceinline__ void decode_bf16(uint32_t w, float scale, uint32_t& lo, uint32_t& hi) {
    if (FMT == kQ8Int8) {
        const uint32_t s2 = upper_halves(scale, scale);
        const uint32_t p = __byte_perm(w, 0x43434343u, 0x4140);
        const uint32_t q = __byte_perm(w, 0x43434343u, 0x4342);
        lo = mul_bf16x2(sub_bf16x2(p & 0xFF7FFF7Fu, p & 0xFF80FF80u), s2);
        hi = mul_bf16x2(sub_bf16x2(q & 0xFF7FFF7Fu, q & 0xFF80FF80u), s2);
        return;
    }
    const float4 v = q8_decode4<FMT>(w);
    lo = upper_halves(v.x * scale, v.y * scale);
    hi = upper_halves(v.z * scale, v.w * scale);
}

// D += A B^T, A in tensor memory, for one CTA or (leader's thread) the pair.
template <bool PAIR>
__device__ __forceinline__ void mma_bf16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}
// Arrival on a barrier, in both CTAs of a pair, when the MMAs so far are done.
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar) {
    if (PAIR)
        mma_commit_pair_multicast(bar, 0x3);
    else
        mma_commit(bar);
}

// First feature and column of a tile: neighbouring tiles run down groups of 8
// rows of tiles, so that the clusters at work share operands in L2.
template <class C>
__device__ __forceinline__ void tile_at(const Q8WgradShare& sh, int tile, int& d0, int& n0) {
    const int per_group = GROUP_M * sh.tiles_n;
    const int group = tile / per_group, within = tile - group * per_group;
    const int rows = min(sh.tiles_d - group * GROUP_M, GROUP_M);
    const int column = within / rows;
    d0 = (group * GROUP_M + within - column * rows) * C::TD;
    n0 = column * C::TN;
}

// The work of one cluster (or CTA), piece by piece: a whole tile, or a run of stages of
// a shared tile.  A run may cover parts of several tiles; a part of a tile goes to slot (run + tile) of the partial sums, so that the slots of
// one tile follow one another in the order of its stages.
template <class C>
struct Pieces {
    int u;          // next unit
    int run, b, e;  // the current run, its stages left

    __device__ __forceinline__ Pieces() : u(blockIdx.x / C::CTAS), run(0), b(0), e(0) {}

    __device__ __forceinline__ bool next(const Q8WgradShare& sh, Unit& w) {
        int tile = u;
        w.kb_begin = 0;
        w.nkb = sh.stages;
        w.slot = -1;
        if (b >= e) {
            if (u >= sh.whole + sh.runs) return false;
            if (u >= sh.whole) {
                run = u - sh.whole;
                b = q8_wgrad_cut(sh, run);
                e = q8_wgrad_cut(sh, run + 1);
            }
            u += gridDim.x / C::CTAS;
        }
        if (b < e) {
            const int t = b / sh.stages;
            tile = sh.whole + t;
            w.kb_begin = b - t * sh.stages;
            w.nkb = min(sh.stages - w.kb_begin, e - b);
            b += w.nkb;
            if (w.nkb < sh.stages) w.slot = run + t;
        }
        tile_at<C>(sh, tile, w.m0, w.n0);
        return true;
    }
};

// Adds the partial sums of the shared tiles, in the order of their stages, and
// writes dW, 256 threads a block.
//   Q = 1: a thread adds four columns of G rows at once, B partials of each in
//   flight;
//   Q = 4: for few outputs with many partials, each bound by the latency of
//   its loads: four lanes share a group of four columns, each adding a
//   contiguous quarter of the partials, B in flight, and their sums are added
//   in order.
template <class C, int Q, int G, int B>
__global__ void __launch_bounds__(256)
q8_wgrad_sum_kernel(const float* __restrict__ parts, Q8WgradShare sh, float* __restrict__ dw,
                    long long lddw, bool vec, int D, int N, float alpha, float beta, int mode) {
    constexpr int kPart = C::TD * C::TN;
    constexpr int kRows = 256 / Q / (C::TN / 4);  // of a block, in each of G passes
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int q = Q == 1 ? 0 : lane / (32 / Q);
    const int group = warp * (32 / Q) + lane % (32 / Q);  // of 256 / Q groups of four columns
    const int col = 4 * (group % (C::TN / 4));
    const int row0 = kRows * G * static_cast<int>(blockIdx.x) + group / (C::TN / 4);
    for (int t = blockIdx.y; t < sh.shared; t += gridDim.y) {
        // the runs that hold the tile's first and last stage
        int first = t * sh.group_runs, n = sh.group_runs;
        if (sh.group_stages != sh.stages) {
            first = q8_wgrad_run(sh, t * sh.stages);
            n = q8_wgrad_run(sh, (t + 1) * sh.stages - 1) - first + 1;
        }
        pdl_wait();  // the partial sums: only indices before it
        if (n == 1) continue;  // written by its cluster
        int d0, n0;
        tile_at<C>(sh, sh.whole + t, d0, n0);
        const int per = (n + Q - 1) / Q;
        const int i1 = n0 + col < N ? min(n, (q + 1) * per) : 0;
        const float* src = parts + static_cast<long long>(first + t) * kPart + col;
        float4 sum[G];
        int row[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            sum[g] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            row[g] = row0 + g * kRows;
        }
        for (int i0 = q * per; i0 < i1; i0 += B) {
            float4 v[G][B];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int k = 0; k < B; ++k)
                    if (i0 + k < i1 && d0 + row[g] < D)
                        v[g][k] = __ldcg(reinterpret_cast<const float4*>(
                            src + static_cast<long long>(i0 + k) * kPart + row[g] * C::TN));
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int k = 0; k < B; ++k)
                    if (i0 + k < i1 && d0 + row[g] < D) {
                        sum[g].x += v[g][k].x;
                        sum[g].y += v[g][k].y;
                        sum[g].z += v[g][k].z;
                        sum[g].w += v[g][k].w;
                    }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            // lanes of the first quarter gather the others' sums, in order
            float4 all = sum[g];
#pragma unroll
            for (int k = 1; k < Q; ++k) {
                const int from = lane % (32 / Q) + k * (32 / Q);
                all.x += __shfl_sync(0xffffffffu, sum[g].x, from);
                all.y += __shfl_sync(0xffffffffu, sum[g].y, from);
                all.z += __shfl_sync(0xffffffffu, sum[g].z, from);
                all.w += __shfl_sync(0xffffffffu, sum[g].w, from);
            }
            if (q == 0 && i1 > 0 && d0 + row[g] < D)
                store4(dw + static_cast<long long>(d0 + row[g]) * lddw, n0 + col, N, all, vec,
                       alpha, beta, mode);
        }
    }
}

// A thread's accumulators to the rows below one another at p: partial sums,
// which are read again at once, or dW, which is first to leave the L2 cache for
// operands that are still to be read (8192 x 8192 outputs of 64 tokens 52.4 us
// against 54.2, of 256 96.4 against 98.4, of 512 158.4 against 161.2; through
// shared memory and bulk stores 51.4, 93.9 and 157.2, but 4096 x 4096 of one
// token 19.0 against 17.5, whose time is that of the last tiles).
template <bool DW>
__device__ __forceinline__ void store_columns(const float (&acc)[EPI_COLS], float* p, long long ld,
                                              int rows) {
    const auto put = [](float* at, float v) {
        if (DW)
            __stcs(at, v);
        else
            *at = v;
    };
    if (rows >= EPI_COLS) {
#pragma unroll
        for (int j = 0; j < EPI_COLS; ++j) put(p + j * ld, acc[j]);
    } else {
#pragma unroll
        for (int j = 0; j < EPI_COLS; ++j)
            if (j < rows) put(p + j * ld, acc[j]);
    }
}

// Features that each CTA holds of a tile with `left` features from its first
// to the last of x: all of them, or in a matrix's last tiles as few blocks of
// 32 as cover the rest, so that the MMAs are no wider than they need to be.
template <class C>
__device__ __forceinline__ int cta_features(int left) {
    const int each = (left + C::CTAS - 1) / C::CTAS;
    return min(C::CTA_D, (each + 31) & ~31);
}

// SHIFTED: rows of dY that do not start on 16-byte boundaries, as TMA loads
// must.  Four row strides are a multiple of 16 bytes whatever the stride, so
// the rows t = 4 i + c of each residue c form a matrix that a tensor map can
// describe, from the 16-byte boundary at or before its first element: its
// columns then lie shifts[c] (0 .. 3 floats, two bits each) further right, and
// a box four columns wider holds the tile's.  Such a stage is four boxes of 8
// rows, and the splitter adds the shift; no padded copy of dY is made.
template <bool PAIR, int FMT, bool SHIFTED>
__global__ void __launch_bounds__(WgradCfg<PAIR>::THREADS, 1)
q8_wgrad_kernel(const __grid_constant__ Q8WgradMaps tmY, unsigned shifts,
                     const __grid_constant__ CUtensorMap tmC,
                     const __grid_constant__ CUtensorMap tmS, float* __restrict__ dw,
                     long long lddw, float* __restrict__ parts, int D, int N, int T,
                     Q8WgradShare share, int chunk, unsigned* fault, long long timeout_ns,
                     float alpha, float beta, int scale_mode) {
    using C = WgradCfg<PAIR>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_addr(smem);
    const uint32_t full0 = sbase + C::BAR_OFF;      // own: a copy stage has landed
    const uint32_t free0 = full0 + 8 * C::RAW;      // own: its readers are done
    const uint32_t empty0 = free0 + 8 * C::RAW;     // own, multicast commit: operands read
    const uint32_t ready0 = empty0 + 8 * STAGES;    // operands written
    const uint32_t accf = ready0 + 8 * STAGES;      // own, multicast commit
    const uint32_t acce = accf + 8;                 // leader: 8 warps a CTA
    const uint32_t drain = acce + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::BAR_OFF + C::NBARS * 8);
    const uint32_t abort_flag = smem_addr(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0;

    if (threadIdx.x == 0) {
        for (int c = 0; c < (SHIFTED ? 4 : 1); ++c) prefetch_tmap(&tmY.map[c]);
        prefetch_tmap(&tmC);
        prefetch_tmap(&tmS);
        for (int r = 0; r < C::RAW; ++r) {
            mbar_init(full0 + 8 * r, 1);
            mbar_init(free0 + 8 * r, C::CONV_WARPS);
        }
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(empty0 + 8 * s, 1);
            // in the leader also the relay of the peer's
            mbar_init(ready0 + 8 * s, C::CONV_WARPS + (PAIR && rank == 0 ? 1 : 0));
        }
        mbar_init(accf, 1);
        mbar_init(acce, C::CTAS * C::EPI_WARPS);
        mbar_init(drain, 1);
        st_shared_volatile(abort_flag, 0u);
        fence_barrier_init();
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(smem_addr(tmem_slot), C::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_addr(tmem_slot), C::TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if (PAIR)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    // The peer's arrivals on its ready barriers, passed on to the leader's: relay
    // i of RELAYS takes every RELAYS-th stage.  A release at cluster scope
    // takes ~650 ns on this part, more than the MMAs of a stage (400 ns), so
    // several warps have one each in flight.
    auto relay = [&](int i) {
        const uint32_t ready_leader = map_to_cta(ready0, 0);
        int total = 0;
        Unit w;
        for (Pieces<C> todo; todo.next(share, w);) total += w.nkb;
        for (int it = i; it < total; it += C::RELAYS) {
            const int s = it % STAGES;
            if (!role_wait(ready0 + 8 * s, (it / STAGES) & 1, timeout_ns, fault, kFaultFullBarrier,
                           abort_flag))
                break;
            mbar_arrive_cluster(ready_leader + 8 * s);
        }
    };

    if (warp < 4) {
        regs_dec<C::REGS_CONTROL>();
        if (warp == 0) {
            if (lane == 0) {
                // -------------------------- TMA producer ------------------------------
                int it = 0;
                bool ok = true;
                Unit w;
                for (Pieces<C> todo; ok && todo.next(share, w);) {
                    const int dc = w.m0 + static_cast<int>(rank) * cta_features<C>(D - w.m0);
                    const int nc = w.n0 + static_cast<int>(rank) * C::CTA_N;
                    // exponents: the aligned 16 blocks that hold this CTA's
                    const int bc = (dc / kQ8Block) & ~15;
                    for (int kb = 0; kb < w.nkb; ++kb, ++it) {
                        const int r = it % C::RAW;
                        if (it >= C::RAW &&
                            !role_wait(free0 + 8 * r, ((it / C::RAW) & 1) ^ 1, timeout_ns, fault,
                                       kFaultEmptyBarrier, abort_flag)) {
                            ok = false;
                            break;
                        }
                        const int t0 = (w.kb_begin + kb) * C::KT;
                        const uint32_t fb = full0 + 8 * r;
                        const uint32_t yb = sbase + C::Y_OFF + r * C::Y_SLOT;
                        mbar_arrive_expect_tx(
                            fb, (SHIFTED ? C::Y_SLOT : C::Y_BYTES) + C::C_BYTES + C::S_BYTES);
                        if (SHIFTED) {
                            // a residue without rows (T < 4) reads beyond its map: zeros
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                tma_load_2d(yb + c * C::SHIFT_GROUP, &tmY.map[c], fb, nc,
                                            c < T ? t0 / 4 : C::KT);
                        } else {
                            tma_load_2d(yb, &tmY.map[0], fb, nc, t0);
                        }
#pragma unroll
                        for (int c = 0; c < C::CTA_D / 128; ++c)
                            tma_load_2d(sbase + C::C_OFF + r * C::C_BYTES + c * C::C_BOX_BYTES, &tmC,
                                        fb, dc + 128 * c, t0);
                        tma_load_2d(sbase + C::S_OFF + r * C::S_BYTES, &tmS, fb, bc, t0);
                    }
                }
                // wind down: this CTA's copies have landed, and the MMAs' commits
                // have reached its operand stages
                const long long tail = ok ? timeout_ns : timeout_ns / 8 + 1000;
                for (int j = (it > C::RAW ? it - C::RAW : 0); j < it; ++j)
                    mbar_wait(full0 + 8 * (j % C::RAW), (j / C::RAW) & 1, tail, fault, kFaultDrain);
                for (int j = (it > STAGES ? it - STAGES : 0); j < it; ++j)
                    mbar_wait(empty0 + 8 * (j % STAGES), (j / STAGES) & 1, tail, fault, kFaultDrain);
            }
            __syncwarp();
        } else if (warp == 1) {
            if (lane == 0 && rank == 0) {
                // -------------------------- MMA issuer (of a pair: the leader) --------
                int it = 0;
                int g = 0;  // chunks issued
                bool ok = true;
                Unit w;
                for (Pieces<C> todo; ok && todo.next(share, w);) {
                    const uint32_t idesc =
                        C::IDESC |
                        static_cast<uint32_t>(C::CTAS * cta_features<C>(D - w.m0) / 8) << 17;
                    for (int c0 = 0; c0 < w.nkb && ok; c0 += chunk, ++g) {
                        // the single accumulator: chunk g - 1 has been drained
                        if (g >= 1 && !role_wait(acce, (g - 1) & 1, timeout_ns, fault,
                                                 kFaultAccumBarrier, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const int c1 = min(w.nkb, c0 + chunk);
                        for (int kb = c0; kb < c1; ++kb, ++it) {
                            const int s = it % STAGES;
                            if (!role_wait<PAIR>(ready0 + 8 * s, (it / STAGES) & 1, timeout_ns,
                                                 fault, kFaultFullBarrier, abort_flag)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint64_t x = xhat_desc(sbase + s * C::XB_BYTES);
                            const uint32_t b0 =
                                tmem_base + static_cast<uint32_t>(C::OP_COL0 + C::OP_COLS * s);
                            const uint32_t b1 = b0 + C::PART_COLS, b2 = b1 + C::PART_COLS;
#pragma unroll
                            for (int k = 0; k < C::KT / C::UK; ++k) {
                                // 16 rows of 128 bytes; 16 tokens are 8 columns
                                const uint64_t xk = x + static_cast<uint64_t>((k * C::UK * 128) >> 4);
                                const uint32_t kc = static_cast<uint32_t>(k * C::UK / 2);
                                const uint32_t acc = (kb > c0 || k > 0) ? 1u : 0u;
                                mma_bf16_tmem_a<PAIR>(tmem_base, b2 + kc, xk, idesc, acc);
                                mma_bf16_tmem_a<PAIR>(tmem_base, b1 + kc, xk, idesc, 1u);
                                mma_bf16_tmem_a<PAIR>(tmem_base, b0 + kc, xk, idesc, 1u);
                            }
                            commit<PAIR>(empty0 + 8 * s);
                        }
                        if (!ok) break;
                        commit<PAIR>(accf);
                    }
                }
                if (PAIR)
                    mma_commit_pair(drain);
                else
                    mma_commit(drain);
                mbar_wait(drain, 0, ok ? timeout_ns : timeout_ns / 8 + 1000, fault, kFaultDrain);
            } else if (PAIR && lane == 0) {
                relay(0);
            }
            __syncwarp();
        } else if (PAIR && rank == 1 && lane == 0) {
            // ------------------------------ relays (warps 2-3 of the peer) ------------
            relay(warp - 1);
        }
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------ dY splitters (warps 4-7) ----------------------
        regs_dec<C::REGS_SPLIT>();
        const int q = warp & 3;
        uint32_t at[4];  // SHIFTED: a residue's rows in a stage, and their shift
#pragma unroll
        for (int c = 0; c < 4; ++c)
            at[c] = static_cast<uint32_t>(c * C::SHIFT_GROUP) + 4u * ((shifts >> (2 * c)) & 3u);
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
        int it = 0;
        bool ok = true;
        Unit w;
        for (Pieces<C> todo; ok && todo.next(share, w);) {
            const bool columns = w.n0 + static_cast<int>(rank) * C::CTA_N + 32 * q < N;
            for (int kb = 0; kb < w.nkb; ++kb, ++it) {
                const int s = it % STAGES, raw = it % C::RAW;
                bool got = role_wait(full0 + 8 * raw, (it / C::RAW) & 1, timeout_ns, fault,
                                     kFaultFullBarrier, abort_flag);
                if (got && it >= STAGES)
                    got = role_wait(empty0 + 8 * s, ((it / STAGES) & 1) ^ 1, timeout_ns, fault,
                                    kFaultEmptyBarrier, abort_flag);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                // the MMAs that read this stage before are done
                tc_fence_after();
                const uint32_t src = sbase + C::Y_OFF + raw * C::Y_SLOT +
                                     static_cast<uint32_t>(4 * (32 * q + lane));
                const uint32_t col =
                    lane_base + static_cast<uint32_t>(C::OP_COL0 + C::OP_COLS * s);
                // 16 tokens at a time: this warpgroup runs on 48 registers.  Lanes of
                // columns beyond dY's last keep what they hold: no output reads them.
#pragma unroll
                for (int h = 0; h < (columns ? C::KT / 16 : 0); ++h) {
                    float y[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint32_t t = static_cast<uint32_t>(16 * h + i);
                        y[i] = lds_f32(SHIFTED ? src + at[i & 3] + (t >> 2) * C::SHIFT_PITCH
                                               : src + t * (4 * C::CTA_N));
                    }
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
                        uint32_t p[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            p[i] = upper_halves(y[2 * i], y[2 * i + 1]);
                            if (part < 2) drop_upper(y[2 * i], y[2 * i + 1]);
                        }
                        tmem_st_32x32b_x8(col + static_cast<uint32_t>(part * C::PART_COLS + 8 * h),
                                          p);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(ready0 + 8 * s);
                    mbar_arrive(free0 + 8 * raw);
                }
            }
        }
        __syncwarp();
    } else if (warp < 12) {
        // ------------------------------ x^ decoders (warps 8-11) ----------------------
        // A lane takes eight codes of a token row: 16 lanes load 128 contiguous
        // bytes, and each eight lanes store the eight 16-byte chunks of one row of
        // one 64-feature group.
        regs_dec<C::REGS_DECODE>();
        constexpr int kRowLanes = C::CTA_D / 8;         // 16 or 32
        constexpr int kStep = 32 / kRowLanes;           // rows a warp takes at once
        constexpr int kItems = C::KT / 4 / kStep;       // 4 or 8
        const int c = lane % kRowLanes;
        const int row0 = C::KT / 4 * (warp - 8) + lane / kRowLanes;
        int it = 0;
        bool ok = true;
        Unit w;
        for (Pieces<C> todo; ok && todo.next(share, w);) {
            const int dc = w.m0 + static_cast<int>(rank) * cta_features<C>(D - w.m0);
            const uint32_t sc = static_cast<uint32_t>(((dc / kQ8Block) & 15) + (c >> 2));
            for (int kb = 0; kb < w.nkb; ++kb, ++it) {
                const int s = it % STAGES, raw = it % C::RAW;
                const bool got = role_wait(full0 + 8 * raw, (it / C::RAW) & 1, timeout_ns, fault,
                                           kFaultFullBarrier, abort_flag);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                const uint32_t codes = sbase + C::C_OFF + raw * C::C_BYTES +
                                       (c >> 4) * C::C_BOX_BYTES + 8 * (c & 15);
                const uint32_t exps = sbase + C::S_OFF + raw * C::S_BYTES + sc;
                const uint32_t dst = sbase + s * C::XB_BYTES + (c >> 3) * C::GROUP_BYTES;
                uint32_t q[kItems][2], ex[kItems];
#pragma unroll
                for (int i = 0; i < kItems; ++i) {
                    const uint32_t r = static_cast<uint32_t>(row0 + kStep * i);
                    lds_u32x2(codes + r * 128u, q[i]);
                    ex[i] = lds_u8(exps + 16u * r);
                }
                if (it >= STAGES) {
                    const bool can = role_wait(empty0 + 8 * s, ((it / STAGES) & 1) ^ 1, timeout_ns,
                                               fault, kFaultEmptyBarrier, abort_flag);
                    if (!__all_sync(0xffffffffu, can)) {
                        ok = false;
                        break;
                    }
                }
#pragma unroll
                for (int i = 0; i < kItems; ++i) {
                    const uint32_t r = static_cast<uint32_t>(row0 + kStep * i);
                    uint32_t v[4];
                    const float scale = q8_scale<FMT>(ex[i]);
                    decode_bf16<FMT>(q[i][0], scale, v[0], v[1]);
                    decode_bf16<FMT>(q[i][1], scale, v[2], v[3]);
                    const uint32_t chunk = static_cast<uint32_t>(c & 7) ^ (r & 7u);
                    sts_u32x4(dst + r * 128u + (chunk << 4), v[0], v[1], v[2], v[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(ready0 + 8 * s);
                    mbar_arrive(free0 + 8 * raw);
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------ epilogue (warps 12-19) ------------------------
        regs_inc<C::REGS_EPI>();
        const int e = warp - 12;
        const int q = warp & 3;                  // lanes 32 q .. 32 q + 31
        const int col0 = (e >> 2) * EPI_COLS;    // accumulator columns: features
        const int nl = static_cast<int>(rank) * C::CTA_N + 32 * q + lane;
        const uint32_t acce_leader = PAIR ? map_to_cta(acce, 0) : acce;
        const uint32_t tbase = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                               static_cast<uint32_t>(col0);
        float acc[EPI_COLS];
        int g = 0;
        bool ok = true;
        Unit w;
        for (Pieces<C> todo; ok && todo.next(share, w);) {
#pragma unroll
            for (int i = 0; i < EPI_COLS; ++i) acc[i] = 0.0f;
            for (int c0 = 0; c0 < w.nkb; c0 += chunk, ++g) {
                const bool got = role_wait(accf, g & 1, timeout_ns, fault, kFaultAccumBarrier,
                                           abort_flag);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int j0 = 0; j0 < EPI_COLS / 16; j0 += C::DRAIN_BATCH) {
                    uint32_t r[C::DRAIN_BATCH][16];
#pragma unroll
                    for (int b = 0; b < C::DRAIN_BATCH; ++b)
                        tmem_ld_32x32b_x16(tbase + 16 * (j0 + b), r[b]);
#pragma unroll
                    for (int b = 0; b < C::DRAIN_BATCH; ++b) tmem_ld_wait(r[b]);
#pragma unroll
                    for (int b = 0; b < C::DRAIN_BATCH; ++b) {
                        const int j = j0 + b;
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[16 * j + i] += __uint_as_float(r[b][i]);
                    }
                }
                // the loads have completed: the arrival orders no writes
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR)
                        mbar_arrive_remote(acce_leader);
                    else
                        mbar_arrive(acce);
                }
            }
            if (!ok) break;
            const int n = w.n0 + nl;
            const int rows = D - (w.m0 + col0);
            // Code that runs once a tile is bound by the fetching of its
            // instructions: the usual stores are as few as can be.
            if (n >= N) {
            } else if (w.slot >= 0) {
                float* p = parts + static_cast<long long>(w.slot) * (C::TD * C::TN) +
                           col0 * C::TN + nl;
                store_columns<false>(acc, p, C::TN, rows);
            } else {
                float* p = dw + static_cast<long long>(w.m0 + col0) * lddw + n;
                if (scale_mode == kStorePlain) {
                    store_columns<true>(acc, p, lddw, rows);
                } else {
#pragma unroll
                    for (int j = 0; j < EPI_COLS; ++j, p += lddw)
                        if (j < rows) *p = scale1(acc[j], p, alpha, beta, scale_mode);
                }
            }
        }
        __syncwarp();
    }

    // neither CTA of a pair may leave while the other can still reach its shared
    // or tensor memory
    tc_fence_before();
    if (PAIR)
        cluster_sync();
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if (PAIR)
            tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
        else
            tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

// Shared-memory attribute of the kernel on device `dev`, once (the ABI's
// mutex is held).  The register rebalancing would wait for ever for registers
// that the block was not launched with, so a build in which the compiler took
// fewer than REGS_LAUNCH a thread is refused here.
template <bool PAIR, int FMT, bool SHIFTED>
cudaError_t configure(int dev) {
    using C = WgradCfg<PAIR>;
    constexpr int kDevices = 64;
    static bool done[kDevices] = {};
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, q8_wgrad_kernel<PAIR, FMT, SHIFTED>);
    if (e != cudaSuccess) return e;
    if (attr.numRegs < C::REGS_LAUNCH) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(q8_wgrad_kernel<PAIR, FMT, SHIFTED>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e == cudaSuccess) done[dev] = true;
    return e;
}

template <bool PAIR, int FMT, bool SHIFTED>
cudaError_t launch(const Q8WgradTmemArgs& a, cudaStream_t s, int dev, int sm_count) {
    using C = WgradCfg<PAIR>;
    cudaError_t e = configure<PAIR, FMT, SHIFTED>(dev);
    if (e != cudaSuccess) return e;
    const long long units = static_cast<long long>(a.share.whole) + a.share.runs;
    const int slots = sm_count / C::CTAS;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0] = pdl_attribute();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(C::CTAS * static_cast<int>(units < slots ? units : slots));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, q8_wgrad_kernel<PAIR, FMT, SHIFTED>, a.tmY, a.shifts, a.tmC, a.tmS,
                           a.dw, a.lddw, a.parts, a.cols, a.N, a.rows, a.share, a.chunk, a.fault,
                           a.timeout_ns, a.alpha, a.beta, a.mode);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// The kernel that adds the shared tiles' partial sums.
template <bool PAIR>
cudaError_t launch_sum(const Q8WgradTmemArgs& a, cudaStream_t s) {
    using C = WgradCfg<PAIR>;
    constexpr int kRowsInFlight = 2;
    const bool vec = a.lddw % 4 == 0 && reinterpret_cast<uintptr_t>(a.dw) % 16 == 0;
    // four lanes an output group where a tile has many partials
    const bool quarters = a.share.runs >= 8LL * a.share.shared;
    const int rows = quarters ? 64 / (C::TN / 4) : kRowsInFlight * 256 / (C::TN / 4);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.gridDim = dim3(C::TD / rows, a.share.shared < 65535 ? a.share.shared : 65535);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(
        &cfg,
        quarters ? q8_wgrad_sum_kernel<C, 4, 1, 10> : q8_wgrad_sum_kernel<C, 1, kRowsInFlight, 4>,
        static_cast<const float*>(a.parts), a.share, a.dw, a.lddw, vec, a.cols, a.N, a.alpha,
        a.beta, a.mode);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool PAIR>
cudaError_t launch_form(const Q8WgradTmemArgs& a, cudaStream_t s, int dev, int sm_count) {
    cudaError_t e;
    if (a.format == kQ8Int8)
        e = a.shifted ? launch<PAIR, kQ8Int8, true>(a, s, dev, sm_count)
                      : launch<PAIR, kQ8Int8, false>(a, s, dev, sm_count);
    else
        e = a.shifted ? launch<PAIR, kQ8E4m3, true>(a, s, dev, sm_count)
                      : launch<PAIR, kQ8E4m3, false>(a, s, dev, sm_count);
    if (e != cudaSuccess || !a.share.shared) return e;
    return launch_sum<PAIR>(a, s);
}

}  // namespace

Q8WgradTile q8_wgrad_tile(bool pair) {
    using P = WgradCfg<true>;
    return {P::TD, pair ? P::TN : WgradCfg<false>::TN, P::KT};
}

size_t q8_wgrad_parts_bytes(const Q8WgradShare& sh, bool pair) {
    if (!sh.shared) return 0;
    const Q8WgradTile t = q8_wgrad_tile(pair);
    return (static_cast<size_t>(sh.runs) + sh.shared) * (t.features * t.columns * 4);
}

cudaError_t launch_q8_wgrad_tmem(const Q8WgradTmemArgs& a, cudaStream_t s, int dev, int sm_count) {
    return a.pair ? launch_form<true>(a, s, dev, sm_count) : launch_form<false>(a, s, dev, sm_count);
}

}  // namespace gemm_f32_impl
