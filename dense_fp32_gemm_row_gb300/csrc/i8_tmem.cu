// i8_tmem.cu -- the product of 8-bit integer matrices on the tensor core:
//   acc[t][n] = sum_k a[t][k] b[n][k],  y = acc sa[t] sb[n]
// and the gated product of two of them, h = act(g) u.
//
// Arithmetic.  8-bit integers are exactly fp16 numbers, their products are at
// most 2^14, and sums of up to 1024 of them at most 2^24, so an fp32
// accumulator holds every partial sum of an 896-deep chunk exactly, in whatever
// order the tensor core adds.  Chunks are added up in registers, as floats
// while that is exact and as 32-bit integers beyond it: the sums are exact, and
// the same for any tile, split or kernel.
// (This part's integer MMAs run far below its 16-bit ones, and 8-bit floats
// hold 4 significant bits: an 8-bit integer takes two of them, a product four
// MMAs at twice the rate.)
//
// Shape.  The weights' codes become the MMA's A operand, in tensor memory: a
// thread reads its row of the stage and writes its lane.  The tokens' become B,
// in shared memory, K-major with 128-byte swizzle.  D is the transposed tile,
// lane n, column t, so that a warp stores 32 consecutive channels of a token.
// Conversion is 5 instructions for four codes: a code with its sign bit flipped
// in the low mantissa bits of 1024 is 1152 + code, less 1152.
//
// Three forms.  A cluster of two CTAs computes 256 channels x up to 256 tokens
// with cta_group::2 MMAs, each CTA holding 128 channels in its tensor memory
// and half of the tokens in its shared memory.  Per 16 columns of K an SM's
// tensor core works 128 cycles, and its shared memory moves 4 KB for the weights
// (copy in, read out) and 12 KB for the tokens (copy in, read out, fp16 in,
// MMA): all that it can.  (Both operands in shared memory would take one and a
// half times as long, one CTA with 128 x 256 tiles 1.7 times.)  Or one CTA
// computes 128 x up to 128, or up to 64 with more stages and a third warpgroup
// to convert them, with two accumulators in turn; their tiles may be split over
// K.  The gated form has 16 channels of the gate and the same of up in the lanes
// of a warp, which exchange sums by a shuffle.
//
// 640 threads per CTA, 768 for narrow tiles, registers rebalanced at start
// (launched at 96 or 80 each):
//   warp 0       TMA loads of a 128-column stage of raw codes;
//   warp 1       tensor-memory allocation; in a single CTA or the pair's leader it
//                issues the MMAs and commits;
//   warps 1-2 of a pair's peer  relay: one lane each tells the leader, in turn,
//                that the peer's operands of a stage are written;
//   then 8 (12)  conversion, a warpgroup a stage: weights to fp16 in tensor memory
//                (its warp q: lanes 32 q ..), tokens to fp16 in shared memory;
//   the last 8   per chunk add the accumulator to the sums in their registers
//                (warp e of them: lanes 32 (e % 4) .., half e / 4 of the columns);
//                at the end of a unit scale and store them.
// Splits of a tile are a cluster where the clusters fit the GPU at once: they send
// their sums to its first CTA, when its stages are free, and that adds them up.
// Otherwise they write them to the workspace, and of each warp's part the split
// that comes last, by a counter, adds the others' to its own.  The order makes no
// difference to integers.
// Waits are bounded and wind down as in the GEMM kernels.
//
// What set the speed, 8192 x 8192 x 8192, pairs: chunks' sums converted to
// integers one by one, at 16 a clock and SM, 928 us; added as floats 852; token
// scales loaded past the outputs' stores, which may alias them, 790; stages of
// 128 columns instead of 64, as each role's turn takes some 300 cycles whatever
// a stage holds, 663; the MMA and copy warps whole instead of one lane each, so
// that descriptors are the warp's and not a lane's, 634 to 640: 1720 TFLOP/s, 90
// % of the rate of the library's bf16 product.  Of that the waits for the
// accumulator at the end of each chunk take 65 (without them 573, 1920 TFLOP/s)
// and the peer's relay 23.  One token to a few hundred are bound by the start
// (3.2 us to the first MMA's end and the store of the last tile), then by 0.28 us
// a stage or the weights' way from HBM: 1000 x 1023 x 1025 7.1 us, 64 x 8192 x 8192
// 17.8 (with splits that meet in the workspace 19.1).
#include <cstdint>

#include "device_sync.cuh"
#include "gemm_internal.h"
#include "i8_output.cuh"
#include "tcgen05.cuh"
#include "tf32x3_common.cuh"

namespace gemm_f32_impl {
namespace {

using namespace gemm_f32_dev;

// Stages of K, 128 each, that one accumulator adds up, and the largest sum to
// which another such is added exactly in fp32: 896 products of up to 2^14 are
// 2^24 - 2^21.
constexpr int kStageK = 128;
constexpr int kChunk = 7;
constexpr int kEarlyStages = 3;  // prefetched before the kernel's turn
constexpr float kMostBefore = 16777216.0f - kChunk * kStageK * 16384.0f;

// A pair's CTA, a single one, and a single one for tiles of up to 64 tokens,
// which has room for more stages and a third warpgroup that converts: there the
// weights' way from DRAM is what a stage takes.
enum Form { kPair, kWide, kNarrow };

template <Form FORM>
struct I8Cfg {
    static constexpr bool PAIR = FORM == kPair, NARROW = FORM == kNarrow;
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int LANES = 128;                // rows of weights of a CTA
    static constexpr int TOK = NARROW ? 64 : 128;    // tokens of a CTA, at most
    static constexpr int COLS = TOK * CTAS;          // accumulator columns
    static constexpr int KT = kStageK;               // K a stage
    static constexpr int UK = 16;                    // K an MMA
    static constexpr int RAW = NARROW ? 5 : 3;       // stages of raw codes
    static constexpr int STAGES = NARROW ? 6 : 4;    // stages of MMA operands
    static constexpr int GROUPS = NARROW ? 3 : 2;    // warpgroups that convert, a stage each
    static constexpr int ACCS = PAIR ? 1 : 2;        // accumulators
    static constexpr int B_HALF = TOK * 128;         // tokens in fp16: rows of 64, K halves
    static constexpr int B_BYTES = 2 * B_HALF;
    static constexpr int W_RAW = LANES * KT;
    static constexpr int T_RAW = TOK * KT;
    static constexpr int RAW_BYTES = W_RAW + T_RAW;
    static constexpr int RAW_OFF = STAGES * B_BYTES;
    static constexpr int EPI_WARPS = 8;
    static constexpr int BAR_OFF = RAW_OFF + RAW * RAW_BYTES;
    static constexpr int CONV_WARPS = 4;             // of a stage
    static constexpr int RELAYS = 2;
    // A wait by parity has to come after the end of the barrier's phase before.
    // Each barrier's stages belong to one warpgroup of the conversion and to one
    // relay, which take theirs in order; raw slots, whose number the groups do not
    // divide, have a barrier for each group.
    static constexpr int FULLS = GROUPS * RAW;
    // full, free (raw stages), empty, ready (per operand stage), acc_full and
    // acc_empty (per accumulator), drain, room, joined (per warp of the epilogue)
    static constexpr int NBARS = FULLS + RAW + 2 * STAGES + 2 * ACCS + 2 + EPI_WARPS;
    static constexpr int SMEM_BYTES = BAR_OFF + NBARS * 8 + 16 + 1024;
    static constexpr int EPI_WARP0 = 4 + 4 * GROUPS;
    static constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
    static constexpr int TMEM_COLS = 512;
    static constexpr int OP_COL0 = ACCS * COLS;      // operand stage s at OP_COL0 + 64 s
    static constexpr int OP_COLS = KT / 2;
    static constexpr int EPI_COLS = COLS / 2;        // of a warp, at most
    static constexpr int REGS_LAUNCH = NARROW ? 80 : 96;
    static constexpr int REGS_CONTROL = 32, REGS_CONV = 56, REGS_EPI = NARROW ? 136 : 168;
    // D fp32, A and B fp16, both K-major, M = 128 a CTA; N is added
    static constexpr uint32_t IDESC = (1u << 4) | (static_cast<uint32_t>(LANES * CTAS >> 4) << 24);
    static_assert(REGS_CONTROL + GROUPS * REGS_CONV + EPI_WARPS / 4 * REGS_EPI <=
                      THREADS / 128 * REGS_LAUNCH,
                  "register shares");
    static_assert(OP_COL0 + STAGES * OP_COLS <= TMEM_COLS, "tensor-memory columns");
    static_assert(KT == 128, "two swizzled halves of K");
    static_assert(STAGES % GROUPS == 0 && (!PAIR || RELAYS == GROUPS) && RAW < STAGES,
                  "phases of the barriers");
    static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
    static_assert(EPI_WARPS == kI8CountersPerTile, "counters of a split tile");
};

__device__ __forceinline__ uint4 lds_u32x4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void sts_u32x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                          uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
// Eight words to two neighbouring 16-byte chunks of a swizzled row, the first even.
__device__ __forceinline__ void sts_u32x8(uint32_t addr, const uint32_t (&h)[8]) {
    sts_u32x4(addr, h[0], h[1], h[2], h[3]);
    sts_u32x4(addr ^ 16u, h[4], h[5], h[6], h[7]);
}
// Whether the warp is the last of `all` that call this with one counter, which is
// then 0 again: what the others wrote before their calls is visible to it.
__device__ __forceinline__ bool last_to_come(int* counter, int all) {
    int before = 0;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        asm volatile("fence.acq_rel.gpu;" ::: "memory");
        asm volatile("atom.relaxed.gpu.global.add.s32 %0, [%1], 1;"
                     : "=r"(before)
                     : "l"(counter)
                     : "memory");
        asm volatile("fence.acq_rel.gpu;" ::: "memory");
        if (before == all - 1)
            asm volatile("st.relaxed.gpu.global.s32 [%0], 0;" ::"l"(counter) : "memory");
    }
    __syncwarp();
    return __shfl_sync(0xffffffffu, before, 0) == all - 1;
}

// Sums to another CTA of the cluster, counted by its barrier there.
__device__ __forceinline__ void send_f32x4(uint32_t to, uint32_t bar, const float* v) {
    asm volatile(
        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, "
        "[%5];" ::"r"(to),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"(bar)
        : "memory");
}

// Offset of a 16-byte chunk: rows of 128 bytes, 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t chunk) {
    return row * 128u + ((chunk ^ (row & 7u)) << 4);
}

// A scale, which the kernel before may have written: not before the wait for that
// kernel, and apart from that whenever it suits, past stores that it cannot alias.
__device__ __forceinline__ float load_scale(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// One unit of work: a split of a tile.
struct Work {
    int tile, c0, t0;        // its first channel and token
    int kb_begin, nkb;       // stages
};
template <bool PAIR, bool GATED>
__device__ __forceinline__ bool work_at(const I8Share& sh, int u, Work& w) {
    if (u >= sh.tiles_c * sh.tiles_t * sh.splits) return false;
    w.tile = u / sh.splits;
    const int split = u - w.tile * sh.splits;
    w.kb_begin = static_cast<int>(static_cast<long long>(sh.stages) * split / sh.splits);
    w.nkb = static_cast<int>(static_cast<long long>(sh.stages) * (split + 1) / sh.splits) - w.kb_begin;
    // neighbouring tiles run down groups of 8 rows of tiles, so that the CTAs at
    // work share operands in L2
    const int per_group = GROUP_M * sh.tiles_t;
    const int group = w.tile / per_group, within = w.tile - group * per_group;
    const int rows = min(sh.tiles_c - group * GROUP_M, GROUP_M);
    const int column = within / rows;
    w.c0 = (group * GROUP_M + within - column * rows) * (128 * (PAIR ? 2 : 1) / (GATED ? 2 : 1));
    w.t0 = column * sh.tokens * (PAIR ? 2 : 1);
    return true;
}

// Tokens that each CTA holds of a tile with `left` tokens from its first to the
// last: all of them, or in the last tiles as few groups of 16 as cover the rest,
// so that the MMAs are no wider than they need to be.
template <bool PAIR>
__device__ __forceinline__ int cta_tokens(int tokens, int left) {
    const int each = PAIR ? (left + 1) / 2 : left;
    return min(tokens, (each + 15) & ~15);
}

__device__ __forceinline__ void add_pair(float& a, float& b, uint32_t x, uint32_t y) {
    asm("{\n\t.reg .b64 s, t;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 t, {%2, %3};\n\t"
        "add.rn.f32x2 s, s, t;\n\tmov.b64 {%0, %1}, s;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(x), "r"(y));
}

// Adds an accumulator's columns to acc, which holds floats or (`whole`) 32-bit
// integers; loaded() once it has been read.
template <int COLS, typename F>
__device__ __forceinline__ void add_columns(float (&acc)[COLS], uint32_t tbase, int count,
                                            bool whole, F loaded) {
    if (whole) {
#pragma unroll
        for (int j = 0; j < COLS; j += 16) {
            if (j >= count) break;
            uint32_t r[16];
            tmem_ld_32x32b_x16(tbase + j, r);
            tmem_ld_wait(r);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[j + i] = __int_as_float(__float_as_int(acc[j + i]) +
                                            __float2int_rn(__uint_as_float(r[i])));
        }
        loaded();
        return;
    }
    if (count <= 0) loaded();
#pragma unroll
    for (int j = 0; j < COLS; j += 32) {
        if (j >= count) break;
        uint32_t r[2][16];
        tmem_ld_32x32b_x16(tbase + j, r[0]);
        tmem_ld_32x32b_x16(tbase + j + 16, r[1]);
        tmem_ld_wait(r[0]);
        tmem_ld_wait(r[1]);
        if (j + 32 >= count) loaded();
#pragma unroll
        for (int i = 0; i < 32; i += 2)
            add_pair(acc[j + i], acc[j + i + 1], r[i / 16][i % 16], r[i / 16][i % 16 + 1]);
    }
}

// To 32-bit integers, unless another accumulator can be added to each sum of
// the warp exactly.  (Conversions run at an eighth of the rate of additions:
// with every chunk converted 8192 x 8192 x 8192 took 928 us.)
template <int COLS>
__device__ __forceinline__ void keep_exact(float (&acc)[COLS], bool& whole) {
    if (whole) return;
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < COLS; ++i) most = fmaxf(most, fabsf(acc[i]));
    if (!__any_sync(0xffffffffu, most > kMostBefore)) return;
    whole = true;
#pragma unroll
    for (int i = 0; i < COLS; ++i) acc[i] = __int_as_float(__float2int_rn(acc[i]));
}

// The scale of column j from registers that hold 32 a time, lane by lane.
template <int N>
__device__ __forceinline__ float scale_of(const float (&token)[N], int j) {
    return __shfl_sync(0xffffffffu, token[j / 32], j % 32);
}

// value(j) to p + j ld for the first `left` columns of `count`, in groups of 16
// without a branch among them: acc stays in registers, and the columns' loads,
// shuffles and stores overlap.
template <int COLS, typename T, typename F>
__device__ __forceinline__ void put_columns(const float (&acc)[COLS], int count, int left, T* p,
                                            long long ld, F value) {
#pragma unroll
    for (int j = 0; j < COLS; j += 16) {
        if (j >= count) break;
        T v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = value(j + i);
#pragma unroll
        for (int i = 0; i < 16; ++i, p += ld)
            if (j + i < left) *p = v[i];
    }
}

__device__ __forceinline__ void put_float(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_float(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The gated product of a warp whose lanes 0 .. 15 hold the gate's sums of 16
// channels and lanes 16 .. 31 up's: of each two tokens the lower lanes finish the
// first and the upper the second.
template <int COLS, int ACT, typename T>
__device__ __forceinline__ void put_gated(const float (&acc)[COLS], const float (&token)[COLS / 32],
                                          float channel, float channel_up, int count, int left,
                                          T* p, long long ld) {
    const int upper = (threadIdx.x >> 4) & 1;
    p += upper * ld;
    left -= upper;
#pragma unroll
    for (int j = 0; j < COLS; j += 16) {
        if (j >= count) break;
        float h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = j + 2 * i;
            const float st = __shfl_sync(0xffffffffu, token[k / 32], k % 32 + upper);
            const float own = upper ? acc[k + 1] : acc[k];
            const float other = __shfl_xor_sync(0xffffffffu, upper ? acc[k] : acc[k + 1], 16);
            const float gate = i8_value(upper ? other : own, st, channel);
            const float up = i8_value(upper ? own : other, st, channel_up);
            h[i] = i8_act<ACT>(gate) * up;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i, p += 2 * ld)
            if (j + 2 * i < left) put_float(p, h[i]);
    }
}

template <Form FORM, int ACT>
__global__ void __launch_bounds__(I8Cfg<FORM>::THREADS, 1)
i8_tmem_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmC, I8TmemArgs p) {
    using C = I8Cfg<FORM>;
    constexpr bool PAIR = C::PAIR;
    constexpr bool GATED = ACT != kI8NoAct;
    constexpr int STAGES = C::STAGES;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_addr(smem);
    const uint32_t full0 = sbase + C::BAR_OFF;      // own: a raw stage has landed
    const uint32_t free0 = full0 + 8 * C::FULLS;    // own: its readers are done
    const uint32_t empty0 = free0 + 8 * C::RAW;     // own, multicast commit: operands read
    const uint32_t ready0 = empty0 + 8 * STAGES;    // operands written
    const uint32_t accf = ready0 + 8 * STAGES;      // own, multicast commit
    const uint32_t acce = accf + 8 * C::ACCS;       // leader: 8 warps a CTA
    const uint32_t drain = acce + 8 * C::ACCS;
    const uint32_t room0 = drain + 8;               // a cluster's others: its first has room
    const uint32_t joined0 = room0 + 8;             // its first: the others' sums, a warp's
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::BAR_OFF + C::NBARS * 8);
    const uint32_t abort_flag = smem_addr(tmem_slot + 1);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
    const bool cluster = PAIR || p.share.clusters;
    const int first = blockIdx.x / C::CTAS, step = gridDim.x / C::CTAS;
    const long long timeout_ns = p.timeout_ns;
    unsigned* const fault = p.fault;
    const I8Share& share = p.share;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        if (GATED) prefetch_tmap(&tmC);
        for (int r = 0; r < C::FULLS; ++r) mbar_init(full0 + 8 * r, 1);
        for (int r = 0; r < C::RAW; ++r) mbar_init(free0 + 8 * r, C::CONV_WARPS);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(empty0 + 8 * s, 1);
            // in the leader also the relay of the peer's
            mbar_init(ready0 + 8 * s, C::CONV_WARPS + (PAIR && rank == 0 ? 1 : 0));
        }
        for (int a = 0; a < C::ACCS; ++a) {
            mbar_init(accf + 8 * a, 1);
            mbar_init(acce + 8 * a, C::CTAS * C::EPI_WARPS);
        }
        mbar_init(drain, 1);
        mbar_init(room0, 1);
        for (int e = 0; e < C::EPI_WARPS; ++e) mbar_init(joined0 + 8 * e, 1);
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
    if (cluster)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // While the kernel before ends, the weights' way to L2 is begun, which reads
    // no value: 24 x 8192 x 8192 17.5 to 16.7 us, 64 x 4096 x 4096 11.2 to 10.6.
    // (One stage 17.1, six 17.0; by all tiles of tokens nothing more.)
    if (!PAIR && warp == 3 && elect_lane()) {
        Work w;
        if (work_at<PAIR, GATED>(share, first, w) && w.t0 == 0)
            for (int kb = w.kb_begin; kb < w.kb_begin + min(w.nkb, kEarlyStages); ++kb) {
                tma_prefetch_2d(&tmB, kb * C::KT, w.c0);
                if (GATED) tma_prefetch_2d(&tmC, kb * C::KT, w.c0);
            }
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();

    // The peer's arrivals on its ready barriers, passed on to the leader's: relay
    // i of RELAYS takes every RELAYS-th stage (a release at cluster scope takes
    // ~650 ns, more than the MMAs of a stage).
    auto relay = [&](int i) {
        const uint32_t ready_leader = map_to_cta(ready0, 0);
        int total = 0;
        Work w;
        for (int u = first; work_at<PAIR, GATED>(share, u, w); u += step) total += w.nkb;
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
            // ------------------------------ TMA producer ------------------------------
            const bool elected = elect_lane();
            int it = 0;
            int r = 0, f = 0;  // raw slot and its phase, barrier
            uint32_t r_phase = 1;
            bool ok = true;
            Work w;
            const uint32_t bytes = C::W_RAW + static_cast<uint32_t>(share.tokens * C::KT);
            for (int u = first; ok && work_at<PAIR, GATED>(share, u, w); u += step) {
                const int tok0 = w.t0 + rank * cta_tokens<PAIR>(share.tokens, p.T - w.t0);
                const int ch0 = w.c0 + rank * (GATED ? C::LANES / 2 : C::LANES);
                int k0 = w.kb_begin * C::KT;
                for (int kb = 0; kb < w.nkb; ++kb, ++it, k0 += C::KT) {
                    if (it >= C::RAW &&
                        !__all_sync(0xffffffffu,
                                    role_wait(free0 + 8 * r, r_phase, timeout_ns, fault,
                                              kFaultEmptyBarrier, abort_flag))) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full0 + 8 * f;
                    const uint32_t wb = sbase + C::RAW_OFF + r * C::RAW_BYTES;
                    if (elected) {
                        mbar_arrive_expect_tx(fb, bytes);
                        tma_load_2d(wb, &tmB, fb, k0, ch0);
                        if (GATED) tma_load_2d(wb + C::W_RAW / 2, &tmC, fb, k0, ch0);
                        tma_load_2d(wb + C::W_RAW, &tmA, fb, k0, tok0);
                    }
                    if (++f == C::FULLS) f = 0;
                    if (++r == C::RAW) {
                        r = 0;
                        r_phase ^= 1;
                    }
                }
            }
            // wind down: this CTA's copies have landed, and the MMAs' commits have
            // reached its operand stages
            if (elected) {
                const long long tail = ok ? timeout_ns : timeout_ns / 8 + 1000;
                for (int j = (it > C::RAW ? it - C::RAW : 0); j < it; ++j)
                    mbar_wait(full0 + 8 * (j % C::FULLS), (j / C::FULLS) & 1, tail, fault,
                              kFaultDrain);
                for (int j = (it > STAGES ? it - STAGES : 0); j < it; ++j)
                    mbar_wait(empty0 + 8 * (j % STAGES), (j / STAGES) & 1, tail, fault, kFaultDrain);
            }
            __syncwarp();
        } else if (warp == 1) {
            if (rank == 0) {
                // -------------------------- MMA issuer (of a pair: the leader) --------
                // The whole warp waits, so that descriptors and addresses are the warp's
                // and not a lane's; one lane issues.
                const bool elected = elect_lane();
                int s = 0;            // operand stage, and its phase
                uint32_t phase = 0;
                int g = 0;            // chunks issued
                bool ok = true;
                Work w;
                const uint64_t x0 = smem_desc_sw128_kmajor(sbase);
                for (int u = first; ok && work_at<PAIR, GATED>(share, u, w); u += step) {
                    const uint32_t idesc =
                        C::IDESC | static_cast<uint32_t>(
                                       C::CTAS * cta_tokens<PAIR>(share.tokens, p.T - w.t0) / 8)
                                       << 17;
                    for (int c0 = 0; c0 < w.nkb && ok; c0 += kChunk, ++g) {
                        const int b = g % C::ACCS;
                        // the accumulator: its last chunk has been drained
                        if (g >= C::ACCS &&
                            !__all_sync(0xffffffffu,
                                        role_wait(acce + 8 * b, ((g / C::ACCS) - 1) & 1, timeout_ns,
                                                  fault, kFaultAccumBarrier, abort_flag))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tmem_base + static_cast<uint32_t>(b * C::COLS);
                        const int c1 = min(w.nkb, c0 + kChunk);
                        for (int kb = c0; kb < c1; ++kb) {
                            if (!__all_sync(0xffffffffu,
                                            role_wait<PAIR>(ready0 + 8 * s, phase, timeout_ns, fault,
                                                            kFaultFullBarrier, abort_flag))) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint64_t x = x0 + static_cast<uint64_t>(s * (C::B_BYTES >> 4));
                            const uint32_t a =
                                tmem_base + static_cast<uint32_t>(C::OP_COL0 + C::OP_COLS * s);
                            if (elected) {
#pragma unroll
                                for (int k = 0; k < C::KT / C::UK; ++k)
                                    // 16 columns of K: 32 bytes of a row, 8 columns of tensor
                                    // memory
                                    mma_f16_tmem_a<PAIR>(
                                        d, a + 8u * k,
                                        x + (k / 4) * (C::B_HALF >> 4) + 2u * (k % 4), idesc,
                                        (kb > c0 || k > 0) ? 1u : 0u);
                                mma_commit_form<PAIR>(empty0 + 8 * s);
                            }
                            if (++s == STAGES) {
                                s = 0;
                                phase ^= 1;
                            }
                        }
                        if (!ok) break;
                        if (elected) mma_commit_form<PAIR>(accf + 8 * b);
                    }
                }
                if (elected) {
                    if (PAIR)
                        mma_commit_pair(drain);
                    else
                        mma_commit(drain);
                    if (!mbar_wait(drain, 0, ok ? timeout_ns : timeout_ns / 8 + 1000, fault,
                                   kFaultDrain))
                        ok = false;
                }
                ok = __all_sync(0xffffffffu, ok);
                // The first CTA of a cluster: its MMAs are done, and with them (its operands
                // were ready) its copies and their conversion: its stages are free.  The
                // release is at cluster scope, as the others' sums overwrite what this CTA's
                // threads wrote and read there; it takes long, but not on the epilogue's path.
                if (!PAIR && share.clusters && ok && lane > 0 && lane < share.splits &&
                    cluster_ctarank() == 0)
                    mbar_arrive_cluster(map_to_cta(room0, lane));
                __syncwarp();
            } else if (PAIR && lane == 0) {
                relay(0);
            }
            __syncwarp();
        } else if (PAIR && rank == 1 && warp == 2 && lane == 0) {
            // ------------------------------ the other relay ---------------------------
            relay(1);
        }
        __syncwarp();
    } else if (warp < C::EPI_WARP0) {
        // ------------------------------ conversion -------------------------------------
        // A warpgroup takes every second or third stage, a half of K at a time.  Weights: a
        // thread has its lane's row (gated: 16 of a warp's lanes the gate's, 16
        // up's).  Tokens: a lane takes 16 codes; each eight lanes load from two rows
        // whose numbers differ in bits 0 and 2, so that both the codes and the two
        // chunks that they store lie in all banks.
        regs_dec<C::REGS_CONV>();
        constexpr int kItems = C::TOK / 8 / 4;
        constexpr uint32_t kItemBytes = 32 * 128;
        const int q = warp & 3;
        const uint32_t row = static_cast<uint32_t>(
            !GATED ? 32 * q + lane : (lane < 16 ? 0 : C::LANES / 2) + 16 * q + (lane & 15));
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
        const uint32_t c = static_cast<uint32_t>(lane & 3);
        const uint32_t row0 =
            static_cast<uint32_t>(8 * q + ((lane >> 3) ^ ((lane & 4) ? 5 : 0)));
        const uint32_t weights_at = swizzled(row, 0);  // of the first chunk
        const uint32_t tokens_at = swizzled(row0, c), fp16_at = swizzled(row0, 2u * c);
        const int group = (warp >> 2) - 1;
        // its next stage of all, operand stage and raw slot and barrier, with phases
        int it = group, s = group, raw = group % C::RAW, f = group;
        uint32_t s_phase = 1, f_phase = 0;
        int base = 0;
        bool ok = true;
        Work w;
        for (int u = first; ok && work_at<PAIR, GATED>(share, u, w); base += w.nkb, u += step) {
            const int rows = cta_tokens<PAIR>(share.tokens, p.T - w.t0);
            const int items = (rows - 8 * q + 31) / 32;  // of this warp: 8 rows each
            for (; it < base + w.nkb; it += C::GROUPS) {
                const bool got = role_wait(full0 + 8 * f, f_phase, timeout_ns, fault,
                                           kFaultFullBarrier, abort_flag);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                // chunk c of a row of 128 bytes lies at (c << 4) ^ (row % 8 << 4) in it
                const uint32_t src = sbase + C::RAW_OFF + raw * C::RAW_BYTES;
                const uint32_t from_w = src + weights_at, from_x = src + C::W_RAW + tokens_at;
                const uint32_t to_x = sbase + s * C::B_BYTES + fp16_at;
                const uint32_t col =
                    lane_base + static_cast<uint32_t>(C::OP_COL0 + C::OP_COLS * s);
                uint4 v[4], x[kItems];
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) v[i] = lds_u32x4(from_w ^ (i << 4));
#pragma unroll
                for (int i = 0; i < kItems; ++i)
                    if (items == kItems) x[i] = lds_u32x4(from_x + kItemBytes * i);
                if (it >= STAGES) {
                    const bool can = role_wait(empty0 + 8 * s, s_phase, timeout_ns, fault,
                                               kFaultEmptyBarrier, abort_flag);
                    if (!__all_sync(0xffffffffu, can)) {
                        ok = false;
                        break;
                    }
                }
                // the MMAs that read this stage before are done
                tc_fence_after();
                // the second half's codes are loaded as the first's are converted
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) {
                    uint32_t h[8];
                    decode_f16(v[i], h);
                    v[i] = lds_u32x4(from_w ^ ((i + 4u) << 4));
                    tmem_st_32x32b_x8(col + 8u * i, h);
                }
                if (items == kItems) {
#pragma unroll
                    for (int i = 0; i < kItems; ++i) {
                        uint32_t h[8];
                        decode_f16(x[i], h);
                        x[i] = lds_u32x4((from_x ^ 64u) + kItemBytes * i);
                        sts_u32x8(to_x + kItemBytes * i, h);
                    }
                } else {
                    for (int i = 0; i < items; ++i) {
                        uint32_t h[8];
                        decode_f16(lds_u32x4(from_x + kItemBytes * i), h);
                        sts_u32x8(to_x + kItemBytes * i, h);
                        decode_f16(lds_u32x4((from_x ^ 64u) + kItemBytes * i), h);
                        sts_u32x8(to_x + C::B_HALF + kItemBytes * i, h);
                    }
                }
                // every code has been read
                __syncwarp();
                if (lane == 0) mbar_arrive(free0 + 8 * raw);
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) {
                    uint32_t h[8];
                    decode_f16(v[i], h);
                    tmem_st_32x32b_x8(col + 32u + 8u * i, h);
                }
                if (items == kItems) {
#pragma unroll
                    for (int i = 0; i < kItems; ++i) {
                        uint32_t h[8];
                        decode_f16(x[i], h);
                        sts_u32x8(to_x + C::B_HALF + kItemBytes * i, h);
                    }
                }
                fence_proxy_async_smem();
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ready0 + 8 * s);
                if ((s += C::GROUPS) >= STAGES) {
                    s -= STAGES;
                    s_phase ^= 1;
                }
                if ((f += C::GROUPS) >= C::FULLS) {
                    f -= C::FULLS;
                    f_phase ^= 1;
                }
                raw = (raw + C::GROUPS) % C::RAW;
            }
        }
        __syncwarp();
    } else {
        // ------------------------------ epilogue ---------------------------------------
        // Every warp walks through all units whatever happens, so that the counters of
        // split tiles come round to 0.
        regs_inc<C::REGS_EPI>();
        const int e = warp - C::EPI_WARP0;
        const int q = warp & 3;                  // lanes 32 q .. 32 q + 31
        const int half = e >> 2;
        const int n_lane = GATED ? rank * (C::LANES / 2) + 16 * q + (lane & 15)
                                 : rank * C::LANES + 32 * q + lane;
        const uint32_t acce_leader = PAIR ? map_to_cta(acce, 0) : acce;
        float acc[C::EPI_COLS];
        int g = 0;
        bool ok = true;
        Work w;
        for (int u = first; work_at<PAIR, GATED>(share, u, w); u += step) {
            const int cols = C::CTAS * cta_tokens<PAIR>(share.tokens, p.T - w.t0);
            const int each = (cols + 31) / 32 * 16;
            const int col0 = half * each;
            const int count = min(each, cols - col0);  // of this warp: groups of 16, or none
#pragma unroll
            for (int i = 0; i < C::EPI_COLS; ++i) acc[i] = 0.0f;
            bool whole = false;  // acc holds 32-bit integers
            // the tokens' scales, 32 of them lane by lane, long before their use
            float token[C::EPI_COLS / 32];
#pragma unroll
            for (int i = 0; i < C::EPI_COLS / 32; ++i) {
                // (of tokens that there are not the last one's, which nothing uses)
                token[i] = load_scale(p.as + min(w.t0 + col0 + 32 * i + lane, p.T - 1));
            }
            for (int c0 = 0; ok && c0 < w.nkb; c0 += kChunk, ++g) {
                const int b = g % C::ACCS;
                const bool got = role_wait(accf + 8 * b, (g / C::ACCS) & 1, timeout_ns, fault,
                                           kFaultAccumBarrier, abort_flag);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tbase = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                       static_cast<uint32_t>(b * C::COLS + col0);
                add_columns<C::EPI_COLS>(acc, tbase, count, whole, [&] {
                    // the loads have completed: the arrival orders no writes
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR)
                            mbar_arrive_remote(acce_leader + 8 * b);
                        else
                            mbar_arrive(acce + 8 * b);
                    }
                });
                // off the MMAs' path
                if (c0 + kChunk < w.nkb) keep_exact<C::EPI_COLS>(acc, whole);
            }
            if (!PAIR && share.splits > 1) {
                if (count <= 0) continue;
                if (!whole)
#pragma unroll
                    for (int j = 0; j < C::EPI_COLS; ++j)
                        acc[j] = __int_as_float(__float2int_rn(acc[j]));
                whole = true;
                // a warp's lanes' sums of four columns lie side by side
                const uint32_t slice = static_cast<uint32_t>(col0 * C::LANES + q * count * 32) * 4u +
                                       16u * static_cast<uint32_t>(lane);
                const uint32_t part = static_cast<uint32_t>(share.tokens) * (4u * C::LANES);
                if (share.clusters) {
                    const int split = u - w.tile * share.splits;
                    if (!ok) continue;
                    if (split == 0) {
                        if (lane == 0)
                            mbar_arrive_expect_tx(joined0 + 8 * e,
                                                  (share.splits - 1) * count * (4 * 32));
                        const bool got = role_wait<true>(joined0 + 8 * e, 0, timeout_ns, fault,
                                                         kFaultAccumBarrier, abort_flag);
                        ok = __all_sync(0xffffffffu, got);
                        for (int s = 0; ok && s < share.splits - 1; ++s) {
#pragma unroll
                            for (int j = 0; j < C::EPI_COLS; j += 4) {
                                if (j % 16 == 0 && j >= count) break;
                                const uint4 more = lds_u32x4(sbase + s * part + slice + j * 128);
                                const uint32_t m[4] = {more.x, more.y, more.z, more.w};
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    acc[j + i] = __int_as_float(__float_as_int(acc[j + i]) +
                                                                static_cast<int>(m[i]));
                            }
                        }
                    } else {
                        const bool got = role_wait<true>(room0, 0, timeout_ns, fault,
                                                         kFaultAccumBarrier, abort_flag);
                        if (!__all_sync(0xffffffffu, got)) continue;
                        const uint32_t to = map_to_cta(sbase + (split - 1) * part + slice, 0);
                        const uint32_t bar = map_to_cta(joined0 + 8 * e, 0);
#pragma unroll
                        for (int j = 0; j < C::EPI_COLS; j += 4) {
                            if (j % 16 == 0 && j >= count) break;
                            send_f32x4(to + j * 128, bar, acc + j);
                        }
                        continue;
                    }
                } else {
                    const long long slot = static_cast<long long>(share.tokens) * C::LANES;
                    int* const mine = p.parts + u * slot + col0 * C::LANES + 32 * q + lane;
#pragma unroll
                    for (int j = 0; j < C::EPI_COLS; j += 16) {
                        if (j >= count) break;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            __stcg(mine + (j + i) * C::LANES, __float_as_int(acc[j + i]));
                    }
                    if (!last_to_come(p.counters + C::EPI_WARPS * w.tile + e, share.splits)) continue;
                    const int* const all = p.parts + w.tile * share.splits * slot + col0 * C::LANES +
                                           32 * q + lane;
                    for (int s = 0; s < share.splits; ++s) {
                        if (w.tile * share.splits + s == u) continue;
#pragma unroll
                        for (int j = 0; j < C::EPI_COLS; j += 16) {
                            if (j >= count) break;
                            int more[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                more[i] = __ldcg(all + s * slot + (j + i) * C::LANES);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                acc[j + i] = __int_as_float(__float_as_int(acc[j + i]) + more[i]);
                        }
                    }
                }
            }
            // from here the sums as floats, or as the integers they are
            const bool integers = !GATED && p.type == kI8Int32;
            if (whole && !integers) {
#pragma unroll
                for (int j = 0; j < C::EPI_COLS; ++j)
                    acc[j] = __int2float_rn(__float_as_int(acc[j]));
            } else if (!whole && integers) {
#pragma unroll
                for (int j = 0; j < C::EPI_COLS; ++j)
                    acc[j] = __int_as_float(__float2int_rn(acc[j]));
            }
            const int n = w.c0 + n_lane;
            const bool mine = ok && n < p.N;
            const float channel = load_scale(p.bs + min(n, p.N - 1));
            const int t_first = w.t0 + col0;
            if (GATED) {
                const float channel_up = load_scale(p.cs + min(n, p.N - 1));
                const int left = mine ? min(count, p.T - t_first) : 0;
                const long long at = static_cast<long long>(t_first) * p.ldy + n;
                if (p.type == kI8Bfloat16)
                    put_gated<C::EPI_COLS, ACT>(acc, token, channel, channel_up, count, left,
                                                static_cast<__nv_bfloat16*>(p.y) + at, p.ldy);
                else
                    put_gated<C::EPI_COLS, ACT>(acc, token, channel, channel_up, count, left,
                                                static_cast<float*>(p.y) + at, p.ldy);
            } else {
                const int left = mine ? min(count, p.T - t_first) : 0;
                const long long at = static_cast<long long>(t_first) * p.ldy + n;
                if (p.type == kI8Int32)
                    put_columns<C::EPI_COLS>(acc, count, left, static_cast<int*>(p.y) + at, p.ldy,
                                             [&](int j) { return __float_as_int(acc[j]); });
                else if (p.type == kI8Bfloat16)
                    put_columns<C::EPI_COLS>(
                        acc, count, left, static_cast<__nv_bfloat16*>(p.y) + at, p.ldy, [&](int j) {
                            return __float2bfloat16_rn(
                                i8_value(acc[j], scale_of(token, j), channel));
                        });
                else
                    put_columns<C::EPI_COLS>(
                        acc, count, left, static_cast<float*>(p.y) + at, p.ldy,
                        [&](int j) { return i8_value(acc[j], scale_of(token, j), channel); });
            }
        }
        __syncwarp();
    }

    // no CTA of a cluster may leave while another can still reach its shared or
    // tensor memory
    tc_fence_before();
    if (cluster)
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
template <Form FORM, int ACT>
cudaError_t configure(int dev) {
    using C = I8Cfg<FORM>;
    constexpr int kDevices = 64;
    static bool done[kDevices] = {};
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, i8_tmem_kernel<FORM, ACT>);
    if (e != cudaSuccess) return e;
    if (attr.numRegs < C::REGS_LAUNCH) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(i8_tmem_kernel<FORM, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM_BYTES);
    if (e == cudaSuccess) done[dev] = true;
    return e;
}

template <Form FORM, int ACT>
cudaError_t launch(const I8TmemMaps& maps, const I8TmemArgs& a, cudaStream_t s, int dev,
                   int sm_count) {
    using C = I8Cfg<FORM>;
    cudaError_t e = configure<FORM, ACT>(dev);
    if (e != cudaSuccess) return e;
    const long long units =
        static_cast<long long>(a.share.tiles_c) * a.share.tiles_t * a.share.splits;
    const int slots = sm_count / C::CTAS;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0] = pdl_attribute();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C::PAIR ? 2 : a.share.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(C::CTAS * static_cast<int>(units < slots ? units : slots));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = C::PAIR || a.share.clusters ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, i8_tmem_kernel<FORM, ACT>, maps.a, maps.b, maps.c, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int ACT>
cudaError_t launch_form(const I8TmemMaps& maps, const I8TmemArgs& a, bool pair, cudaStream_t s,
                        int dev, int sm_count) {
    if (pair) return launch<kPair, ACT>(maps, a, s, dev, sm_count);
    return a.share.tokens <= I8Cfg<kNarrow>::TOK ? launch<kNarrow, ACT>(maps, a, s, dev, sm_count)
                                                 : launch<kWide, ACT>(maps, a, s, dev, sm_count);
}

}  // namespace

bool i8_joins_in_clusters(int splits, int tokens) {
    using W = I8Cfg<kWide>;
    using N = I8Cfg<kNarrow>;
    const int room = tokens <= N::TOK ? N::BAR_OFF : W::BAR_OFF;
    return splits > 1 && splits <= 8 && (splits - 1) * tokens * (4 * W::LANES) <= room;
}

int i8_most_clusters(int splits, int dev) {
    constexpr int kDevices = 64;
    static int known[kDevices][9] = {};  // and 1
    if (dev < 0 || dev >= kDevices || splits < 2 || splits > 8) return 0;
    int& n = known[dev][splits];
    if (!n) {
        using C = I8Cfg<kNarrow>;
        if (configure<kNarrow, kI8NoAct>(dev) != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = splits;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(splits);
        cfg.blockDim = dim3(C::THREADS);
        cfg.dynamicSmemBytes = C::SMEM_BYTES;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, i8_tmem_kernel<kNarrow, kI8NoAct>, &cfg) !=
            cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        n = clusters + 1;
    }
    return n - 1;
}

I8Tile i8_tile(bool pair) {
    using P = I8Cfg<kPair>;
    return {pair ? 2 * P::LANES : P::LANES, P::TOK, P::KT};
}

size_t i8_parts_bytes(const I8Share& s) {
    if (s.splits < 2 || s.clusters) return 0;
    return static_cast<size_t>(s.tiles_c) * s.tiles_t * s.splits * s.tokens * I8Cfg<kWide>::LANES * 4;
}

cudaError_t launch_i8_tmem(const I8TmemMaps& maps, const I8TmemArgs& a, bool pair, int act,
                           cudaStream_t s, int dev, int sm_count) {
    if (act == kActSilu) return launch_form<kActSilu>(maps, a, pair, s, dev, sm_count);
    if (act == kActGelu) return launch_form<kActGelu>(maps, a, pair, s, dev, sm_count);
    return launch_form<kI8NoAct>(maps, a, pair, s, dev, sm_count);
}

}  // namespace gemm_f32_impl
