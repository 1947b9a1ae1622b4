// i8_tmem.cu -- the product of 8-bit integer matrices on the tensor core:
//   acc[t][n] = sum_k a[t][k] b[n][k],  y = acc sa[t] sb[n]
// and the gated product of two of them, h = act(g) u.
//
// Arithmetic.  8-bit integers are exactly fp16 numbers, their products are at
// most 2^14, and sums of up to 1024 of them at most 2^24, so an fp32
// accumulator holds every partial sum of a 1024-deep chunk exactly, in
// whatever order the tensor core adds.  Chunks are added up in 32-bit integer
// registers: the sums are exact, and the same for any tile, split or kernel.
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
// Two forms.  A cluster of two CTAs computes 256 channels x up to 256 tokens
// with cta_group::2 MMAs, each CTA holding 128 channels in its tensor memory
// and half of the tokens in its shared memory: per 16 columns of K an SM's
// tensor core works 128 cycles, and its shared memory moves 4 KB for the
// weights (copy in, read out) and 12 KB for the tokens (copy in, read out, fp16
// in, MMA).  Or one CTA computes 128 x up to 128, with two accumulators in
// turn, its tiles split over K for few tokens.  The gated form has gate and up
// channels in the two halves of a CTA's lanes, 64 each, and the warps of one
// half exchange values with those of the other through shared memory.
//
// 640 threads per CTA, registers rebalanced at start (launched at 96 each):
//   warp 0       one lane: TMA loads of a 64-column stage of raw codes;
//   warp 1       tensor-memory allocation; one lane (of a pair: the leader's)
//                issues the MMAs and commits;
//   warps 1-3 of a pair's peer  relay: one lane each tells the leader, in turn,
//                that the peer's operands of a stage are written;
//   warps 4-7    weights to fp16 in tensor memory (warp 4 + q: lanes 32 q ..);
//   warps 8-11   tokens to fp16 in shared memory;
//   warps 12-19  per chunk add the accumulator to 32-bit integers in registers
//                (warp 12 + e: lanes 32 (e % 4) .., half e / 4 of the columns);
//                at the end of a unit scale and store them.
// Splits of a tile write their sums to the workspace, and the one that comes
// last, by a counter a tile, adds the others' to its own: nothing waits, and
// the order makes no difference to integers.
// Waits are bounded and wind down as in the GEMM kernels.
#include <cstdint>

#include "device_sync.cuh"
#include "gemm_internal.h"
#include "i8_output.cuh"
#include "tcgen05.cuh"
#include "tf32x3_common.cuh"

namespace gemm_f32_impl {
namespace {

using namespace gemm_f32_dev;

constexpr int kNoAct = -1;

template <bool PAIR_>
struct I8Cfg {
    static constexpr bool PAIR = PAIR_;
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int LANES = 128;                // rows of weights of a CTA
    static constexpr int TOK = 128;                  // tokens of a CTA, at most
    static constexpr int COLS = TOK * CTAS;          // accumulator columns
    static constexpr int KT = 64;                    // K a stage
    static constexpr int UK = 16;                    // K an MMA
    static constexpr int CHUNK = 1024 / KT;          // stages of an exact fp32 sum
    static constexpr int RAW = 6;                    // stages of raw codes
    static constexpr int STAGES = 7;                 // stages of MMA operands
    static constexpr int ACCS = PAIR ? 1 : 2;        // accumulators
    static constexpr int B_BYTES = TOK * KT * 2;     // tokens in fp16, rows of 128 bytes
    static constexpr int W_RAW = LANES * KT;
    static constexpr int T_RAW = TOK * KT;
    static constexpr int RAW_BYTES = W_RAW + T_RAW;
    static constexpr int RAW_OFF = STAGES * B_BYTES;
    static constexpr int EXCH_OFF = RAW_OFF + RAW * RAW_BYTES;
    static constexpr int EXCH_WARP = 16 * 32 * 4;    // a warp's 16 columns
    static constexpr int EPI_WARPS = 8;
    static constexpr int BAR_OFF = EXCH_OFF + EPI_WARPS * EXCH_WARP;
    static constexpr int CONV_WARPS = 4 + 4;
    // full, free (per raw stage), empty, ready (per operand stage), acc_full and
    // acc_empty (per accumulator), drain
    static constexpr int NBARS = 2 * RAW + 2 * STAGES + 2 * ACCS + 1;
    static constexpr int SMEM_BYTES = BAR_OFF + NBARS * 8 + 16 + 1024;
    static constexpr int THREADS = 640;
    static constexpr int TMEM_COLS = 512;
    static constexpr int OP_COL0 = 256;              // operand stage s at OP_COL0 + 32 s
    static constexpr int OP_COLS = KT / 2;
    static constexpr int RELAYS = 3;
    static constexpr int EPI_COLS = COLS / 2;        // of a warp, at most
    static constexpr int REGS_LAUNCH = 96;
    static constexpr int REGS_CONTROL = 40, REGS_WEIGHTS = 56, REGS_TOKENS = 48, REGS_EPI = 168;
    // D fp32, A and B fp16, both K-major, M = 128 a CTA; N is added
    static constexpr uint32_t IDESC = (1u << 4) | (static_cast<uint32_t>(LANES * CTAS >> 4) << 24);
    static_assert(REGS_CONTROL + REGS_WEIGHTS + REGS_TOKENS + 2 * REGS_EPI <= 5 * REGS_LAUNCH,
                  "register shares");
    static_assert(OP_COL0 + STAGES * OP_COLS <= TMEM_COLS && ACCS * COLS <= OP_COL0,
                  "tensor-memory columns");
    static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
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
__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts_f32(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// Barrier `id` of the CTA's named ones, for `threads` of its threads.
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Four codes as two words of two fp16 numbers.
__device__ __forceinline__ void decode_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t bias = 0x64806480u;  // 1024 + 128, twice
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(bias));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(bias));
}

// Offset of a 16-byte chunk in a raw stage: rows of 64 bytes, 64-byte swizzle.
__device__ __forceinline__ uint32_t raw_at(uint32_t row, uint32_t chunk) {
    return row * 64u + ((chunk ^ ((row >> 1) & 3u)) << 4);
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

// f(j, acc[j]) for the first `left` columns, unrolled: acc stays in registers.
template <int COLS, typename F>
__device__ __forceinline__ void for_columns(const int (&acc)[COLS], int left, F f) {
#pragma unroll
    for (int j = 0; j < COLS; j += 16) {
        if (j + 16 <= left) {
#pragma unroll
            for (int i = 0; i < 16; ++i) f(j + i, acc[j + i]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (j + i < left) f(j + i, acc[j + i]);
        }
    }
}

template <bool PAIR, int ACT>
__global__ void __launch_bounds__(I8Cfg<PAIR>::THREADS, 1)
i8_tmem_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmC, I8TmemArgs p) {
    using C = I8Cfg<PAIR>;
    constexpr bool GATED = ACT != kNoAct;
    constexpr int STAGES = C::STAGES;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_addr(smem);
    const uint32_t full0 = sbase + C::BAR_OFF;      // own: a raw stage has landed
    const uint32_t free0 = full0 + 8 * C::RAW;      // own: its readers are done
    const uint32_t empty0 = free0 + 8 * C::RAW;     // own, multicast commit: operands read
    const uint32_t ready0 = empty0 + 8 * STAGES;    // operands written
    const uint32_t accf = ready0 + 8 * STAGES;      // own, multicast commit
    const uint32_t acce = accf + 8 * C::ACCS;       // leader: 8 warps a CTA
    const uint32_t drain = acce + 8 * C::ACCS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::BAR_OFF + C::NBARS * 8);
    const uint32_t abort_flag = smem_addr(tmem_slot + 1);
    const uint32_t last_flag = smem_addr(tmem_slot + 2);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
    const int first = blockIdx.x / C::CTAS, step = gridDim.x / C::CTAS;
    const long long timeout_ns = p.timeout_ns;
    unsigned* const fault = p.fault;
    const I8Share& share = p.share;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        if (GATED) prefetch_tmap(&tmC);
        for (int r = 0; r < C::RAW; ++r) {
            mbar_init(full0 + 8 * r, 1);
            mbar_init(free0 + 8 * r, C::CONV_WARPS);
        }
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
            if (lane == 0) {
                // -------------------------- TMA producer ------------------------------
                int it = 0;
                bool ok = true;
                Work w;
                const uint32_t bytes = C::W_RAW + static_cast<uint32_t>(share.tokens * C::KT);
                for (int u = first; ok && work_at<PAIR, GATED>(share, u, w); u += step) {
                    const int tok0 = w.t0 + rank * cta_tokens<PAIR>(share.tokens, p.T - w.t0);
                    const int ch0 = w.c0 + rank * (GATED ? C::LANES / 2 : C::LANES);
                    for (int kb = 0; kb < w.nkb; ++kb, ++it) {
                        const int r = it % C::RAW;
                        if (it >= C::RAW &&
                            !role_wait(free0 + 8 * r, ((it / C::RAW) & 1) ^ 1, timeout_ns, fault,
                                       kFaultEmptyBarrier, abort_flag)) {
                            ok = false;
                            break;
                        }
                        const int k0 = (w.kb_begin + kb) * C::KT;
                        const uint32_t fb = full0 + 8 * r;
                        const uint32_t wb = sbase + C::RAW_OFF + r * C::RAW_BYTES;
                        mbar_arrive_expect_tx(fb, bytes);
                        tma_load_2d(wb, &tmB, fb, k0, ch0);
                        if (GATED) tma_load_2d(wb + C::W_RAW / 2, &tmC, fb, k0, ch0);
                        tma_load_2d(wb + C::W_RAW, &tmA, fb, k0, tok0);
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
                Work w;
                for (int u = first; ok && work_at<PAIR, GATED>(share, u, w); u += step) {
                    const uint32_t idesc =
                        C::IDESC | static_cast<uint32_t>(
                                       C::CTAS * cta_tokens<PAIR>(share.tokens, p.T - w.t0) / 8)
                                       << 17;
                    for (int c0 = 0; c0 < w.nkb && ok; c0 += C::CHUNK, ++g) {
                        const int b = g % C::ACCS;
                        // the accumulator: its last chunk has been drained
                        if (g >= C::ACCS &&
                            !role_wait(acce + 8 * b, ((g / C::ACCS) - 1) & 1, timeout_ns, fault,
                                       kFaultAccumBarrier, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tmem_base + static_cast<uint32_t>(b * C::COLS);
                        const int c1 = min(w.nkb, c0 + C::CHUNK);
                        for (int kb = c0; kb < c1; ++kb, ++it) {
                            const int s = it % STAGES;
                            if (!role_wait<PAIR>(ready0 + 8 * s, (it / STAGES) & 1, timeout_ns,
                                                 fault, kFaultFullBarrier, abort_flag)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint64_t x = smem_desc_sw128_kmajor(sbase + s * C::B_BYTES);
                            const uint32_t a =
                                tmem_base + static_cast<uint32_t>(C::OP_COL0 + C::OP_COLS * s);
#pragma unroll
                            for (int k = 0; k < C::KT / C::UK; ++k)
                                // 16 columns of K: 32 bytes of a row, 8 columns of tensor memory
                                mma_f16_tmem_a<PAIR>(d, a + 8u * k, x + 2u * k, idesc,
                                                     (kb > c0 || k > 0) ? 1u : 0u);
                            mma_commit_form<PAIR>(empty0 + 8 * s);
                        }
                        if (!ok) break;
                        mma_commit_form<PAIR>(accf + 8 * b);
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
        // ------------------------------ weights (warps 4-7) ----------------------------
        regs_dec<C::REGS_WEIGHTS>();
        const int q = warp & 3;
        const uint32_t row = static_cast<uint32_t>(32 * q + lane);
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
        int it = 0;
        bool ok = true;
        Work w;
        for (int u = first; ok && work_at<PAIR, GATED>(share, u, w); u += step) {
            for (int kb = 0; kb < w.nkb; ++kb, ++it) {
                const int s = it % STAGES, raw = it % C::RAW;
                const bool got = role_wait(full0 + 8 * raw, (it / C::RAW) & 1, timeout_ns, fault,
                                           kFaultFullBarrier, abort_flag);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                const uint32_t src = sbase + C::RAW_OFF + raw * C::RAW_BYTES;
                uint4 v[C::KT / 16];
#pragma unroll
                for (int c = 0; c < C::KT / 16; ++c)
                    v[c] = lds_u32x4(src + raw_at(row, static_cast<uint32_t>(c)));
                if (it >= STAGES) {
                    const bool can = role_wait(empty0 + 8 * s, ((it / STAGES) & 1) ^ 1, timeout_ns,
                                               fault, kFaultEmptyBarrier, abort_flag);
                    if (!__all_sync(0xffffffffu, can)) {
                        ok = false;
                        break;
                    }
                }
                // the MMAs that read this stage before are done
                tc_fence_after();
                const uint32_t col =
                    lane_base + static_cast<uint32_t>(C::OP_COL0 + C::OP_COLS * s);
#pragma unroll
                for (int c = 0; c < C::KT / 16; c += 2) {
                    uint32_t h[16];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        decode_f16(v[c + i].x, h[8 * i], h[8 * i + 1]);
                        decode_f16(v[c + i].y, h[8 * i + 2], h[8 * i + 3]);
                        decode_f16(v[c + i].z, h[8 * i + 4], h[8 * i + 5]);
                        decode_f16(v[c + i].w, h[8 * i + 6], h[8 * i + 7]);
                    }
                    tmem_st_32x32b_x16(col + static_cast<uint32_t>(8 * c), h);
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
        // ------------------------------ tokens (warps 8-11) ----------------------------
        // A lane takes 16 codes: four lanes load a row's 64 bytes, and eight lanes
        // store two rows' chunks in all banks.
        regs_dec<C::REGS_TOKENS>();
        constexpr int kItems = C::TOK / 8 / 4;
        const uint32_t c = static_cast<uint32_t>(lane & 3);
        const uint32_t row0 = static_cast<uint32_t>(8 * (warp - 8) + (lane >> 2));
        int it = 0;
        bool ok = true;
        Work w;
        for (int u = first; ok && work_at<PAIR, GATED>(share, u, w); u += step) {
            const int rows = cta_tokens<PAIR>(share.tokens, p.T - w.t0);
            const int items = (rows - 8 * (warp - 8) + 31) / 32;  // of this warp: 8 rows each
            for (int kb = 0; kb < w.nkb; ++kb, ++it) {
                const int s = it % STAGES, raw = it % C::RAW;
                const bool got = role_wait(full0 + 8 * raw, (it / C::RAW) & 1, timeout_ns, fault,
                                           kFaultFullBarrier, abort_flag);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                const uint32_t src = sbase + C::RAW_OFF + raw * C::RAW_BYTES + C::W_RAW;
                const uint32_t dst = sbase + s * C::B_BYTES;
                uint4 v[kItems];
#pragma unroll
                for (int i = 0; i < kItems; ++i)
                    if (i < items) v[i] = lds_u32x4(src + raw_at(row0 + 32u * i, c));
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
                    if (i >= items) break;
                    const uint32_t r = row0 + 32u * i;
                    uint32_t h[8];
                    decode_f16(v[i].x, h[0], h[1]);
                    decode_f16(v[i].y, h[2], h[3]);
                    decode_f16(v[i].z, h[4], h[5]);
                    decode_f16(v[i].w, h[6], h[7]);
                    const uint32_t at = dst + r * 128u;
                    sts_u32x4(at + (((2u * c) ^ (r & 7u)) << 4), h[0], h[1], h[2], h[3]);
                    sts_u32x4(at + (((2u * c + 1u) ^ (r & 7u)) << 4), h[4], h[5], h[6], h[7]);
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
        // All eight warps walk through the same units whatever happens, so that the
        // named barriers always find them.
        regs_inc<C::REGS_EPI>();
        const int e = warp - 12;
        const int q = warp & 3;                  // lanes 32 q .. 32 q + 31
        const int half = e >> 2;
        const int n_lane = GATED ? rank * (C::LANES / 2) + 32 * (q & 1) + lane
                                 : rank * C::LANES + 32 * q + lane;
        const float* const scales = GATED && q >= 2 ? p.cs : p.bs;
        const uint32_t acce_leader = PAIR ? map_to_cta(acce, 0) : acce;
        const uint32_t exchange = sbase + C::EXCH_OFF + 4u * lane;
        int acc[C::EPI_COLS];
        int g = 0;
        bool ok = true;
        Work w;
        for (int u = first; work_at<PAIR, GATED>(share, u, w); u += step) {
            const int cols = C::CTAS * cta_tokens<PAIR>(share.tokens, p.T - w.t0);
            const int each = (cols + 31) / 32 * 16;
            const int col0 = half * each;
            const int count = min(each, cols - col0);  // of this warp: groups of 16, or none
#pragma unroll
            for (int i = 0; i < C::EPI_COLS; ++i) acc[i] = 0;
            for (int c0 = 0; ok && c0 < w.nkb; c0 += C::CHUNK, ++g) {
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
#pragma unroll
                for (int j = 0; j < C::EPI_COLS / 16; ++j) {
                    if (16 * j >= count) break;
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(tbase + 16u * j, r);
                    tmem_ld_wait(r);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[16 * j + i] += __float2int_rn(__uint_as_float(r[i]));
                }
                // the loads have completed: the arrival orders no writes
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR)
                        mbar_arrive_remote(acce_leader + 8 * b);
                    else
                        mbar_arrive(acce + 8 * b);
                }
            }
            if (!PAIR && share.splits > 1) {
                const long long slot = static_cast<long long>(share.tokens) * C::LANES;
                int* const mine = p.parts + u * slot + col0 * C::LANES + 32 * q + lane;
#pragma unroll
                for (int j = 0; j < C::EPI_COLS; ++j)
                    if (j < count) __stcg(mine + j * C::LANES, acc[j]);
                __threadfence();
                named_sync(1, 32 * C::EPI_WARPS);
                if (e == 0 && lane == 0) {
                    const bool last = atomicAdd(p.counters + w.tile, 1) == share.splits - 1;
                    if (last) atomicExch(p.counters + w.tile, 0);  // for the next call
                    st_shared_volatile(last_flag, last ? 1u : 0u);
                    __threadfence();
                }
                named_sync(1, 32 * C::EPI_WARPS);
                if (!ld_shared_volatile(last_flag)) continue;
                const int* const all = p.parts + w.tile * share.splits * slot + col0 * C::LANES +
                                       32 * q + lane;
                for (int s = 0; s < share.splits; ++s) {
                    if (w.tile * share.splits + s == u) continue;
#pragma unroll
                    for (int j = 0; j < C::EPI_COLS; ++j)
                        if (j < count) acc[j] += __ldcg(all + s * slot + j * C::LANES);
                }
            }
            const int n = w.c0 + n_lane;
            const bool mine = ok && n < p.N;
            const float channel = n < p.N ? scales[n] : 0.0f;
            const int t_first = w.t0 + col0;
            if (GATED) {
                // Of each two groups of 16 columns the gate's warp finishes the first
                // and up's the second: both give the other its values of the other.
                const int own = q >> 1;
                const uint32_t to = exchange + static_cast<uint32_t>(e * C::EXCH_WARP);
                const uint32_t from = exchange + static_cast<uint32_t>((e ^ 2) * C::EXCH_WARP);
#pragma unroll
                for (int j = 0; j < C::EPI_COLS; j += 32) {
                    if (j >= count) break;
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float first_t = p.as[min(t_first + j + i, p.T - 1)];
                        const float second_t = p.as[min(t_first + j + 16 + i, p.T - 1)];
                        const float a0 = i8_value(acc[j + i], first_t, channel);
                        const float a1 = i8_value(acc[j + 16 + i], second_t, channel);
                        v[i] = own ? a1 : a0;
                        sts_f32(to + 128u * i, own ? a0 : a1);
                    }
                    named_sync(2 + half * 2 + (q & 1), 64);
                    const int t = t_first + j + 16 * own;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float other = lds_f32(from + 128u * i);
                        if (mine && j + 16 * own + i < count && t + i < p.T) {
                            const float gate = own ? other : v[i], up = own ? v[i] : other;
                            put_output(p.y, static_cast<long long>(t + i) * p.ldy + n, p.type,
                                       act_value<ACT>(gate) * up);
                        }
                    }
                    named_sync(2 + half * 2 + (q & 1), 64);
                }
            } else if (mine) {
                const long long at = static_cast<long long>(t_first) * p.ldy + n;
                const float* const token = p.as + t_first;
                const int left = min(count, p.T - t_first);
                if (p.type == kI8Int32)
                    for_columns<C::EPI_COLS>(acc, left, [&](int j, int v) {
                        static_cast<int*>(p.y)[at + j * p.ldy] = v;
                    });
                else if (p.type == kI8Bfloat16)
                    for_columns<C::EPI_COLS>(acc, left, [&](int j, int v) {
                        put_output(p.y, at + j * p.ldy, kI8Bfloat16,
                                   i8_value(v, token[j], channel));
                    });
                else
                    for_columns<C::EPI_COLS>(acc, left, [&](int j, int v) {
                        put_output(p.y, at + j * p.ldy, kI8Float, i8_value(v, token[j], channel));
                    });
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
template <bool PAIR, int ACT>
cudaError_t configure(int dev) {
    using C = I8Cfg<PAIR>;
    constexpr int kDevices = 64;
    static bool done[kDevices] = {};
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, i8_tmem_kernel<PAIR, ACT>);
    if (e != cudaSuccess) return e;
    if (attr.numRegs < C::REGS_LAUNCH) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(i8_tmem_kernel<PAIR, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM_BYTES);
    if (e == cudaSuccess) done[dev] = true;
    return e;
}

template <bool PAIR, int ACT>
cudaError_t launch(const I8TmemMaps& maps, const I8TmemArgs& a, cudaStream_t s, int dev,
                   int sm_count) {
    using C = I8Cfg<PAIR>;
    cudaError_t e = configure<PAIR, ACT>(dev);
    if (e != cudaSuccess) return e;
    const long long units =
        static_cast<long long>(a.share.tiles_c) * a.share.tiles_t * a.share.splits;
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
    e = cudaLaunchKernelEx(&cfg, i8_tmem_kernel<PAIR, ACT>, maps.a, maps.b, maps.c, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int ACT>
cudaError_t launch_form(const I8TmemMaps& maps, const I8TmemArgs& a, bool pair, cudaStream_t s,
                        int dev, int sm_count) {
    return pair ? launch<true, ACT>(maps, a, s, dev, sm_count)
                : launch<false, ACT>(maps, a, s, dev, sm_count);
}

}  // namespace

I8Tile i8_tile(bool pair) {
    using P = I8Cfg<true>;
    return {pair ? 2 * P::LANES : P::LANES, P::TOK, P::KT};
}

size_t i8_parts_bytes(const I8Share& s) {
    if (s.splits < 2) return 0;
    return static_cast<size_t>(s.tiles_c) * s.tiles_t * s.splits * s.tokens * I8Cfg<false>::LANES * 4;
}

cudaError_t launch_i8_tmem(const I8TmemMaps& maps, const I8TmemArgs& a, bool pair, int act,
                           cudaStream_t s, int dev, int sm_count) {
    if (act == kActSilu) return launch_form<kActSilu>(maps, a, pair, s, dev, sm_count);
    if (act == kActGelu) return launch_form<kActGelu>(maps, a, pair, s, dev, sm_count);
    return launch_form<kNoAct>(maps, a, pair, s, dev, sm_count);
}

}  // namespace gemm_f32_impl
