// q8_wgrad_tmem.cu -- the weight gradient from an 8-bit checkpoint on the
// tensor core:  dW[d][n] = sum_t x^[t][d] dY[t][n].
//
// Arithmetic.  Every value of the checkpoint is exactly a bf16 number.  A
// float of dY is exactly the sum of three: b0 its upper 16 bits, b1 the upper
// 16 bits of y - b0, b2 = y - b0 - b1 (8 significant bits each, truncated, so
// the differences are exact).  Three bf16 MMAs a step, x^ b2 + x^ b1 + x^ b0,
// thus form exact products of the fp32 values; what is rounded is the
// accumulation.  The tensor core truncates its running fp32 sum at each
// addition (an error of about 2^-24 * 0.7 of the sum, always towards zero),
// so a tensor-memory sum covers one chunk of tokens and is then added, with
// rounding, into fp32 registers.  (Two bf16 parts would leave 2^-17 of each
// product; TF32 parts need two MMAs at half the rate.)
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
// A cluster of two CTAs computes a tile of 256 features x 256 columns with
// cta_group::2 MMAs (M = 256 columns n across the pair, N = 256 features, K =
// 16 tokens), CTA rank r holding columns n0 + 128 r .. in its tensor memory
// and features d0 + 128 r .. in its shared memory.  Per 16 tokens an SM's
// tensor core works 3 x 128 cycles and reads 12 KB of shared memory, half
// its share; dY in shared memory as well (both operands, three parts) would
// take more than the whole.
//
// 512 threads per CTA, registers rebalanced at start (launched at 128 each):
//   warp 0      one lane: TMA loads of a 32-token stage (dY 128 columns x 32,
//               codes 128 x 32, exponents 16 x 32), five stages deep;
//   warp 1      tensor-memory allocation for the pair; in the leader one lane
//               issues the MMAs; in the peer one lane relays its decoder's
//               and splitters' arrivals to the leader, one a stage;
//   warps 2-3   decode x^ to bf16 in shared memory, half of a stage each;
//   warps 4-7   split dY into tensor memory (warp 4 + q: lanes 32 q ..);
//   warps 8-15  per chunk add the accumulator (warp 8 + e: lanes 32 (e % 4)
//               .., columns 128 (e / 4) ..) into 128 registers a thread; at
//               the end of a unit store them: a warp writes 32 consecutive
//               columns of one row of dW.
// Tensor memory: 256 accumulator columns, then five operand stages of 48 (three
// parts of 32 tokens, two to a column).
//
// Few tiles and many tokens: the tokens are split over clusters into partial
// sums, added in split order by the GEMM's reduction kernel.
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

struct WgradCfg {
    static constexpr int TD = 256, TN = 256;  // features, columns of a tile
    static constexpr int HALF = 128;          // of each, per CTA
    static constexpr int KT = 32;             // tokens a stage
    static constexpr int UK = 16;             // tokens an MMA
    static constexpr int STAGES = 5;
    static constexpr int XB_BYTES = HALF * KT * 2;   // x^ in bf16: two 64-feature groups
    static constexpr int GROUP_BYTES = 64 * KT * 2;  // rows of 128 bytes, a token each
    static constexpr int Y_BYTES = HALF * KT * 4;
    static constexpr int C_BYTES = HALF * KT;
    static constexpr int S_BYTES = 16 * KT;
    // the swizzled x^ stages first: each 1024-byte aligned
    static constexpr int Y_OFF = STAGES * XB_BYTES;
    static constexpr int C_OFF = Y_OFF + STAGES * Y_BYTES;
    static constexpr int S_OFF = C_OFF + STAGES * C_BYTES;
    static constexpr int BAR_OFF = S_OFF + STAGES * S_BYTES;
    // full, empty, ready, splitters converted (peer), acc_full, acc_empty, drain
    static constexpr int NBARS = 4 * STAGES + 3;
    static constexpr int SMEM_BYTES = BAR_OFF + NBARS * 8 + 16 + 1024;
    static constexpr int THREADS = 512;
    static constexpr int TMEM_COLS = 512;
    static constexpr int OP_COL0 = TD;               // operand stage s at OP_COL0 + 48 s
    static constexpr int PART_COLS = KT / 2;
    static constexpr int OP_COLS = 3 * PART_COLS;
    static constexpr int EPI_WARPS = 8;
    static constexpr int REGS_LOW = 56, REGS_HIGH = 200;
    static constexpr int DRAIN_BATCH = 4;
    // D fp32, A and B bf16, B with its N axis contiguous, M = 256, N = 256
    static constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) |
                                      (static_cast<uint32_t>(TD >> 3) << 17) |
                                      (static_cast<uint32_t>(TN >> 4) << 24);
    static_assert(2 * 128 * REGS_LOW + 2 * 128 * REGS_HIGH == 65536, "register shares");
    static_assert(OP_COL0 + STAGES * OP_COLS <= TMEM_COLS, "tensor-memory columns");
    static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
};

// Shared-memory descriptor of the x^ stage: N-contiguous with 128-byte
// swizzle.  Rows of 64 features (128 bytes), one a token; eight rows make a
// 1024-byte swizzle group (stride byte offset, along K); the next 64 features
// lie GROUP_BYTES further on (leading byte offset, along N).
__device__ __forceinline__ uint64_t xhat_desc(uint32_t addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(WgradCfg::GROUP_BYTES >> 4) << 16;
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
__device__ __forceinline__ void lds_u32x4(uint32_t addr, uint32_t (&v)[4]) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
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

// Four codes as two words of two bf16 values each, exact.
template <int FMT>
__device__ __forceinline__ void decode_bf16(uint32_t w, float scale, uint32_t& lo, uint32_t& hi) {
    const float4 v = q8_decode4<FMT>(w);
    lo = upper_halves(v.x * scale, v.y * scale);
    hi = upper_halves(v.z * scale, v.w * scale);
}

__device__ __forceinline__ void mma_bf16_pair_tmem_a(uint32_t d_tmem, uint32_t a_tmem,
                                                     uint64_t b_desc, uint32_t idesc,
                                                     uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <int FMT>
__global__ void __launch_bounds__(WgradCfg::THREADS, 1)
q8_wgrad_pair_kernel(const __grid_constant__ CUtensorMap tmY,
                     const __grid_constant__ CUtensorMap tmC,
                     const __grid_constant__ CUtensorMap tmS, float* __restrict__ out,
                     long long ldo, long long split_stride, int D, int N, int T, int kb_per_split,
                     int splits, int chunk, unsigned* fault, long long timeout_ns, float alpha,
                     float beta, int scale_mode) {
    using C = WgradCfg;
    constexpr int STAGES = C::STAGES;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_addr(smem);
    const uint32_t full0 = sbase + C::BAR_OFF;      // own: the stage's copies
    const uint32_t empty0 = full0 + 8 * STAGES;     // own, multicast commit
    const uint32_t ready0 = empty0 + 8 * STAGES;    // decoder (leader: and splitters, relay)
    const uint32_t split0 = ready0 + 8 * STAGES;    // peer: its four splitter warps
    const uint32_t accf = split0 + 8 * STAGES;      // own, multicast commit
    const uint32_t acce = accf + 8;                 // leader: 8 warps x 2 CTAs
    const uint32_t drain = acce + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::BAR_OFF + C::NBARS * 8);
    const uint32_t abort_flag = smem_addr(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1;
    const int nclusters = gridDim.x >> 1;
    const int tiles_d = (D - 1) / C::TD + 1;
    const int tiles_n = (N - 1) / C::TN + 1;
    const int units = tiles_d * tiles_n * splits;
    const int kb_total = (T - 1) / C::KT + 1;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tmY);
        prefetch_tmap(&tmC);
        prefetch_tmap(&tmS);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
            // in the leader every arrival the MMA lane needs: two decoder
            // warps, four splitter warps, the peer's relay
            mbar_init(ready0 + 8 * s, rank == 0 ? 2 + 4 + 1 : 2);
            mbar_init(split0 + 8 * s, 4);
        }
        mbar_init(accf, 1);
        mbar_init(acce, 2 * C::EPI_WARPS);
        mbar_init(drain, 1);
        st_shared_volatile(abort_flag, 0u);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(tmem_slot), C::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    if (warp < 8) {
        regs_dec<C::REGS_LOW>();
        if (warp == 0) {
            if (lane == 0) {
                // -------------------------- TMA producer (both CTAs) ------------------
                int it = 0;
                bool ok = true;
                for (int u = cluster; u < units && ok; u += nclusters) {
                    const Unit w = decode(u, tiles_d, tiles_n, kb_per_split, kb_total, C::TN, C::TD);
                    const int dc = w.m0 + static_cast<int>(rank) * C::HALF;
                    const int nc = w.n0 + static_cast<int>(rank) * C::HALF;
                    // exponents: the aligned 16 blocks that hold this CTA's four
                    const int bc = (dc / kQ8Block) & ~15;
                    for (int kb = 0; kb < w.nkb; ++kb, ++it) {
                        const int s = it % STAGES;
                        if (it >= STAGES &&
                            !role_wait(empty0 + 8 * s, ((it / STAGES) & 1) ^ 1, timeout_ns, fault,
                                       kFaultEmptyBarrier, abort_flag)) {
                            ok = false;
                            break;
                        }
                        const int t0 = (w.kb_begin + kb) * C::KT;
                        const uint32_t fb = full0 + 8 * s;
                        mbar_arrive_expect_tx(fb, C::Y_BYTES + C::C_BYTES + C::S_BYTES);
                        tma_load_2d(sbase + C::Y_OFF + s * C::Y_BYTES, &tmY, fb, nc, t0);
                        tma_load_2d(sbase + C::C_OFF + s * C::C_BYTES, &tmC, fb, dc, t0);
                        tma_load_2d(sbase + C::S_OFF + s * C::S_BYTES, &tmS, fb, bc, t0);
                    }
                }
                // wind down: this CTA's copies have landed and its stages have
                // been released by the MMAs
                const long long tail = ok ? timeout_ns : timeout_ns / 8 + 1000;
                for (int j = (it > STAGES ? it - STAGES : 0); j < it; ++j) {
                    mbar_wait(full0 + 8 * (j % STAGES), (j / STAGES) & 1, tail, fault, kFaultDrain);
                    mbar_wait(empty0 + 8 * (j % STAGES), (j / STAGES) & 1, tail, fault, kFaultDrain);
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            if (lane == 0 && rank == 0) {
                // -------------------------- MMA issuer (leader) -----------------------
                int it = 0;
                int g = 0;  // chunks issued
                bool ok = true;
                for (int u = cluster; u < units && ok; u += nclusters) {
                    const Unit w = decode(u, tiles_d, tiles_n, kb_per_split, kb_total, C::TN, C::TD);
                    for (int c0 = 0; c0 < w.nkb && ok; c0 += chunk, ++g) {
                        // the single accumulator: both epilogues have drained chunk g - 1
                        if (g >= 1 && !role_wait(acce, (g - 1) & 1, timeout_ns, fault,
                                                 kFaultAccumBarrier, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const int c1 = min(w.nkb, c0 + chunk);
                        for (int kb = c0; kb < c1; ++kb, ++it) {
                            const int s = it % STAGES;
                            if (!role_wait(ready0 + 8 * s, (it / STAGES) & 1, timeout_ns, fault,
                                           kFaultFullBarrier, abort_flag)) {
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
                                mma_bf16_pair_tmem_a(tmem_base, b2 + kc, xk, C::IDESC, acc);
                                mma_bf16_pair_tmem_a(tmem_base, b1 + kc, xk, C::IDESC, 1u);
                                mma_bf16_pair_tmem_a(tmem_base, b0 + kc, xk, C::IDESC, 1u);
                            }
                            mma_commit_pair_multicast(empty0 + 8 * s, 0x3);
                        }
                        if (!ok) break;
                        mma_commit_pair_multicast(accf, 0x3);
                    }
                }
                mma_commit_pair(drain);
                mbar_wait(drain, 0, ok ? timeout_ns : timeout_ns / 8 + 1000, fault, kFaultDrain);
            } else if (lane == 0) {
                // -------------------------- relay (peer CTA) --------------------------
                const uint32_t ready_leader = map_to_cta(ready0, 0);
                int it = 0;
                bool ok = true;
                for (int u = cluster; u < units && ok; u += nclusters) {
                    const Unit w = decode(u, tiles_d, tiles_n, kb_per_split, kb_total, C::TN, C::TD);
                    for (int kb = 0; kb < w.nkb; ++kb, ++it) {
                        const int s = it % STAGES;
                        const uint32_t par = (it / STAGES) & 1;
                        if (!role_wait(ready0 + 8 * s, par, timeout_ns, fault, kFaultFullBarrier,
                                       abort_flag) ||
                            !role_wait(split0 + 8 * s, par, timeout_ns, fault, kFaultFullBarrier,
                                       abort_flag)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_cluster(ready_leader + 8 * s);
                    }
                }
            }
            __syncwarp();
        } else if (warp < 4) {
            // ------------------------------ x^ decoders (warps 2-3, both CTAs) --------
            // A lane takes 16 codes (features 16 c .. 16 c + 15 of a token row, c =
            // lane % 8) and writes them as two 16-byte chunks of the row of group
            // c / 4.  Lanes of the second group write their odd chunk first, so that
            // the eight lanes of a store pass cover all banks.
            const int c = lane & 7;
            const int odd = c >> 2;
            const int row0 = 16 * (warp - 2) + (lane >> 3);
            int it = 0;
            bool ok = true;
            for (int u = cluster; u < units && ok; u += nclusters) {
                const Unit w = decode(u, tiles_d, tiles_n, kb_per_split, kb_total, C::TN, C::TD);
                const int dc = w.m0 + static_cast<int>(rank) * C::HALF;
                const uint32_t sc = static_cast<uint32_t>(((dc / kQ8Block) & 15) + (c >> 1));
                for (int kb = 0; kb < w.nkb; ++kb, ++it) {
                    const int s = it % STAGES;
                    const bool got = role_wait(full0 + 8 * s, (it / STAGES) & 1, timeout_ns, fault,
                                               kFaultFullBarrier, abort_flag);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    const uint32_t codes = sbase + C::C_OFF + s * C::C_BYTES;
                    const uint32_t exps = sbase + C::S_OFF + s * C::S_BYTES + sc;
                    const uint32_t dst = sbase + s * C::XB_BYTES + odd * C::GROUP_BYTES;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t r = static_cast<uint32_t>(row0 + 4 * i);
                        uint32_t q[4], v[8];
                        lds_u32x4(codes + r * C::HALF + 16 * c, q);
                        const float scale = q8_scale<FMT>(lds_u8(exps + 16 * r));
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            decode_bf16<FMT>(q[j], scale, v[2 * j], v[2 * j + 1]);
                        const uint32_t row = dst + r * 128u;
                        const uint32_t k0 = static_cast<uint32_t>(2 * (c & 3));
                        const uint32_t at0 = row + ((k0 ^ (r & 7u)) << 4);
                        const uint32_t at1 = row + (((k0 + 1u) ^ (r & 7u)) << 4);
                        if (odd) {
                            sts_u32x4(at1, v[4], v[5], v[6], v[7]);
                            sts_u32x4(at0, v[0], v[1], v[2], v[3]);
                        } else {
                            sts_u32x4(at0, v[0], v[1], v[2], v[3]);
                            sts_u32x4(at1, v[4], v[5], v[6], v[7]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ready0 + 8 * s);
                }
            }
            __syncwarp();
        } else {
            // ------------------------------ dY splitters (warps 4-7, both CTAs) -------
            const int q = warp & 3;
            const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
            int it = 0;
            bool ok = true;
            for (int u = cluster; u < units && ok; u += nclusters) {
                const Unit w = decode(u, tiles_d, tiles_n, kb_per_split, kb_total, C::TN, C::TD);
                for (int kb = 0; kb < w.nkb; ++kb, ++it) {
                    const int s = it % STAGES;
                    const bool got = role_wait(full0 + 8 * s, (it / STAGES) & 1, timeout_ns, fault,
                                               kFaultFullBarrier, abort_flag);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    const uint32_t src = sbase + C::Y_OFF + s * C::Y_BYTES +
                                         static_cast<uint32_t>(4 * (32 * q + lane));
                    const uint32_t col =
                        lane_base + static_cast<uint32_t>(C::OP_COL0 + C::OP_COLS * s);
                    // 16 tokens at a time: this warpgroup runs on 56 registers
#pragma unroll
                    for (int h = 0; h < C::KT / 16; ++h) {
                        float y[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            y[i] = lds_f32(src + static_cast<uint32_t>(16 * h + i) * (4 * C::HALF));
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
                    if (lane == 0) mbar_arrive((rank == 0 ? ready0 : split0) + 8 * s);
                }
            }
            __syncwarp();
        }
    } else {
        // ------------------------------ epilogue (warps 8-15, both CTAs) --------------
        regs_inc<C::REGS_HIGH>();
        const int e = warp - 8;
        const int q = warp & 3;                  // lanes 32 q .. 32 q + 31
        const int col0 = (e >> 2) * EPI_COLS;    // accumulator columns: features
        const int nl = static_cast<int>(rank) * C::HALF + 32 * q + lane;
        const uint32_t acce_leader = map_to_cta(acce, 0);
        const uint32_t tbase = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                               static_cast<uint32_t>(col0);
        float acc[EPI_COLS];
        int g = 0;
        bool ok = true;
        for (int u = cluster; u < units && ok; u += nclusters) {
            const Unit w = decode(u, tiles_d, tiles_n, kb_per_split, kb_total, C::TN, C::TD);
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
                        if (c0 == 0) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) acc[16 * j + i] = __uint_as_float(r[b][i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) acc[16 * j + i] += __uint_as_float(r[b][i]);
                        }
                    }
                }
                // the loads have completed: the arrival orders no writes
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(acce_leader);
            }
            if (!ok) break;
            const int n = w.n0 + nl;
            if (n < N) {
                float* p = out + static_cast<long long>(w.split) * split_stride +
                           static_cast<long long>(w.m0 + col0) * ldo + n;
                const int rows = D - (w.m0 + col0);
#pragma unroll
                for (int j = 0; j < EPI_COLS; ++j, p += ldo)
                    if (j < rows) *p = scale1(acc[j], p, alpha, beta, scale_mode);
            }
        }
        __syncwarp();
    }

    // neither CTA may leave while its partner can still reach its shared or
    // tensor memory
    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    }
}

// Shared-memory attribute of the kernel on device `dev`, once (the ABI's
// mutex is held).  The register rebalancing waits for ever unless the block
// was launched with the whole register file, so a build in which the
// compiler took fewer than 128 registers a thread is refused here.
template <int FMT>
cudaError_t configure(int dev) {
    constexpr int kDevices = 64;
    static bool done[kDevices] = {};
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, q8_wgrad_pair_kernel<FMT>);
    if (e != cudaSuccess) return e;
    if (attr.numRegs * WgradCfg::THREADS < 65536) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(q8_wgrad_pair_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             WgradCfg::SMEM_BYTES);
    if (e == cudaSuccess) done[dev] = true;
    return e;
}

}  // namespace

Q8WgradTile q8_wgrad_tile() { return {WgradCfg::TD, WgradCfg::TN, WgradCfg::KT}; }

cudaError_t launch_q8_wgrad_pair(const Q8WgradPairArgs& a, cudaStream_t s, int dev, int sm_count) {
    using C = WgradCfg;
    cudaError_t e = a.format == kQ8Int8 ? configure<kQ8Int8>(dev) : configure<kQ8E4m3>(dev);
    if (e != cudaSuccess) return e;
    const int tiles = ((a.cols - 1) / C::TD + 1) * ((a.N - 1) / C::TN + 1);
    const int units = tiles * a.splits;
    const int clusters = units < sm_count / 2 ? units : sm_count / 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1] = pdl_attribute();
    cfg.gridDim = dim3(2 * clusters);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg,
                           a.format == kQ8Int8 ? q8_wgrad_pair_kernel<kQ8Int8>
                                               : q8_wgrad_pair_kernel<kQ8E4m3>,
                           a.tmY, a.tmC, a.tmS, a.out, a.ldo, a.split_stride, a.cols, a.N, a.rows,
                           a.kb_per_split, a.splits, a.chunk, a.fault, a.timeout_ns, a.alpha,
                           a.beta, a.mode);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace gemm_f32_impl
