// q8_api.cu -- the C ABI of the 8-bit activation checkpoints: argument
// checks, the edge rules and kernel dispatch.  Empty matrices are a
// successful no-op, as in the GEMM entry points; nothing here exits the
// process.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <limits>

#include "gemm_f32.h"
#include "gemm_internal.h"

using namespace gemm_f32_impl;

#define Q8_TRY(expr)                                  \
    do {                                              \
        const int st_ = (expr);                       \
        if (st_ != GEMM_F32_SUCCESS) return st_;      \
    } while (0)

namespace {

// A matrix in memory, in bytes: `rows` rows of `width` bytes, `stride` apart.
struct Region {
    const void* base;
    long long rows, width, stride;
};

// Whether two regions share a byte.  Matrices with the same stride may lie
// side by side in the same rows of one buffer (the halves of a wider
// product): then they are apart when their columns are.  With different
// strides, address ranges that meet count as shared.
bool share(const Region& a, const Region& b) {
    if (!a.base || !b.base || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.base), b0 = reinterpret_cast<uintptr_t>(b.base);
    const uintptr_t a1 = a0 + static_cast<uintptr_t>((a.rows - 1) * a.stride + a.width);
    const uintptr_t b1 = b0 + static_cast<uintptr_t>((b.rows - 1) * b.stride + b.width);
    if (a1 <= b0 || b1 <= a0) return false;
    if (a.stride != b.stride || a.rows == 1 || b.rows == 1) return true;
    // b's first byte, counted from the start of the row of a that holds it
    const long long diff = static_cast<long long>(b0) - static_cast<long long>(a0);
    const long long at = ((diff % a.stride) + a.stride) % a.stride;
    return !(at >= a.width && at + b.width <= a.stride);
}

bool bad_dims(long long rows, long long cols, long long ld) {
    return ld < (cols > 1 ? cols : 1) ||
           (rows > 0 && ld > std::numeric_limits<long long>::max() / 16 / rows);
}

// A float (or, elem = 2, bf16) matrix argument: pointer present and aligned
// to its element, row stride at least the row.
int check_matrix(const void* p, long long rows, long long cols, long long ld, int elem) {
    if (bad_dims(rows, cols, ld) || !p) return GEMM_F32_ERR_INVALID_VALUE;
    if (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(elem - 1))
        return GEMM_F32_ERR_INVALID_VALUE;
    return GEMM_F32_SUCCESS;
}

Region region(const void* p, long long rows, long long cols, long long ld, int elem) {
    return {p, rows, cols * elem, ld * elem};
}

long long blocks_of(long long cols) {
    return (cols + GEMM_F32_Q8_BLOCK - 1) / GEMM_F32_Q8_BLOCK;
}

int check_shape(const gemm_f32_q8* q) {
    if (!q || q->rows < 0 || q->cols < 0) return GEMM_F32_ERR_INVALID_VALUE;
    if (q->format != GEMM_F32_Q8_INT8 && q->format != GEMM_F32_Q8_E4M3)
        return GEMM_F32_ERR_INVALID_VALUE;
    return GEMM_F32_SUCCESS;
}

// The arrays of a nonempty checkpoint: 16-byte aligned, row strides multiples
// of 16 bytes that hold a row.
int check_arrays(const gemm_f32_q8* q) {
    if (!q->codes || !q->scales) return GEMM_F32_ERR_INVALID_VALUE;
    if ((reinterpret_cast<uintptr_t>(q->codes) | reinterpret_cast<uintptr_t>(q->scales)) & 15u)
        return GEMM_F32_ERR_INVALID_VALUE;
    if ((q->ldcodes & 15) || (q->ldscales & 15)) return GEMM_F32_ERR_INVALID_VALUE;
    if (bad_dims(q->rows, q->cols, q->ldcodes) ||
        bad_dims(q->rows, blocks_of(q->cols), q->ldscales))
        return GEMM_F32_ERR_INVALID_VALUE;
    return GEMM_F32_SUCCESS;
}

Region codes_of(const gemm_f32_q8* q) { return region(q->codes, q->rows, q->cols, q->ldcodes, 1); }
Region scales_of(const gemm_f32_q8* q) {
    return region(q->scales, q->rows, blocks_of(q->cols), q->ldscales, 1);
}

// Outputs that share memory with one another or with an input.
int check_apart(const Region* out, int nout, const Region* in, int nin) {
    for (int i = 0; i < nout; ++i) {
        for (int j = i + 1; j < nout; ++j)
            if (share(out[i], out[j])) return GEMM_F32_ERR_INVALID_VALUE;
        for (int j = 0; j < nin; ++j)
            if (share(out[i], in[j])) return GEMM_F32_ERR_INVALID_VALUE;
    }
    return GEMM_F32_SUCCESS;
}

bool same_shape(const gemm_f32_q8* a, const gemm_f32_q8* b) {
    return a->rows == b->rows && a->cols == b->cols && a->format == b->format;
}

Q8In in_of(const gemm_f32_q8* q) { return {q->codes, q->scales, q->ldcodes, q->ldscales}; }
Q8Out out_of(const gemm_f32_q8* q) { return {q->codes, q->scales, q->ldcodes, q->ldscales}; }

long long round_up(long long x, long long m) { return (x + m - 1) / m * m; }

// The tensor-core weight gradient's times in microseconds, fitted to calls
// with each choice forced (a stage is 32 tokens of a tile): what a call takes
// more than one of single CTAs; a stage of units that run through the tokens
// side by side and share operands in L2; of units that are all at different
// tokens, with operands that fit L2 and beyond it; the second kernel, and
// writing and adding one partial sum.
// Measured in calls back to back, shared against whole: 4096 x 1280 x 2048 (40
// tiles on 76 pairs) 52.8 against 72.2 us, 4096 x 1536 x 2304 (54) 66.9 against
// 73.5, 16384 x 1280 x 2048 169 against 267; not taken, by the calls of the fit:
// 4096 x 2048 x 2048 (64) 79.3 against 76.5, 16384 x 2048 x 2048 287 against
// 277.  Single CTAs against pairs: 8192 x 8192 x 8192 2.20 against 2.00 ms, 4096
// x 2048 x 2048 81 against 74 us, 16384 x 8192 x 32 81 against 139 to 150, 8192
// x 4096 x 384 62 against 72, and replayed from a graph 64 x 512 x 512 6.3
// against 6.8.  The old dW (beta) is not counted.
struct WgradTimes {
    double more, stage, apart, far, sum, part;
};
constexpr WgradTimes kWgradPair = {1.5, 0.53, 0.57, 0.65, 4.4, 0.06};
constexpr WgradTimes kWgradSingle = {0.0, 0.59, 0.62, 0.70, 4.0, 0.02};
constexpr double kWgradL2Bytes = 64e6;
// what sharing has to save of the whole call: back to back the largest calls
// are at the power limit and gain nothing from a shorter last round (8192 x
// 8192 x 8192, 36 of 1024 tiles in halves: 2.00 against 1.93 ms)
constexpr double kWgradLeastGain = 0.05;

// Stages per tensor-core sum, 256 tokens: relative error 7e-7 (2-norm; an fp32
// product in one running sum has 1.6e-6 at 8192 tokens, in sums over ranges
// 5e-7 to 7e-7), most of it one way: 6e-7 towards zero.  Each sum costs the
// MMAs a wait of ~0.23 us: 128 tokens, 4e-7, were 2.2 % slower at 8192 x 8192
// x 8192, 512 tokens, 1.4e-6, 0.8 % faster.  Units of up to 512 tokens, where
// an fp32 product has no more than 4e-7 either (2.1e-7 at 128 tokens, 2.9e-7 at
// 256), pay for 128 with two waits.
constexpr int kWgradChunk = 8, kWgradShortChunk = 4, kWgradShortStages = 16;

// The CUDA-core kernel, which has no pipeline to fill and no descriptors, for
// a few tokens and small outputs (measured in calls back to back, against the
// tensor-core kernel's single CTAs, in microseconds: 16 x 512 x 512 5.6 and 6.3,
// 16 x 1024 x 1024 5.7 and 6.6, 32 x 512 x 512 5.6 and 6.3, 24 x 300 x 300 6.1
// and 6.8; but 4 x 2048 x 2048 10.5 and 8.1, 64 x 512 x 512 8.3 and 7.0, 64 x 64
// x 64 8.2 and 6; replayed from a graph, in the same order, 2.7 and 5.8, 3.9 and
// 6.0, 3.7 and 5.8, 4.2 and 6.0, 9.0 and 7.3, 5.5 and 6.3, 5.4 and 5.3).
constexpr int kFfmaTokens = 32;
constexpr double kFfmaOutputs = 1 << 20, kFfmaProducts = 1.7e7;

// Shares out the last `shared` tiles in groups of `group` tiles, `runs` a group.
void cut_tiles(Q8WgradShare* s, int shared, int group, int runs) {
    s->whole -= shared;
    s->shared = shared;
    s->group_stages = group * s->stages;
    s->group_runs = runs;
    s->per = s->group_stages / runs;
    s->extra = s->group_stages % runs;
    s->runs = shared / group * runs;
}

// How the tiles of a weight gradient are shared out over the CTA pairs, or the
// single CTAs, and the time that should take.  Requested splits: every tile in
// that many runs.  Otherwise whole tiles for as many rounds as they fill, and
// the rest shared by all units where that shortens the last round by more than
// the partial sums cost.
Q8WgradShare share_wgrad(const Q8WgradArgs& a, bool pair, int splits, int sm_count, double* us) {
    const Q8WgradTile tile = q8_wgrad_tile(pair);
    const WgradTimes& time = pair ? kWgradPair : kWgradSingle;
    Q8WgradShare s = {};
    s.tiles_d = (a.cols - 1) / tile.features + 1;
    s.tiles_n = (a.N - 1) / tile.columns + 1;
    s.stages = (a.rows - 1) / tile.tokens + 1;
    s.whole = s.tiles_d * s.tiles_n;
    const int units = pair ? sm_count / 2 : sm_count;
    const int rounds = (s.whole - 1) / units + 1;
    const int rest = splits > 0 ? s.whole : s.whole % units;
    const long long all = static_cast<long long>(rest) * s.stages;
    const double whole_us = time.stage * s.stages;
    *us = time.more + whole_us * rounds;
    if (all == 0 || all > std::numeric_limits<int>::max()) return s;
    if (splits > 0) {
        const int n = splits < s.stages ? splits : s.stages;
        if (n > 1) cut_tiles(&s, rest, 1, n);
        return s;
    }
    // the same number of runs for every tile, which start side by side; or as
    // many as there are units, over tile boundaries
    const double least = whole_us * (1.0 - kWgradLeastGain * rounds);
    const int each = std::min(units / rest, s.stages / 4);
    const int through = static_cast<int>(std::min<long long>(units, all / 4));
    double each_us = whole_us, through_us = whole_us;
    if (each > 1)
        each_us = time.stage * ((s.stages - 1) / each + 1) + time.sum + time.part * each * rest;
    if (through > rest) {
        const bool far = a.rows * (4.0 * a.N + a.cols) > kWgradL2Bytes;
        through_us = (far ? time.far : time.apart) * static_cast<double>((all - 1) / through + 1) +
                     time.sum + time.part * (through + rest);
    }
    if (each_us < least && each_us <= through_us) {
        cut_tiles(&s, rest, 1, each);
        *us += each_us - whole_us;
    } else if (through_us < least) {
        cut_tiles(&s, rest, rest, through);
        *us += through_us - whole_us;
    }
    return s;
}

// The tensor maps of dY (rows x N, row stride ld): see q8_wgrad_tmem.cu.
int map_dy(const float* dy, long long ld, int rows, int N, Q8WgradTmemArgs* k) {
    const Q8WgradTile tile = q8_wgrad_tile(false);
    const int box = tile.columns;
    const uintptr_t base = reinterpret_cast<uintptr_t>(dy);
    if (rows == 1) ld = round_up(N, 4);  // never used
    if (base % 16 == 0 && ld % 4 == 0)
        return call_tensor_map(&k->tmY.map[0], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dy, N, rows, 4 * ld,
                               box, tile.tokens);
    k->shifted = 1;
    for (int c = 0; c < 4; ++c) {
        const int row = c < rows ? c : 0;
        const uintptr_t first = base + static_cast<uintptr_t>(row * ld) * 4;
        const unsigned shift = static_cast<unsigned>(first % 16 / 4);
        k->shifts |= shift << (2 * c);
        Q8_TRY(call_tensor_map(&k->tmY.map[c], CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                               reinterpret_cast<const void*>(first - 4 * shift),
                               static_cast<long long>(N) + shift, (rows - 1 - row) / 4 + 1, 16 * ld,
                               box + 4, tile.tokens / 4));
    }
    return GEMM_F32_SUCCESS;
}

int status(cudaError_t e) { return e == cudaSuccess ? GEMM_F32_SUCCESS : static_cast<int>(e); }

}  // namespace

extern "C" {

int gemm_f32_q8_store(const float* X, long long ldx, const gemm_f32_q8* q, cudaStream_t stream) {
    Q8_TRY(check_shape(q));
    if (q->rows == 0 || q->cols == 0) return GEMM_F32_SUCCESS;
    Q8_TRY(check_arrays(q));
    Q8_TRY(check_matrix(X, q->rows, q->cols, ldx, 4));
    const Region out[] = {codes_of(q), scales_of(q)};
    const Region in[] = {region(X, q->rows, q->cols, ldx, 4)};
    Q8_TRY(check_apart(out, 2, in, 1));
    std::lock_guard<std::mutex> lock(api_mutex());
    CallState c;
    Q8_TRY(call_state(stream, &c));
    return status(launch_q8_store(X, ldx, q->rows, q->cols, q->format, out_of(q),
                                  {stream, c.sm_count}));
}

int gemm_f32_q8_restore(const gemm_f32_q8* q, void* X, long long ldx, int type,
                        cudaStream_t stream) {
    Q8_TRY(check_shape(q));
    if (type != GEMM_F32_Q8_TO_F32 && type != GEMM_F32_Q8_TO_BF16)
        return GEMM_F32_ERR_INVALID_VALUE;
    if (q->rows == 0 || q->cols == 0) return GEMM_F32_SUCCESS;
    const int elem = type == GEMM_F32_Q8_TO_F32 ? 4 : 2;
    Q8_TRY(check_arrays(q));
    Q8_TRY(check_matrix(X, q->rows, q->cols, ldx, elem));
    const Region out[] = {region(X, q->rows, q->cols, ldx, elem)};
    const Region in[] = {codes_of(q), scales_of(q)};
    Q8_TRY(check_apart(out, 1, in, 2));
    std::lock_guard<std::mutex> lock(api_mutex());
    CallState c;
    Q8_TRY(call_state(stream, &c));
    return status(launch_q8_restore(in_of(q), q->rows, q->cols, q->format, X, ldx, elem == 2,
                                    {stream, c.sm_count}));
}

int gemm_f32_q8_gated(int act, const float* G, long long ldg, const float* U, long long ldu,
                      float* H, long long ldh, const gemm_f32_q8* gq, const gemm_f32_q8* uq,
                      cudaStream_t stream) {
    if (act != GEMM_F32_ACT_SILU && act != GEMM_F32_ACT_GELU) return GEMM_F32_ERR_INVALID_VALUE;
    Q8_TRY(check_shape(gq));
    Q8_TRY(check_shape(uq));
    if (!same_shape(gq, uq)) return GEMM_F32_ERR_INVALID_VALUE;
    const int rows = gq->rows, cols = gq->cols;
    if (rows == 0 || cols == 0) return GEMM_F32_SUCCESS;
    Q8_TRY(check_arrays(gq));
    Q8_TRY(check_arrays(uq));
    Q8_TRY(check_matrix(G, rows, cols, ldg, 4));
    Q8_TRY(check_matrix(U, rows, cols, ldu, 4));
    Q8_TRY(check_matrix(H, rows, cols, ldh, 4));
    const Region out[] = {region(H, rows, cols, ldh, 4), codes_of(gq), scales_of(gq), codes_of(uq),
                          scales_of(uq)};
    const Region in[] = {region(G, rows, cols, ldg, 4), region(U, rows, cols, ldu, 4)};
    Q8_TRY(check_apart(out, 5, in, 2));
    std::lock_guard<std::mutex> lock(api_mutex());
    CallState c;
    Q8_TRY(call_state(stream, &c));
    GatedArgs a = {G, U, H, ldg, ldu, ldh, out_of(gq), out_of(uq), rows, cols, gq->format, act};
    return status(launch_q8_gated(a, {stream, c.sm_count}));
}

int gemm_f32_q8_gated_backward(int act, const gemm_f32_q8* gq, const gemm_f32_q8* uq,
                               const float* dH, long long lddh, float* dG, long long lddg,
                               float* dU, long long lddu, const gemm_f32_q8* hq,
                               cudaStream_t stream) {
    if (act != GEMM_F32_ACT_SILU && act != GEMM_F32_ACT_GELU) return GEMM_F32_ERR_INVALID_VALUE;
    Q8_TRY(check_shape(gq));
    Q8_TRY(check_shape(uq));
    if (!same_shape(gq, uq)) return GEMM_F32_ERR_INVALID_VALUE;
    if (hq) {
        Q8_TRY(check_shape(hq));
        if (!same_shape(gq, hq)) return GEMM_F32_ERR_INVALID_VALUE;
    }
    const int rows = gq->rows, cols = gq->cols;
    if (rows == 0 || cols == 0) return GEMM_F32_SUCCESS;
    Q8_TRY(check_arrays(gq));
    Q8_TRY(check_arrays(uq));
    if (hq) Q8_TRY(check_arrays(hq));
    Q8_TRY(check_matrix(dH, rows, cols, lddh, 4));
    Q8_TRY(check_matrix(dG, rows, cols, lddg, 4));
    Q8_TRY(check_matrix(dU, rows, cols, lddu, 4));
    Region out[4] = {region(dG, rows, cols, lddg, 4), region(dU, rows, cols, lddu, 4)};
    const Region in[] = {region(dH, rows, cols, lddh, 4), codes_of(gq), scales_of(gq), codes_of(uq),
                         scales_of(uq)};
    int nout = 2;
    if (hq) {
        out[nout++] = codes_of(hq);
        out[nout++] = scales_of(hq);
    }
    Q8_TRY(check_apart(out, nout, in, 5));
    std::lock_guard<std::mutex> lock(api_mutex());
    CallState c;
    Q8_TRY(call_state(stream, &c));
    GatedBackwardArgs a = {in_of(gq), in_of(uq), dH, dG, dU, lddh, lddg, lddu,
                           hq ? out_of(hq) : Q8Out{nullptr, nullptr, 0, 0},
                           rows, cols, gq->format, act};
    return status(launch_q8_gated_backward(a, {stream, c.sm_count}));
}

int gemm_f32_q8_wgrad(const gemm_f32_q8* x, const float* dY, long long lddy, int N, float alpha,
                      float beta, float* dW, long long lddw, int algo, int splits,
                      cudaStream_t stream) {
    Q8_TRY(check_shape(x));
    if (N < 0 || splits < 0 || splits > GEMM_F32_MAX_SPLITS) return GEMM_F32_ERR_INVALID_VALUE;
    if (algo != GEMM_F32_ALGO_AUTO && algo != GEMM_F32_ALGO_FFMA &&
        (algo < GEMM_F32_ALGO_3XBF16 || algo > GEMM_F32_ALGO_3XBF16_SINGLE))
        return GEMM_F32_ERR_INVALID_VALUE;
    if (x->cols == 0 || N == 0) return GEMM_F32_SUCCESS;
    // more tiles of dW than an index holds: no memory does either
    if (1.0 * x->cols * N > 1e13) return GEMM_F32_ERR_INVALID_VALUE;
    Q8_TRY(check_matrix(dW, x->cols, N, lddw, 4));
    const bool reads = x->rows > 0 && alpha != 0.0f;
    if (x->rows > 0) {
        Q8_TRY(check_arrays(x));
        Q8_TRY(check_matrix(dY, x->rows, N, lddy, 4));
        const Region out[] = {region(dW, x->cols, N, lddw, 4)};
        const Region in[] = {codes_of(x), scales_of(x), region(dY, x->rows, N, lddy, 4)};
        Q8_TRY(check_apart(out, 1, in, 3));
    }
    std::lock_guard<std::mutex> lock(api_mutex());
    CallState c;
    Q8_TRY(call_state(stream, &c));
    if (!reads) return status(launch_scale_c(dW, lddw, x->cols, N, beta, stream));
    Q8WgradArgs a = {in_of(x), dY, dW, lddy, lddw, x->rows, x->cols, N, x->format, alpha, beta,
                     beta != 0.0f ? 2 : alpha == 1.0f ? 0 : 1};
    if (algo == GEMM_F32_ALGO_AUTO)
        algo = x->rows <= kFfmaTokens && 1.0 * x->cols * N <= kFfmaOutputs &&
                       1.0 * x->rows * x->cols * N <= kFfmaProducts
                   ? GEMM_F32_ALGO_FFMA
                   : GEMM_F32_ALGO_3XBF16;
    if (algo == GEMM_F32_ALGO_FFMA) return status(launch_q8_wgrad_ffma(a, stream));

    const Q8WgradTile tile = q8_wgrad_tile(false);
    Q8WgradTmemArgs k = {};
    double pair_us, single_us;
    k.share = share_wgrad(a, true, splits, c.sm_count, &pair_us);
    const Q8WgradShare single = share_wgrad(a, false, splits, c.sm_count, &single_us);
    k.pair = algo == GEMM_F32_ALGO_3XBF16 ? pair_us <= single_us
                                          : algo == GEMM_F32_ALGO_3XBF16_PAIR;
    if (!k.pair) k.share = single;
    unsigned char* ws = nullptr;
    if (k.share.shared)
        Q8_TRY(call_workspace(
            c, stream, kWorkspaceCounterBytes + q8_wgrad_parts_bytes(k.share, k.pair), &ws));
    Q8_TRY(map_dy(dY, lddy, x->rows, N, &k));
    Q8_TRY(call_tensor_map(&k.tmC, CU_TENSOR_MAP_DATA_TYPE_UINT8, x->codes, x->cols, x->rows,
                           x->ldcodes, 128, tile.tokens));
    Q8_TRY(call_tensor_map(&k.tmS, CU_TENSOR_MAP_DATA_TYPE_UINT8, x->scales, blocks_of(x->cols),
                           x->rows, x->ldscales, 16, tile.tokens));
    k.dw = dW;
    k.lddw = lddw;
    k.parts = k.share.shared ? reinterpret_cast<float*>(ws + kWorkspaceCounterBytes) : nullptr;
    k.rows = x->rows;
    k.cols = x->cols;
    k.N = N;
    k.format = x->format;
    const int longest = k.share.shared && !k.share.whole
                            ? (k.share.group_stages - 1) / k.share.group_runs + 1
                            : k.share.stages;
    k.chunk = longest <= kWgradShortStages ? kWgradShortChunk : kWgradChunk;
    k.fault = c.fault;
    k.timeout_ns = kDefaultTimeoutNs;
    k.alpha = alpha;
    k.beta = beta;
    k.mode = a.mode;
    return status(launch_q8_wgrad_tmem(k, stream, c.dev, c.sm_count));
}

}  // extern "C"
