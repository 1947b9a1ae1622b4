// i8_api.cu -- the C ABI of the 8-bit integer linear layers: argument checks,
// the edge rules and kernel dispatch.  Empty matrices are a successful no-op,
// as in the GEMM entry points; nothing here exits the process.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>

#include "arguments.h"
#include "gemm_f32.h"
#include "gemm_internal.h"

using namespace gemm_f32_impl;

#define I8_TRY(expr)                                  \
    do {                                              \
        const int st_ = (expr);                       \
        if (st_ != GEMM_F32_SUCCESS) return st_;      \
    } while (0)

namespace {

int check_shape(const gemm_f32_i8* q) {
    return q && q->rows >= 0 && q->cols >= 0 ? GEMM_F32_SUCCESS : GEMM_F32_ERR_INVALID_VALUE;
}

// The arrays of a matrix with elements: codes 16-byte aligned with a row stride
// that is a multiple of 16 bytes and holds a row.
int check_arrays(const gemm_f32_i8* q) {
    if (!q->codes || !q->scales) return GEMM_F32_ERR_INVALID_VALUE;
    if ((reinterpret_cast<uintptr_t>(q->codes) & 15u) || (q->ld & 15) ||
        (reinterpret_cast<uintptr_t>(q->scales) & 3u))
        return GEMM_F32_ERR_INVALID_VALUE;
    return bad_dims(q->rows, q->cols, q->ld) ? GEMM_F32_ERR_INVALID_VALUE : GEMM_F32_SUCCESS;
}

Region codes_of(const gemm_f32_i8* q) { return region(q->codes, q->rows, q->cols, q->ld, 1); }
Region scales_of(const gemm_f32_i8* q) { return region(q->scales, 1, q->rows, q->rows, 4); }

I8In in_of(const gemm_f32_i8* q) { return {q->codes, q->scales, q->ld}; }

int elem_of(int type) { return type == GEMM_F32_TYPE_BF16 ? 2 : 4; }
bool is_float(int type) { return type == GEMM_F32_TYPE_F32 || type == GEMM_F32_TYPE_BF16; }

int map_codes(CUtensorMap* map, const gemm_f32_i8* q, int k, int rows) {
    return call_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, q->codes, q->cols, q->rows, q->ld, k,
                           rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The tensor-core kernel's times in microseconds, fitted to 3600 calls back to
// back with each form forced (T 9 .. 1024, N 256 .. 16384, K 512 .. 14336, weights
// from DRAM; within 4 to 7 % of them on average): a launch, a stage of 128 columns
// of K and its part for each of a CTA's tokens, a tile and its part a token,
// joining splits in a cluster and each of them, and the same through the workspace.
// Below these, what the weights take from DRAM.  Choices by them take 0.9 % longer
// than the best of all forms, on average of 234 sizes.
struct I8Times {
    float launch, stage, stage_token, tile, tile_token, join, each_join, split, each_split;
};
constexpr I8Times kI8Pair = {4.3f, 0.43f, 0.0016f, 0.5f, 0.0193f, 0.0f, 0.0f, 0.0f, 0.0f};
constexpr I8Times kI8Wide = {3.3f, 0.445f, 0.0001f, 0.0f, 0.016f, 0.6f, 0.9f, 1.9f, 0.97f};
constexpr I8Times kI8Narrow = {3.2f, 0.275f, 0.0002f, 0.27f, 0.0227f, 1.0f, 0.2f, 2.7f, 0.31f};
constexpr float kI8WeightsUsPerMb = 0.19f;
// The same for the kernel for a few tokens: a launch, and a thousand codes of the
// weights that the busiest SM reads, for 9 to 16, 24 and 32 tokens (24 x 8192 x 8192
// 19.2 us, by single CTAs in two splits 16.7; 9 tokens 15.1 and 16.2).  Fitted when
// copies of any size made each step longer: large layers now take up to a seventh less
// than this says, small ones, which end far below the other form's, a third less.
constexpr float kI8StreamLaunch = 3.3f;
constexpr float kI8StreamUsPerK[kI8StreamTokens / 8 - 1] = {0.0245f, 0.0327f, 0.037f};
constexpr int kI8MostSplits = 16;    // that the library chooses
constexpr int kI8NarrowTokens = 64;  // of a CTA, from which on its form is the wide one
constexpr int kI8MostRows = 2147483647 - 1023;
constexpr int kI8MostSplitTiles = kWorkspaceCounterBytes / 4 / kI8CountersPerTile;

int div_up(int a, int b) { return (a - 1) / b + 1; }
int to_16(int a) { return (a + 15) & ~15; }
// the fewest tokens a tile, of at most `most`, that make as few tiles
int even_share(int T, int most) { return to_16(div_up(T, div_up(T, most))); }

struct I8Choice {
    I8Share share;
    bool pair;
    float us;
};

// One way to share a product out, if it is faster than the best so far.
void consider(int T, int N, int K, bool gated, bool pair, int tokens, int splits, int dev,
              int sm_count, I8Choice* best) {
    const I8Tile t = i8_tile(pair);
    const I8Times& time = pair ? kI8Pair : tokens > kI8NarrowTokens ? kI8Wide : kI8Narrow;
    I8Share s = {};
    s.tokens = tokens;
    s.tiles_c = div_up(N, gated ? t.channels / 2 : t.channels);
    s.tiles_t = div_up(T, pair ? 2 * tokens : tokens);
    s.stages = div_up(K, t.k);
    s.splits = std::min(splits, s.stages);
    const long long tiles = static_cast<long long>(s.tiles_c) * s.tiles_t;
    if (tiles > kI8MostSplitTiles) s.splits = 1;
    // requested splits: no more than keep the workspace within bounds
    while (s.splits > 1 && tiles * s.splits > 16LL * sm_count) --s.splits;
    if (s.splits > 1 && i8_joins_in_clusters(s.splits, tokens) &&
        tiles <= i8_most_clusters(s.splits, dev))
        s.clusters = 1;
    const long long rounds = (tiles * s.splits - 1) / (pair ? sm_count / 2 : sm_count) + 1;
    const float loop = rounds * (div_up(s.stages, s.splits) * (time.stage + time.stage_token * tokens) +
                                 time.tile + time.tile_token * tokens);
    const float weights = kI8WeightsUsPerMb * 1e-6f * N * K * (gated ? 2 : 1);
    const float join = s.splits == 1 ? 0.0f
                       : s.clusters  ? time.join + time.each_join * s.splits
                                     : time.split + time.each_split * s.splits;
    const float us = time.launch + std::max(loop, weights) + join;
    if (us < best->us) *best = {s, pair, us};
}

// How a product is shared out: a few tile widths of each form, whole or split so
// that a round's units fill the SMs or half of them, or in as many clusters as run
// at once, whichever should be fastest.
I8Choice share_out(int T, int N, int K, bool gated, int algo, int splits, int dev,
                   int sm_count) {
    I8Choice best = {};
    best.us = std::numeric_limits<float>::max();
    const auto single = [&](int tokens) {
        const I8Tile t = i8_tile(false);
        const long long tiles = static_cast<long long>(div_up(N, gated ? t.channels / 2 : t.channels)) *
                                div_up(T, tokens);
        if (splits > 0) return consider(T, N, K, gated, false, tokens, splits, dev, sm_count, &best);
        const int most = std::min<long long>(std::min(div_up(K, t.k) / 2, kI8MostSplits),
                                             sm_count / tiles);
        consider(T, N, K, gated, false, tokens, 1, dev, sm_count, &best);
        if (most > 1) consider(T, N, K, gated, false, tokens, most, dev, sm_count, &best);
        if (most > 2) consider(T, N, K, gated, false, tokens, (most + 1) / 2, dev, sm_count, &best);
        for (int n = std::min(most, 8); n > 1; --n)
            if (i8_joins_in_clusters(n, tokens) && tiles <= i8_most_clusters(n, dev)) {
                if (n != most) consider(T, N, K, gated, false, tokens, n, dev, sm_count, &best);
                break;
            }
    };
    if (algo != GEMM_F32_ALGO_I8_SINGLE) {
        const int tokens = to_16(div_up(even_share(T, 256), 2));
        consider(T, N, K, gated, true, tokens, 1, dev, sm_count, &best);
        if (tokens > 96) consider(T, N, K, gated, true, 96, 1, dev, sm_count, &best);
        if (tokens > 64) consider(T, N, K, gated, true, 64, 1, dev, sm_count, &best);
    }
    if (algo != GEMM_F32_ALGO_I8_PAIR) {
        const int tokens = even_share(T, kI8NarrowTokens);
        if (T > kI8NarrowTokens) single(even_share(T, 128));
        single(tokens);
        if (tokens > 48) single(48);
        if (tokens > 32) single(32);
        if (tokens > 16) single(16);
    }
    return best;
}

// Both products: y = a b^T, or with c the gated product of b and c.
int product(const gemm_f32_i8* a, const gemm_f32_i8* b, const gemm_f32_i8* c, int act, void* Y,
            int type, long long ldy, int algo, int splits, cudaStream_t stream) {
    if ((algo != GEMM_F32_ALGO_AUTO &&
         (algo < GEMM_F32_ALGO_I8_PAIR || algo > GEMM_F32_ALGO_I8_STREAM)) ||
        splits < 0 || splits > GEMM_F32_MAX_SPLITS)
        return GEMM_F32_ERR_INVALID_VALUE;
    I8_TRY(check_shape(a));
    I8_TRY(check_shape(b));
    if (a->cols != b->cols || a->cols > GEMM_F32_I8_MAX_COLS) return GEMM_F32_ERR_INVALID_VALUE;
    if (c) {
        I8_TRY(check_shape(c));
        if (c->rows != b->rows || c->cols != b->cols) return GEMM_F32_ERR_INVALID_VALUE;
    }
    const int T = a->rows, N = b->rows, K = a->cols;
    if (algo == GEMM_F32_ALGO_I8_STREAM && T > kI8StreamTokens) return GEMM_F32_ERR_INVALID_VALUE;
    if (T == 0 || N == 0) return GEMM_F32_SUCCESS;
    // more tiles than an index holds (no memory does either), or rows whose
    // number plus a tile's it does not
    if (1.0 * T * N > 1e12 || T > kI8MostRows || N > kI8MostRows) return GEMM_F32_ERR_INVALID_VALUE;
    I8_TRY(check_matrix(Y, T, N, ldy, elem_of(type)));
    if (K > 0) {
        I8_TRY(check_arrays(a));
        I8_TRY(check_arrays(b));
        if (c) I8_TRY(check_arrays(c));
        const Region out[] = {region(Y, T, N, ldy, elem_of(type))};
        const Region in[] = {codes_of(a), scales_of(a), codes_of(b), scales_of(b),
                             c ? codes_of(c) : Region{}, c ? scales_of(c) : Region{}};
        I8_TRY(check_apart(out, 1, in, 6));
    }
    std::lock_guard<std::mutex> lock(api_mutex());
    CallState s;
    I8_TRY(call_state(stream, &s));
    if (K == 0)
        return status(launch_zero_rows(Y, ldy * elem_of(type), T,
                                       static_cast<long long>(N) * elem_of(type), stream));
    I8Choice how = {};
    bool stream_form = algo == GEMM_F32_ALGO_I8_STREAM || (algo == GEMM_F32_ALGO_AUTO && T <= 8);
    if (!stream_form) {
        how = share_out(T, N, K, c != nullptr, algo, splits, s.dev, s.sm_count);
        if (algo == GEMM_F32_ALGO_AUTO && T <= kI8StreamTokens) {
            const float codes = 1e-3f * K * i8_stream_channels(T, N, c != nullptr, s.sm_count);
            stream_form = kI8StreamLaunch + kI8StreamUsPerK[(T - 9) / 8] * codes < how.us;
        }
    }
    if (stream_form) {
        const I8StreamArgs p = {in_of(a), in_of(b), c ? in_of(c) : I8In{}, Y, ldy, T, N, K, type,
                                c ? act : -1};
        return status(launch_i8_stream(p, stream, s.dev, s.sm_count));
    }
    const bool pair = how.pair;
    I8TmemArgs k = {};
    k.share = how.share;
    unsigned char* ws = nullptr;
    if (k.share.splits > 1 && !k.share.clusters)
        I8_TRY(call_workspace(s, stream, kWorkspaceCounterBytes + i8_parts_bytes(k.share), &ws));
    const I8Tile tile = i8_tile(pair);
    const int rows = c ? 64 : 128;
    I8TmemMaps maps = {};
    I8_TRY(map_codes(&maps.a, a, tile.k, k.share.tokens));
    I8_TRY(map_codes(&maps.b, b, tile.k, rows));
    if (c) I8_TRY(map_codes(&maps.c, c, tile.k, rows));
    k.as = a->scales;
    k.bs = b->scales;
    k.cs = c ? c->scales : nullptr;
    k.y = Y;
    k.ldy = ldy;
    k.T = T;
    k.N = N;
    k.type = type;
    k.counters = reinterpret_cast<int*>(ws);
    k.parts = reinterpret_cast<int*>(ws + kWorkspaceCounterBytes);
    k.fault = s.fault;
    k.timeout_ns = kDefaultTimeoutNs;
    return status(launch_i8_tmem(maps, k, pair, c ? act : -1, stream, s.dev, s.sm_count));
}

}  // namespace

extern "C" {

int gemm_f32_i8_store(const void* X, int type, long long ldx, const gemm_f32_i8* q,
                      cudaStream_t stream) {
    if (!is_float(type)) return GEMM_F32_ERR_INVALID_VALUE;
    I8_TRY(check_shape(q));
    if (q->rows == 0 || q->cols == 0) return GEMM_F32_SUCCESS;
    I8_TRY(check_arrays(q));
    I8_TRY(check_matrix(X, q->rows, q->cols, ldx, elem_of(type)));
    const Region out[] = {codes_of(q), scales_of(q)};
    const Region in[] = {region(X, q->rows, q->cols, ldx, elem_of(type))};
    I8_TRY(check_apart(out, 2, in, 1));
    std::lock_guard<std::mutex> lock(api_mutex());
    CallState s;
    I8_TRY(call_state(stream, &s));
    I8RowsArgs a = {};
    a.x = X;
    a.ldx = ldx;
    a.codes = q->codes;
    a.scales = q->scales;
    a.ldq = q->ld;
    a.rows = q->rows;
    a.cols = q->cols;
    a.bf16 = type == GEMM_F32_TYPE_BF16;
    return status(launch_i8_rows(a, stream, s.sm_count));
}

int gemm_f32_i8_norm(const void* X, long long ldx, const void* R, long long ldr, const void* W,
                     float eps, int type, void* S, long long lds, const gemm_f32_i8* q,
                     cudaStream_t stream) {
    if (!is_float(type) || !(eps >= GEMM_F32_I8_LEAST_EPS) || !std::isfinite(eps) || (S && !R))
        return GEMM_F32_ERR_INVALID_VALUE;
    I8_TRY(check_shape(q));
    const int rows = q->rows, cols = q->cols, elem = elem_of(type);
    if (rows == 0 || cols == 0) return GEMM_F32_SUCCESS;
    I8_TRY(check_arrays(q));
    I8_TRY(check_matrix(X, rows, cols, ldx, elem));
    I8_TRY(check_matrix(W, 1, cols, cols, elem));
    if (R) I8_TRY(check_matrix(R, rows, cols, ldr, elem));
    if (S) I8_TRY(check_matrix(S, rows, cols, lds, elem));
    const Region out[] = {codes_of(q), scales_of(q), region(S, rows, cols, lds, elem)};
    const Region in[] = {region(X, rows, cols, ldx, elem), region(R, rows, cols, ldr, elem),
                         region(W, 1, cols, cols, elem)};
    I8_TRY(check_apart(out, 3, in, 3));
    std::lock_guard<std::mutex> lock(api_mutex());
    CallState s;
    I8_TRY(call_state(stream, &s));
    const I8RowsArgs a = {X, R, W, S, ldx, ldr, lds, q->codes, q->scales, q->ld, rows, cols,
                          type == GEMM_F32_TYPE_BF16, eps};
    return status(launch_i8_rows(a, stream, s.sm_count));
}

int gemm_f32_i8_matmul(const gemm_f32_i8* a, const gemm_f32_i8* b, void* Y, int type,
                       long long ldy, int algo, int splits, cudaStream_t stream) {
    if (!is_float(type) && type != GEMM_F32_TYPE_I32) return GEMM_F32_ERR_INVALID_VALUE;
    return product(a, b, nullptr, 0, Y, type, ldy, algo, splits, stream);
}

int gemm_f32_i8_gated(int act, const gemm_f32_i8* a, const gemm_f32_i8* gate,
                      const gemm_f32_i8* up, void* H, int type, long long ldh, int algo,
                      int splits, cudaStream_t stream) {
    if ((act != GEMM_F32_ACT_SILU && act != GEMM_F32_ACT_GELU) || !is_float(type) || !up)
        return GEMM_F32_ERR_INVALID_VALUE;
    return product(a, gate, up, act, H, type, ldh, algo, splits, stream);
}

}  // extern "C"
