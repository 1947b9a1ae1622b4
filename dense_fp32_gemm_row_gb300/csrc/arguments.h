// arguments.h -- argument checks that the C ABI files of the 8-bit operators
// share: matrices in memory, and whether they overlap.
#pragma once

#include <cstdint>
#include <limits>

#include <cuda_runtime_api.h>

#include "gemm_f32.h"

namespace gemm_f32_impl {

// A matrix in memory, in bytes: `rows` rows of `width` bytes, `stride` apart.
struct Region {
    const void* base;
    long long rows, width, stride;
};

// Whether two regions share a byte.  Matrices with the same stride may lie
// side by side in the same rows of one buffer (the halves of a wider
// product): then they are apart when their columns are.  With different
// strides, address ranges that meet count as shared.
inline bool share(const Region& a, const Region& b) {
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

inline bool bad_dims(long long rows, long long cols, long long ld) {
    return ld < (cols > 1 ? cols : 1) ||
           (rows > 0 && ld > std::numeric_limits<long long>::max() / 16 / rows);
}

// A float (or, elem = 2, bf16) matrix argument: pointer present and aligned
// to its element, row stride at least the row.
inline int check_matrix(const void* p, long long rows, long long cols, long long ld, int elem) {
    if (bad_dims(rows, cols, ld) || !p) return GEMM_F32_ERR_INVALID_VALUE;
    if (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(elem - 1))
        return GEMM_F32_ERR_INVALID_VALUE;
    return GEMM_F32_SUCCESS;
}

inline Region region(const void* p, long long rows, long long cols, long long ld, int elem) {
    return {p, rows, cols * elem, ld * elem};
}

// Outputs that share memory with one another or with an input.
inline int check_apart(const Region* out, int nout, const Region* in, int nin) {
    for (int i = 0; i < nout; ++i) {
        for (int j = i + 1; j < nout; ++j)
            if (share(out[i], out[j])) return GEMM_F32_ERR_INVALID_VALUE;
        for (int j = 0; j < nin; ++j)
            if (share(out[i], in[j])) return GEMM_F32_ERR_INVALID_VALUE;
    }
    return GEMM_F32_SUCCESS;
}

inline int status(cudaError_t e) {
    return e == cudaSuccess ? GEMM_F32_SUCCESS : static_cast<int>(e);
}

}  // namespace gemm_f32_impl
