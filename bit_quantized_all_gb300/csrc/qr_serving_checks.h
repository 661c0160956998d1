// qr_serving_checks.h -- argument checks that the serving entry points share
// (qr_serving_capi.cu, qr_layer_capi.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/qr.h"

#define QR_EXPORT extern "C" __attribute__((visibility("default")))

namespace qrk {

constexpr int64_t kMostValues = int64_t(1) << 46;  // bound on any offset in values, far from overflow

inline bool dtype_ok(qr_dtype_t d) { return d == QR_FP16 || d == QR_BF16; }
inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}
inline qr_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? QR_OK : QR_ERR_CUDA; }

// A [tokens][heads][dim] operand with strides in values: values from its
// first past its last one, 0 if a stride is out of range.
inline size_t extent_values(int64_t tokens, int heads, int dim, int64_t token_stride, int64_t head_stride) {
    if (heads > 1 && (head_stride < dim || head_stride > kMostValues / heads)) return 0;
    if (tokens > 1 && (token_stride < dim || token_stride > kMostValues / tokens)) return 0;
    return size_t((tokens - 1) * (tokens > 1 ? token_stride : 0) + (heads - 1) * (heads > 1 ? head_stride : 0) + dim);
}
// ... in bytes of 16-bit values
inline size_t extent(int64_t tokens, int heads, int dim, int64_t token_stride, int64_t head_stride) {
    return extent_values(tokens, heads, dim, token_stride, head_stride) * 2;
}

// rows (one per token and head) must not share values with one another
inline bool rows_apart(int64_t tokens, int heads, int dim, int64_t token_stride, int64_t head_stride) {
    if (tokens <= 1 || heads <= 1) return true;
    return token_stride >= (heads - 1) * head_stride + dim || head_stride >= (tokens - 1) * token_stride + dim;
}

}  // namespace qrk
