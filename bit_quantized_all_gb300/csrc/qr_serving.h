// qr_serving.h -- internal host interface between the C ABI of the serving
// operators (qr_serving_capi.cu) and their translation units.  Arguments
// arrive already validated.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/qr.h"

namespace qrk {

// The packed layout of 4-bit weights: tiles of 16 rows x 64 columns, 512
// bytes of codes each, then per (row tile, group) eight (row g, row g + 8)
// pairs of scales, then as many pairs of zero points.
struct W4Layout {
    int row_tiles, chunks, groups;  // groups covers the padded columns
    size_t scales_at, zeros_at, bytes;
};

inline W4Layout w4_layout(int rows, int cols, int group, bool has_zeros) {
    W4Layout l;
    l.row_tiles = rows / 16 + (rows % 16 != 0);
    l.chunks = cols / 64 + (cols % 64 != 0);
    l.groups = group <= 64 ? l.chunks * (64 / group) : l.chunks / 2 + l.chunks % 2;
    l.scales_at = size_t(l.row_tiles) * size_t(l.chunks) * 512;
    l.zeros_at = l.scales_at + size_t(l.row_tiles) * size_t(l.groups) * 32;
    l.bytes = l.zeros_at + (has_zeros ? size_t(l.row_tiles) * size_t(l.groups) * 16 : 0);
    return l;
}

// Up to so many tokens the product runs on mma.sync, above on tcgen05 (16 and
// 17 tokens through 8192 x 8192: 17 and 22 us).
constexpr int kW4FewTokens = 16;

// Rows of x that 16-byte copies can read.
inline bool w4_x_aligned(const void *x, long long tokens, long long stride) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (tokens == 1 || stride % 8 == 0);
}

struct KvPlanArgs {
    const int32_t *cached, *fresh;
    const int32_t *free_blocks;
    int32_t *table, *q_offsets, *kv_lens, *counts;
    int64_t *slots;
    long long max_tokens;
    int requests, block_size, num_free, width;
};

struct KvAttentionArgs {
    const void *q;
    void *out;
    float *lse;
    const int32_t *q_offsets, *kv_lens, *table;
    long long q_token, q_head, out_token, out_head;  // strides in values
    long long tokens;
    int requests, q_heads, width, causal, window, max_q;
    float scale;
    void *workspace;
};

size_t kv_attention_workspace(int requests, long long tokens, int q_heads, int heads, int head_dim);

cudaError_t launch_kv_plan(const KvPlanArgs &a, cudaStream_t s);
cudaError_t launch_kv_append(int dtype, long long tokens, const void *k, const void *v, long long k_token,
                             long long k_head, long long v_token, long long v_head, const int64_t *slots,
                             const qr_kv_cache_t &cache, cudaStream_t s);
cudaError_t launch_kv_attention(int dtype, const KvAttentionArgs &a, const qr_kv_cache_t &cache, cudaStream_t s);
cudaError_t launch_w4_pack(int rows, int cols, int group, const uint8_t *codes, const void *scales,
                           const uint8_t *zeros, void *packed, cudaStream_t s);
cudaError_t launch_w4_quantize(int dtype, int rows, int cols, int group, const void *w, long long w_stride,
                               void *packed, cudaStream_t s);
cudaError_t launch_w4_matvec(int dtype, long long tokens, const void *x, long long x_stride, int rows, int cols,
                             int group, bool has_zeros, const void *packed, void *y, long long y_stride,
                             void *workspace, cudaStream_t s);

}  // namespace qrk
