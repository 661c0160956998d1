// qr_serving_capi.cu -- the extern "C" entry points of the serving operators
// (include/qr.h): host-side argument validation, then a launch on the
// caller's stream.  As for the codec, validation runs before any CUDA call.
//
// Checks, in this order (the first failure is returned):
//   1. null pointers, counts below 1                        -> QR_ERR_INVALID_ARG
//   2. dtypes, head sizes, block sizes, groups not served   -> QR_ERR_UNSUPPORTED
//   3. sizes that overflow, strides below a row, a workspace too small
//                                                           -> QR_ERR_SIZE
//   4. misaligned pointers or strides                       -> QR_ERR_MISALIGNED
//   5. an output overlapping an input                       -> QR_ERR_INVALID_ARG
#include <climits>

#include "qr_serving.h"
#include "qr_serving_checks.h"

namespace {

using namespace qrk;

bool block_size_ok(int b) { return b == 16 || b == 32 || b == 64 || b == 128 || b == 256; }
bool head_dim_ok(int d) { return d >= 16 && d <= 256 && d % 16 == 0; }
bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }

// Checks of the cache that need no call-specific operand; QR_OK or the error.
qr_status_t check_cache(const qr_kv_cache_t *c) {
    if (!c || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return QR_ERR_INVALID_ARG;
    if (c->blocks < 1 || c->heads < 1 || c->block_size < 1 || c->head_dim < 1) return QR_ERR_INVALID_ARG;
    if (!block_size_ok(c->block_size) || !head_dim_ok(c->head_dim) || c->heads > 65535) return QR_ERR_UNSUPPORTED;
    const int64_t page = int64_t(c->block_size) * c->head_dim;
    const int64_t strides[2][2] = {{c->k_block_stride, c->k_head_stride}, {c->v_block_stride, c->v_head_stride}};
    for (const auto &s : strides) {
        if (c->heads > 1 && (s[1] < page || s[1] > kMostValues / c->heads)) return QR_ERR_SIZE;
        if (c->blocks > 1 && (s[0] < page || s[0] > kMostValues / c->blocks)) return QR_ERR_SIZE;
        if (c->heads > 1 && c->blocks > 1 && s[0] < (c->heads - 1) * s[1] + page &&
            s[1] < (c->blocks - 1) * s[0] + page)
            return QR_ERR_SIZE;  // pages that overlap
    }
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4))
        return QR_ERR_MISALIGNED;
    for (const auto &s : strides)
        if ((c->heads > 1 && s[1] % 16) || (c->blocks > 1 && s[0] % 16)) return QR_ERR_MISALIGNED;
    return QR_OK;
}

size_t cache_extent(const qr_kv_cache_t &c, int64_t block_stride, int64_t head_stride) {
    return size_t((c.blocks > 1 ? (c.blocks - 1) * block_stride : 0) + (c.heads > 1 ? (c.heads - 1) * head_stride : 0) +
                  int64_t(c.block_size) * c.head_dim);
}

}  // namespace

QR_EXPORT qr_status_t qr_kv_plan(int requests, const int32_t *cached_lens, const int32_t *new_lens, int block_size,
                                 const int32_t *free_blocks, int num_free, int32_t *block_table, int table_width,
                                 int32_t *q_offsets, int32_t *kv_lens, int64_t *slots, int64_t max_tokens,
                                 int32_t *counts, qr_stream_t stream) {
    if (!cached_lens || !new_lens || !block_table || !q_offsets || !kv_lens || !counts) return QR_ERR_INVALID_ARG;
    if (requests < 1 || table_width < 1 || num_free < 0 || max_tokens < 0) return QR_ERR_INVALID_ARG;
    if ((num_free > 0 && !free_blocks) || (max_tokens > 0 && !slots)) return QR_ERR_INVALID_ARG;
    if (!block_size_ok(block_size) || requests > 65536) return QR_ERR_UNSUPPORTED;
    if (max_tokens > INT_MAX) return QR_ERR_SIZE;
    if (!aligned(cached_lens, 4) || !aligned(new_lens, 4) || !aligned(free_blocks, 4) || !aligned(block_table, 4) ||
        !aligned(q_offsets, 4) || !aligned(kv_lens, 4) || !aligned(counts, 4) || !aligned(slots, 8))
        return QR_ERR_MISALIGNED;
    const size_t lens = size_t(requests) * 4;
    const struct { const void *p; size_t n; } in[3] = {{cached_lens, lens}, {new_lens, lens}, {free_blocks, size_t(num_free) * 4}},
        out[5] = {{block_table, size_t(requests) * size_t(table_width) * 4}, {q_offsets, lens + 4}, {kv_lens, lens},
                  {slots, size_t(max_tokens) * 8}, {counts, 16}};
    for (int i = 0; i < 5; ++i) {
        for (const auto &x : in)
            if (x.n && out[i].n && overlaps(out[i].p, out[i].n, x.p, x.n)) return QR_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (out[i].n && out[j].n && overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return QR_ERR_INVALID_ARG;
    }
    return from_cuda(qrk::launch_kv_plan({cached_lens, new_lens, free_blocks, block_table, q_offsets, kv_lens, counts,
                                          slots, max_tokens, requests, block_size, num_free, table_width},
                                         reinterpret_cast<cudaStream_t>(stream)));
}

QR_EXPORT qr_status_t qr_kv_append(qr_dtype_t dtype, int64_t tokens, const void *k, const void *v,
                                   int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                                   int64_t v_head_stride, const int64_t *slots, const qr_kv_cache_t *cache,
                                   qr_stream_t stream) {
    if (!k || !v || !slots || !cache || tokens < 1) return QR_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return QR_ERR_UNSUPPORTED;
    const qr_status_t st = check_cache(cache);
    if (st != QR_OK) return st;
    if (tokens > INT_MAX) return QR_ERR_SIZE;
    const size_t nk = extent(tokens, cache->heads, cache->head_dim, k_token_stride, k_head_stride);
    const size_t nv = extent(tokens, cache->heads, cache->head_dim, v_token_stride, v_head_stride);
    if (nk == 0 || nv == 0) return QR_ERR_SIZE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return QR_ERR_MISALIGNED;
    if (tokens > 1 && (k_token_stride % 8 || v_token_stride % 8)) return QR_ERR_MISALIGNED;
    if (cache->heads > 1 && (k_head_stride % 8 || v_head_stride % 8)) return QR_ERR_MISALIGNED;
    const size_t scales = size_t(cache->blocks) * size_t(cache->heads) * 4;
    const struct { const void *p; size_t n; } in[3] = {{k, nk}, {v, nv}, {slots, size_t(tokens) * 8}},
        out[4] = {{cache->k_codes, cache_extent(*cache, cache->k_block_stride, cache->k_head_stride)},
                  {cache->v_codes, cache_extent(*cache, cache->v_block_stride, cache->v_head_stride)},
                  {cache->k_scales, scales}, {cache->v_scales, scales}};
    for (const auto &o : out)
        for (const auto &x : in)
            if (overlaps(o.p, o.n, x.p, x.n)) return QR_ERR_INVALID_ARG;
    return from_cuda(qrk::launch_kv_append(dtype, tokens, k, v, k_token_stride, k_head_stride, v_token_stride,
                                           v_head_stride, slots, *cache, reinterpret_cast<cudaStream_t>(stream)));
}

namespace {

size_t attention_workspace(int requests, int64_t tokens, int q_heads, int heads, int head_dim) {
    if (requests < 1 || requests > 65536 || tokens < 1 || tokens > (1 << 30) || heads < 1 || heads > 65535 ||
        q_heads < heads || q_heads % heads || q_heads > 65535 || !head_dim_ok(head_dim))
        return 0;
    return qrk::kv_attention_workspace(requests, tokens, q_heads, heads, head_dim);
}

}  // namespace

QR_EXPORT size_t qr_kv_attention_workspace_bytes(int requests, int64_t tokens, int q_heads, int heads, int head_dim) {
    return attention_workspace(requests, tokens, q_heads, heads, head_dim);
}

QR_EXPORT qr_status_t qr_kv_attention(qr_dtype_t dtype, int requests, int64_t tokens, int q_heads, const void *q,
                                      int64_t q_token_stride, int64_t q_head_stride, const int32_t *q_offsets,
                                      const int32_t *kv_lens, const int32_t *block_table, int table_width,
                                      const qr_kv_cache_t *cache, float scale, int causal, int window, int max_q,
                                      void *out, int64_t out_token_stride, int64_t out_head_stride, float *lse,
                                      void *workspace, size_t workspace_bytes, qr_stream_t stream) {
    if (!q || !q_offsets || !kv_lens || !block_table || !cache || !out || !workspace) return QR_ERR_INVALID_ARG;
    if (requests < 1 || tokens < 1 || q_heads < 1 || table_width < 1 || max_q < 1 || window < 0)
        return QR_ERR_INVALID_ARG;
    if ((window > 0 && !causal) || !(scale == scale) || scale - scale != 0.0f) return QR_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return QR_ERR_UNSUPPORTED;
    const qr_status_t st = check_cache(cache);
    if (st != QR_OK) return st;
    if (requests > 65536 || q_heads % cache->heads || q_heads > 65535) return QR_ERR_UNSUPPORTED;
    // positions minus a window stay within an int
    constexpr int kFar = 1 << 30;
    if (int64_t(table_width) * cache->block_size > INT_MAX - 512 || tokens > kFar ||
        tokens * (q_heads / cache->heads) > kFar)
        return QR_ERR_SIZE;
    const size_t need = attention_workspace(requests, tokens, q_heads, cache->heads, cache->head_dim);
    const size_t nq = extent(tokens, q_heads, cache->head_dim, q_token_stride, q_head_stride);
    const size_t no = extent(tokens, q_heads, cache->head_dim, out_token_stride, out_head_stride);
    if (need == 0 || nq == 0 || no == 0 || workspace_bytes < need) return QR_ERR_SIZE;
    if (!rows_apart(tokens, q_heads, cache->head_dim, out_token_stride, out_head_stride)) return QR_ERR_SIZE;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(q_offsets, 4) ||
        !aligned(kv_lens, 4) || !aligned(block_table, 4) || !aligned(lse, 4))
        return QR_ERR_MISALIGNED;
    if (tokens > 1 && (q_token_stride % 8 || out_token_stride % 8)) return QR_ERR_MISALIGNED;
    if (q_heads > 1 && (q_head_stride % 8 || out_head_stride % 8)) return QR_ERR_MISALIGNED;
    const size_t scales = size_t(cache->blocks) * size_t(cache->heads) * 4, nl = size_t(tokens) * size_t(q_heads) * 4;
    const struct { const void *p; size_t n; } in[8] = {
        {q, nq}, {q_offsets, size_t(requests) * 4 + 4}, {kv_lens, size_t(requests) * 4},
        {block_table, size_t(requests) * size_t(table_width) * 4},
        {cache->k_codes, cache_extent(*cache, cache->k_block_stride, cache->k_head_stride)},
        {cache->v_codes, cache_extent(*cache, cache->v_block_stride, cache->v_head_stride)},
        {cache->k_scales, scales}, {cache->v_scales, scales}},
        outs[3] = {{out, no}, {workspace, need}, {lse, lse ? nl : 0}};
    for (int i = 0; i < 3; ++i) {
        for (const auto &x : in)
            if (outs[i].n && overlaps(outs[i].p, outs[i].n, x.p, x.n)) return QR_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (outs[i].n && overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return QR_ERR_INVALID_ARG;
    }
    // no request has more queries than there are tokens: the workspace is sized
    // by these, so the kernel is picked by no larger number
    const int most_q = max_q < tokens ? max_q : static_cast<int>(tokens);
    return from_cuda(qrk::launch_kv_attention(
        dtype, {q, out, lse, q_offsets, kv_lens, block_table, q_token_stride, q_head_stride, out_token_stride,
                out_head_stride, tokens, requests, q_heads, table_width, causal != 0, window < kFar ? window : kFar, most_q,
                scale, workspace},
        *cache, reinterpret_cast<cudaStream_t>(stream)));
}

QR_EXPORT size_t qr_w4_bytes(int rows, int cols, int group, int has_zeros) {
    if (rows < 1 || cols < 1 || rows > INT_MAX - 64 || cols > INT_MAX - 128 || !group_ok(group)) return 0;
    return qrk::w4_layout(rows, cols, group, has_zeros != 0).bytes;
}

QR_EXPORT qr_status_t qr_w4_pack(int rows, int cols, int group, const uint8_t *codes, const void *scales,
                                 const uint8_t *zeros, void *packed, qr_stream_t stream) {
    if (!codes || !scales || !packed || rows < 1 || cols < 1) return QR_ERR_INVALID_ARG;
    if (!group_ok(group)) return QR_ERR_UNSUPPORTED;
    const size_t need = qr_w4_bytes(rows, cols, group, zeros != nullptr);
    if (need == 0) return QR_ERR_SIZE;
    if (!aligned(packed, 16) || !aligned(scales, 2)) return QR_ERR_MISALIGNED;
    const size_t groups = size_t(cols / group + (cols % group != 0)) * size_t(rows);
    if (overlaps(packed, need, codes, size_t(rows) * size_t(cols / 2 + cols % 2)) ||
        overlaps(packed, need, scales, groups * 2) || (zeros && overlaps(packed, need, zeros, groups)))
        return QR_ERR_INVALID_ARG;
    return from_cuda(qrk::launch_w4_pack(rows, cols, group, codes, scales, zeros, packed,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

QR_EXPORT qr_status_t qr_w4_quantize(qr_dtype_t dtype, int rows, int cols, int group, const void *w,
                                     int64_t w_row_stride, void *packed, qr_stream_t stream) {
    if (!w || !packed || rows < 1 || cols < 1) return QR_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || !group_ok(group)) return QR_ERR_UNSUPPORTED;
    const size_t need = qr_w4_bytes(rows, cols, group, 0), nw = extent(rows, 1, cols, w_row_stride, 0);
    if (need == 0 || nw == 0) return QR_ERR_SIZE;
    if (!aligned(packed, 16) || !aligned(w, 2)) return QR_ERR_MISALIGNED;
    if (overlaps(packed, need, w, nw)) return QR_ERR_INVALID_ARG;
    return from_cuda(qrk::launch_w4_quantize(dtype, rows, cols, group, w, w_row_stride, packed,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

QR_EXPORT size_t qr_w4_matvec_workspace_bytes(int64_t tokens, int cols) {
    if (tokens < 1 || tokens > INT_MAX || cols < 1 || cols > INT_MAX - 128) return 0;
    return size_t(tokens) * (size_t(cols) / 64 + (cols % 64 != 0)) * 128;
}

QR_EXPORT qr_status_t qr_w4_matvec(qr_dtype_t dtype, int64_t tokens, const void *x, int64_t x_row_stride, int rows,
                                   int cols, int group, int has_zeros, const void *packed, void *y,
                                   int64_t y_row_stride, void *workspace, size_t workspace_bytes, qr_stream_t stream) {
    if (!x || !packed || !y || tokens < 1 || rows < 1 || cols < 1) return QR_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || !group_ok(group)) return QR_ERR_UNSUPPORTED;
    const size_t need = qr_w4_bytes(rows, cols, group, has_zeros);
    if (need == 0 || tokens > INT_MAX) return QR_ERR_SIZE;
    const size_t nx = extent(tokens, 1, cols, x_row_stride, 0), ny = extent(tokens, 1, rows, y_row_stride, 0);
    if (nx == 0 || ny == 0) return QR_ERR_SIZE;
    const bool copies = tokens > qrk::kW4FewTokens && !qrk::w4_x_aligned(x, tokens, x_row_stride);
    const size_t nw = copies ? qr_w4_matvec_workspace_bytes(tokens, cols) : 0;
    if (copies && (!workspace || workspace_bytes < nw)) return QR_ERR_SIZE;
    if (!aligned(packed, 16) || !aligned(x, 2) || !aligned(y, 2) || (copies && !aligned(workspace, 16)))
        return QR_ERR_MISALIGNED;
    if (overlaps(y, ny, x, nx) || overlaps(y, ny, packed, need)) return QR_ERR_INVALID_ARG;
    if (copies && (overlaps(workspace, nw, x, nx) || overlaps(workspace, nw, packed, need) || overlaps(workspace, nw, y, ny)))
        return QR_ERR_INVALID_ARG;
    return from_cuda(qrk::launch_w4_matvec(dtype, tokens, x, x_row_stride, rows, cols, group, has_zeros != 0, packed, y,
                                           y_row_stride, workspace, reinterpret_cast<cudaStream_t>(stream)));
}
