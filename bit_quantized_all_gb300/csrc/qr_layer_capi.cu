// qr_layer_capi.cu -- the extern "C" entry points of the norm, the rotary
// positions and the 8-bit product (include/qr.h).  Checks as in
// qr_serving_capi.cu and in the same order; validation runs before any CUDA
// call.
#include <climits>

#include "qr_serving.h"
#include "qr_serving_checks.h"

namespace {

using namespace qrk;

cudaError_t launch_norm(int dtype, int weight, const NormArgs &a, cudaStream_t s) {
    return dtype ? launch_norm_typed<1>(weight, a, s) : launch_norm_typed<0>(weight, a, s);
}

constexpr int kMostCols = 1 << 30;  // so that a loop over a row's values ends below 2^31

cudaStream_t stream_of(qr_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Rows of `width` bytes, `stride` bytes apart.
struct Rows {
    const void *p;
    int64_t rows, stride, width;

    size_t bytes() const { return size_t((rows - 1) * (rows > 1 ? stride : 0) + width); }
};

// No byte in common: the spans are apart, or the rows of one lie between those
// of the other (slices of the same wider rows).
bool apart(const Rows &a, const Rows &b) {
    if (!a.p || !b.p || !overlaps(a.p, a.bytes(), b.p, b.bytes())) return true;
    if (a.rows == 1 || b.rows == 1 || a.stride != b.stride) return false;
    const int64_t s = a.stride;
    if (a.width > s || b.width > s) return false;
    const int64_t d = ((int64_t(reinterpret_cast<uintptr_t>(b.p)) - int64_t(reinterpret_cast<uintptr_t>(a.p))) % s + s) % s;
    return d >= a.width && s - d >= b.width;
}
bool same(const Rows &a, const Rows &b) { return a.p == b.p && (a.rows <= 1 || a.stride == b.stride); }

Rows flat(const void *p, size_t bytes) { return {p, 1, 0, int64_t(bytes)}; }

qr_status_t norm(qr_dtype_t dtype, int64_t tokens, int cols, const void *x, int64_t x_row, const void *residual,
                 int64_t residual_row, void *residual_out, int64_t residual_out_row, const void *weight, int weight_fp32,
                 float eps, bool eight, void *y, int64_t y_row, float *scales, qr_stream_t stream) {
    if (!x || !weight || !y || (eight && !scales) || (residual_out && !residual)) return QR_ERR_INVALID_ARG;
    if (tokens < 1 || cols < 1 || !(eps > 0.0f) || eps - eps != 0.0f) return QR_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return QR_ERR_UNSUPPORTED;
    if (tokens > INT_MAX || cols > kMostCols) return QR_ERR_SIZE;
    if (!extent(tokens, 1, cols, x_row, 0) || !extent(tokens, 1, cols, y_row, 0) ||
        (residual && !extent(tokens, 1, cols, residual_row, 0)) ||
        (residual_out && !extent(tokens, 1, cols, residual_out_row, 0)))
        return QR_ERR_SIZE;
    if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(residual_out, 2) || !aligned(weight, weight_fp32 ? 4 : 2) ||
        !aligned(y, eight ? 16 : 2) || !aligned(scales, 4) || (eight && tokens > 1 && y_row % 16))
        return QR_ERR_MISALIGNED;
    const Rows in[2] = {{x, tokens, x_row * 2, cols * 2ll}, {residual, tokens, residual_row * 2, cols * 2ll}};
    const Rows w = flat(weight, size_t(cols) * (weight_fp32 ? 4 : 2));
    const Rows out[3] = {{residual_out, tokens, residual_out_row * 2, cols * 2ll},
                         {y, tokens, y_row * (eight ? 1 : 2), cols * (eight ? 1ll : 2ll)},
                         flat(scales, size_t(tokens) * 4)};
    for (int i = 0; i < 3; ++i) {
        for (const Rows &r : in)
            if (!apart(out[i], r) && !(same(out[i], r) && (i == 0 || (i == 1 && !eight)))) return QR_ERR_INVALID_ARG;
        if (!apart(out[i], w)) return QR_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (!apart(out[i], out[j])) return QR_ERR_INVALID_ARG;
    }
    NormArgs a = {x, residual, weight, residual_out, y, eight ? scales : nullptr,
                  x_row, residual_row, residual_out_row, y_row, tokens, cols, eps};
    return from_cuda(launch_norm(dtype, weight_fp32 ? 2 : 1, a, stream_of(stream)));
}

}  // namespace

QR_EXPORT qr_status_t qr_q8_quantize(qr_dtype_t dtype, int64_t tokens, int cols, const void *x, int64_t x_row_stride,
                                     int8_t *codes, int64_t codes_row_stride, float *scales, qr_stream_t stream) {
    if (!x || !codes || !scales || tokens < 1 || cols < 1) return QR_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return QR_ERR_UNSUPPORTED;
    if (tokens > INT_MAX || cols > kMostCols) return QR_ERR_SIZE;
    if (!extent(tokens, 1, cols, x_row_stride, 0) || !extent(tokens, 1, cols, codes_row_stride, 0)) return QR_ERR_SIZE;
    if (!aligned(x, 2) || !aligned(codes, 16) || !aligned(scales, 4) || (tokens > 1 && codes_row_stride % 16))
        return QR_ERR_MISALIGNED;
    const Rows rx = {x, tokens, x_row_stride * 2, cols * 2ll}, rc = {codes, tokens, codes_row_stride, cols},
               rs = flat(scales, size_t(tokens) * 4);
    if (!apart(rc, rx) || !apart(rs, rx) || !apart(rc, rs)) return QR_ERR_INVALID_ARG;
    NormArgs a = {x, nullptr, nullptr, nullptr, codes, scales, x_row_stride, 0, 0, codes_row_stride, tokens, cols, 0.0f};
    return from_cuda(launch_norm(dtype, 0, a, stream_of(stream)));
}

QR_EXPORT qr_status_t qr_rms_norm(qr_dtype_t dtype, int64_t tokens, int cols, const void *x, int64_t x_row_stride,
                                  const void *residual, int64_t residual_row_stride, void *residual_out,
                                  int64_t residual_out_row_stride, const void *weight, int weight_fp32, float eps, void *y,
                                  int64_t y_row_stride, qr_stream_t stream) {
    return norm(dtype, tokens, cols, x, x_row_stride, residual, residual_row_stride, residual_out,
                residual_out_row_stride, weight, weight_fp32, eps, false, y, y_row_stride, nullptr, stream);
}

QR_EXPORT qr_status_t qr_rms_norm_q8(qr_dtype_t dtype, int64_t tokens, int cols, const void *x, int64_t x_row_stride,
                                     const void *residual, int64_t residual_row_stride, void *residual_out,
                                     int64_t residual_out_row_stride, const void *weight, int weight_fp32, float eps,
                                     int8_t *codes, int64_t codes_row_stride, float *scales, qr_stream_t stream) {
    return norm(dtype, tokens, cols, x, x_row_stride, residual, residual_row_stride, residual_out,
                residual_out_row_stride, weight, weight_fp32, eps, true, codes, codes_row_stride, scales, stream);
}

QR_EXPORT size_t qr_w8_bytes(int rows, int cols) {
    if (rows < 1 || cols < 1 || rows > kMostCols || cols > kMostCols) return 0;
    return w8_layout(rows, cols).bytes;
}

QR_EXPORT qr_status_t qr_w8_pack(int rows, int cols, const int8_t *codes, int64_t codes_row_stride, const float *scales,
                                 void *packed, qr_stream_t stream) {
    if (!codes || !scales || !packed || rows < 1 || cols < 1) return QR_ERR_INVALID_ARG;
    const size_t need = qr_w8_bytes(rows, cols);
    if (need == 0 || !extent(rows, 1, cols, codes_row_stride, 0)) return QR_ERR_SIZE;
    if (!aligned(packed, 16) || !aligned(scales, 4)) return QR_ERR_MISALIGNED;
    if (overlaps(packed, need, codes, extent_values(rows, 1, cols, codes_row_stride, 0)) ||
        overlaps(packed, need, scales, size_t(rows) * 4))
        return QR_ERR_INVALID_ARG;
    return from_cuda(launch_w8_pack(rows, cols, codes, codes_row_stride, scales, packed, stream_of(stream)));
}

QR_EXPORT qr_status_t qr_w8_quantize(qr_dtype_t dtype, int rows, int cols, const void *w, int64_t w_row_stride,
                                     void *packed, qr_stream_t stream) {
    if (!w || !packed || rows < 1 || cols < 1) return QR_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return QR_ERR_UNSUPPORTED;
    const size_t need = qr_w8_bytes(rows, cols), nw = extent(rows, 1, cols, w_row_stride, 0);
    if (need == 0 || nw == 0) return QR_ERR_SIZE;
    if (!aligned(packed, 16) || !aligned(w, 2)) return QR_ERR_MISALIGNED;
    if (overlaps(packed, need, w, nw)) return QR_ERR_INVALID_ARG;
    return from_cuda(launch_w8_quantize(dtype, rows, cols, w, w_row_stride, packed, stream_of(stream)));
}

QR_EXPORT size_t qr_w8_matmul_workspace_bytes(int64_t tokens, int cols) {
    if (tokens < 1 || tokens > INT_MAX - 256 || cols < 1 || cols > kMostCols) return 0;
    return w8_workspace(tokens, cols);
}

QR_EXPORT qr_status_t qr_w8_matmul(qr_dtype_t dtype, int64_t tokens, const int8_t *x, int64_t x_row_stride,
                                   const float *x_scales, int rows, int cols, const void *packed, void *y,
                                   int64_t y_row_stride, void *workspace, size_t workspace_bytes, qr_stream_t stream) {
    if (!x || !x_scales || !packed || !y || tokens < 1 || rows < 1 || cols < 1) return QR_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return QR_ERR_UNSUPPORTED;
    const size_t need = qr_w8_bytes(rows, cols), most = qr_w8_matmul_workspace_bytes(tokens, cols);
    if (need == 0 || most == 0) return QR_ERR_SIZE;
    const size_t nx = extent_values(tokens, 1, cols, x_row_stride, 0), ny = extent(tokens, 1, rows, y_row_stride, 0);
    if (nx == 0 || ny == 0) return QR_ERR_SIZE;
    const size_t nw = tokens > kW8FewTokens ? most : 0;
    if (nw && (!workspace || workspace_bytes < nw)) return QR_ERR_SIZE;
    if (!aligned(packed, 16) || !aligned(x, 16) || (tokens > 1 && x_row_stride % 16) || !aligned(x_scales, 4) ||
        !aligned(y, 2) || (nw && !aligned(workspace, 16)))
        return QR_ERR_MISALIGNED;
    const struct { const void *p; size_t n; } in[3] = {{x, nx}, {x_scales, size_t(tokens) * 4}, {packed, need}};
    for (const auto &r : in)
        if (overlaps(y, ny, r.p, r.n) || (nw && overlaps(workspace, nw, r.p, r.n))) return QR_ERR_INVALID_ARG;
    if (nw && overlaps(workspace, nw, y, ny)) return QR_ERR_INVALID_ARG;
    const W8Args a = {x, x_scales, static_cast<const uint8_t *>(packed), static_cast<uint16_t *>(y),
                      x_row_stride, y_row_stride, tokens, rows, cols, w8_layout(rows, cols)};
    return from_cuda(launch_w8_matmul(dtype, a, workspace, stream_of(stream)));
}

QR_EXPORT qr_status_t qr_rope(qr_dtype_t dtype, int64_t tokens, int head_dim, int rot_dim, int interleaved,
                              const uint64_t *turns, float factor, const int32_t *positions, int requests,
                              const int32_t *q_offsets, const int32_t *kv_lens, const void *q, int64_t q_token_stride,
                              int64_t q_head_stride, int q_heads, void *q_out, int64_t q_out_token_stride,
                              int64_t q_out_head_stride, const void *k, int64_t k_token_stride, int64_t k_head_stride,
                              int k_heads, void *k_out, int64_t k_out_token_stride, int64_t k_out_head_stride,
                              qr_stream_t stream) {
    if (!turns || !q || !q_out || tokens < 1 || q_heads < 1 || k_heads < 0 || head_dim < 1 || rot_dim < 1)
        return QR_ERR_INVALID_ARG;
    if ((k_heads > 0) != (k != nullptr) || (k_heads > 0) != (k_out != nullptr) || factor - factor != 0.0f)
        return QR_ERR_INVALID_ARG;
    if (!positions && (!q_offsets || !kv_lens || requests < 1)) return QR_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || head_dim % 2 || head_dim > 1024 || rot_dim % 2 || rot_dim > head_dim || q_heads > 65535 ||
        k_heads > 65535 || (!positions && requests > 65536))
        return QR_ERR_UNSUPPORTED;
    if (tokens > INT_MAX) return QR_ERR_SIZE;
    struct Operand {
        const void *p;
        int64_t token, head;
        int heads;
    };
    const Operand in[2] = {{q, q_token_stride, q_head_stride, q_heads}, {k, k_token_stride, k_head_stride, k_heads}},
                  out[2] = {{q_out, q_out_token_stride, q_out_head_stride, q_heads},
                            {k_out, k_out_token_stride, k_out_head_stride, k_heads}};
    const int both = k ? 2 : 1;
    for (int i = 0; i < both; ++i) {
        if (!extent(tokens, in[i].heads, head_dim, in[i].token, in[i].head) ||
            !extent(tokens, out[i].heads, head_dim, out[i].token, out[i].head) ||
            !rows_apart(tokens, out[i].heads, head_dim, out[i].token, out[i].head))
            return QR_ERR_SIZE;
        if (!aligned(in[i].p, 2) || !aligned(out[i].p, 2)) return QR_ERR_MISALIGNED;
    }
    if (!aligned(turns, 8) || !aligned(positions, 4) || (!positions && (!aligned(q_offsets, 4) || !aligned(kv_lens, 4))))
        return QR_ERR_MISALIGNED;
    // a token's heads as one row, its span (where that is wider than the stride
    // between tokens, spans are compared whole)
    auto rows = [&](const Operand &o) {
        return Rows{o.p, tokens, o.token * 2, ((o.heads - 1) * (o.heads > 1 ? o.head : 0) + head_dim) * 2};
    };
    // ... or the heads of one lie between those of the other (queries and keys of
    // a projection whose heads alternate)
    auto heads_apart = [&](const Operand &a, const Operand &b) {
        const int64_t s = a.head * 2, width = head_dim * 2ll;
        if (a.heads < 2 || b.heads < 2 || a.head != b.head || (tokens > 1 && (a.token % a.head || b.token % a.head))) return false;
        const int64_t d = ((int64_t(reinterpret_cast<uintptr_t>(b.p)) - int64_t(reinterpret_cast<uintptr_t>(a.p))) % s + s) % s;
        return d >= width && s - d >= width;
    };
    auto clear = [&](const Operand &a, const Operand &b) { return apart(rows(a), rows(b)) || heads_apart(a, b); };
    auto identical = [&](const Operand &a, const Operand &b) {
        return a.p == b.p && (tokens == 1 || a.token == b.token) && (a.heads == 1 || a.head == b.head);
    };
    const Rows tables[4] = {flat(turns, size_t(rot_dim) * 4), flat(positions, size_t(tokens) * 4),
                            flat(positions ? nullptr : q_offsets, size_t(requests) * 4 + 4),
                            flat(positions ? nullptr : kv_lens, size_t(requests) * 4)};
    for (int i = 0; i < both; ++i) {
        for (int j = 0; j < both; ++j)
            if (!clear(out[i], in[j]) && !(i == j && identical(out[i], in[j]))) return QR_ERR_INVALID_ARG;
        for (const Rows &t : tables)
            if (!apart(rows(out[i]), t)) return QR_ERR_INVALID_ARG;
    }
    if (both == 2 && !clear(out[0], out[1])) return QR_ERR_INVALID_ARG;
    RopeArgs a = {};
    for (int i = 0; i < both; ++i) {
        a.in[i] = static_cast<const uint16_t *>(in[i].p);
        a.out[i] = static_cast<uint16_t *>(const_cast<void *>(out[i].p));
        // (a stride that no second token or head uses is not read)
        a.in_token[i] = tokens > 1 ? in[i].token : 0;
        a.in_head[i] = in[i].heads > 1 ? in[i].head : 0;
        a.out_token[i] = tokens > 1 ? out[i].token : 0;
        a.out_head[i] = out[i].heads > 1 ? out[i].head : 0;
        a.heads[i] = in[i].heads;
    }
    a.turns = reinterpret_cast<const unsigned long long *>(turns);
    a.positions = positions;
    a.q_offsets = positions ? nullptr : q_offsets;
    a.kv_lens = positions ? nullptr : kv_lens;
    a.factor = factor;
    a.tokens = tokens;
    a.requests = requests;
    a.head_dim = head_dim;
    a.rot = rot_dim;
    return from_cuda(launch_rope(dtype, interleaved != 0, a, stream_of(stream)));
}
