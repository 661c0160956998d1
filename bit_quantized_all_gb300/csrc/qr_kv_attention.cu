// qr_kv_attention.cu -- attention over the 8-bit paged cache
// (qr_kv_attention).
#include "qr_device.cuh"
#include "qr_launch.h"
#include "qr_serving.h"

namespace qrk {

struct KvView {
    const int8_t *k, *v;
    const float *ks, *vs;
    long long k_block, k_head, v_block, v_head;
    int blocks, heads, dim, shift;
};

// One warp per (query token, query head).
template <int DT>
__global__ void kv_attention_simple_kernel(KvAttentionArgs a, KvView c) {
    chain_entry();
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const long long t = item / a.q_heads;
    const int j = static_cast<int>(item % a.q_heads);
    if (t >= a.tokens || t >= a.q_offsets[a.requests]) return;
    int lo = 0, hi = a.requests - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.q_offsets[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int r = lo, h = j / (a.q_heads / c.heads), bs = 1 << c.shift;
    const int nq = a.q_offsets[r + 1] - a.q_offsets[r];
    const long long kv = max(0LL, min(static_cast<long long>(a.kv_lens[r]), static_cast<long long>(a.width) << c.shift));
    const long long pos = static_cast<long long>(a.kv_lens[r]) - nq + (t - a.q_offsets[r]);
    const long long end = a.causal ? min(kv, pos + 1) : kv;
    const long long begin = a.window > 0 ? max(0LL, pos - a.window + 1) : 0;
    const uint16_t *q = static_cast<const uint16_t *>(a.q) + t * a.q_token + j * a.q_head;
    auto widen = [](uint16_t u) {
        return DT ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u));
    };
    float qf[8], acc[8], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        qf[i] = lane + 32 * i < c.dim ? widen(q[lane + 32 * i]) : 0.0f;
        acc[i] = 0.0f;
    }
    for (long long i = begin; i < end; ++i) {
        const int b = a.table[static_cast<long long>(r) * a.width + (i >> c.shift)];
        if (b < 0 || b >= c.blocks) continue;
        const long long row = (i & (bs - 1)) * c.dim;
        const int8_t *kp = c.k + b * c.k_block + h * c.k_head + row, *vp = c.v + b * c.v_block + h * c.v_head + row;
        float s = 0.0f;
#pragma unroll
        for (int d = 0; d < 8; ++d)
            if (lane + 32 * d < c.dim) s = __fmaf_rn(qf[d], static_cast<float>(kp[lane + 32 * d]), s);
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        const long long si = static_cast<long long>(b) * c.heads + h;
        s *= a.scale * c.ks[si];
        const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * f + p;
        const float w = p * c.vs[si];
#pragma unroll
        for (int d = 0; d < 8; ++d)
            if (lane + 32 * d < c.dim) acc[d] = __fmaf_rn(w, static_cast<float>(vp[lane + 32 * d]), acc[d] * f);
    }
    uint16_t *out = static_cast<uint16_t *>(a.out) + t * a.out_token + j * a.out_head;
#pragma unroll
    for (int d = 0; d < 8; ++d)
        if (lane + 32 * d < c.dim) {
            const float v = l > 0.0f ? acc[d] / l : 0.0f;
            out[lane + 32 * d] = DT ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
        }
    if (a.lse && lane == 0) a.lse[t * a.q_heads + j] = l > 0.0f ? m + logf(l) : -INFINITY;
}

size_t kv_attention_workspace(int, long long, int, int, int) { return 16; }

cudaError_t launch_kv_attention(int dtype, const KvAttentionArgs &a, const qr_kv_cache_t &cache, cudaStream_t s) {
    KvView c = {static_cast<const int8_t *>(cache.k_codes), static_cast<const int8_t *>(cache.v_codes), cache.k_scales,
                cache.v_scales, cache.k_block_stride, cache.k_head_stride, cache.v_block_stride, cache.v_head_stride,
                cache.blocks, cache.heads, cache.head_dim, 0};
    while ((1 << c.shift) < cache.block_size) ++c.shift;
    const long long warps = a.tokens * a.q_heads;
    return launch_chained(dtype ? kv_attention_simple_kernel<1> : kv_attention_simple_kernel<0>,
                          static_cast<unsigned>((warps + 3) / 4), 128, 0, s, a, c);
}

}  // namespace qrk
