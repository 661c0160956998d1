// qr_kv_attention.cu -- picks the kernel of an attention call.
#include "qr_kv_split.cuh"

namespace qrk {

// The tcgen05 kernel (qr_kv_tc.cu), for head_dim up to 128.
cudaError_t launch_kv_tc(int dtype, const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s);

size_t kv_attention_workspace(int, long long tokens, int q_heads, int heads, int head_dim) {
    // two slots per CTA: of at most 640 CTAs of up to 32 rows (16 above 128
    // dimensions), or of 160 of up to 256
    const size_t dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    size_t rows = size_t(2 * kMostCtas) * (dp <= 128 ? 32 : 16);
    if (dp <= 128 && tokens * (q_heads / heads) > 32) rows = size_t(2 * 160) * 256;
    return kWorkspaceCounters + rows * (dp + 2) * 4;
}

template <int DP, int NT>
static cudaError_t run_split(int dtype, const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s) {
    return c.dim == DP ? run_kv_split<DP, NT, true>(dtype, a, c, group, s)
                       : run_kv_split<DP, NT, false>(dtype, a, c, group, s);
}

cudaError_t launch_kv_attention(int dtype, const KvAttentionArgs &a, const qr_kv_cache_t &cache, cudaStream_t s) {
    const KvView c = kv_view(cache);
    const int group = a.q_heads / c.heads;
    const long long rows = static_cast<long long>(a.max_q) * group;
    if (c.dim <= 128 && rows > 32) return launch_kv_tc(dtype, a, c, group, s);
    if (c.dim <= 64)
        return rows <= 8    ? run_split<64, 1>(dtype, a, c, group, s)
               : rows <= 16 ? run_split<64, 2>(dtype, a, c, group, s)
               : rows <= 24 ? run_split<64, 3>(dtype, a, c, group, s)
                            : run_split<64, 4>(dtype, a, c, group, s);
    if (c.dim <= 128)
        return rows <= 8    ? run_split<128, 1>(dtype, a, c, group, s)
               : rows <= 16 ? run_split<128, 2>(dtype, a, c, group, s)
               : rows <= 24 ? run_split<128, 3>(dtype, a, c, group, s)
                            : run_split<128, 4>(dtype, a, c, group, s);
    return rows <= 8 ? run_split<256, 1>(dtype, a, c, group, s) : run_split<256, 2>(dtype, a, c, group, s);
}

}  // namespace qrk
