// qr_kv_attention.cu -- picks the kernel of an attention call.
#include "qr_kv_split.cuh"

namespace qrk {

// The tcgen05 kernel (qr_kv_tc.cu), for head_dim up to 128.
cudaError_t launch_kv_tc(int dtype, const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s);
// The split kernel (qr_kv_split.cuh).
cudaError_t launch_kv_split_f16(const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s);
cudaError_t launch_kv_split_bf16(const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s);

size_t kv_attention_workspace(int, long long tokens, int q_heads, int heads, int head_dim) {
    // two slots per CTA: of at most 640 CTAs of up to 32 rows (16 above 128
    // dimensions), or of 160 of up to 256
    const size_t dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    size_t rows = size_t(2 * kMostCtas) * (dp <= 128 ? 32 : 16);
    if (dp <= 128 && tokens * (q_heads / heads) > 32) rows = size_t(2 * 160) * 256;
    return kWorkspaceCounters + rows * (dp + 2) * 4;
}

cudaError_t launch_kv_attention(int dtype, const KvAttentionArgs &a, const qr_kv_cache_t &cache, cudaStream_t s) {
    const KvView c = kv_view(cache);
    const int group = a.q_heads / c.heads;
    // Above 32 rows an item the products are tcgen05's: 32 rows over one context
    // of 131075 keys take 80 us split and 107 so, in 64 requests of up to 2048
    // keys 83 and 69; 40 rows 120 and 108, and 135 and 69.
    if (c.dim <= 128 && static_cast<long long>(a.max_q) * group > 32) return launch_kv_tc(dtype, a, c, group, s);
    return dtype ? launch_kv_split_bf16(a, c, group, s) : launch_kv_split_f16(a, c, group, s);
}

}  // namespace qrk
