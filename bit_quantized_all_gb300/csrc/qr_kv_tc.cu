// qr_kv_tc.cu -- the tcgen05 attention kernel's instantiations.
#include "qr_kv_tc.cuh"

namespace qrk {

template <bool BF16>
static cudaError_t pick(const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s) {
    if (c.dim <= 64)
        return c.dim == 64 ? run_kv_tc<64, true, BF16>(a, c, group, s) : run_kv_tc<64, false, BF16>(a, c, group, s);
    return c.dim == 128 ? run_kv_tc<128, true, BF16>(a, c, group, s) : run_kv_tc<128, false, BF16>(a, c, group, s);
}

cudaError_t launch_kv_tc(int dtype, const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s) {
    return dtype ? pick<true>(a, c, group, s) : pick<false>(a, c, group, s);
}

}  // namespace qrk
