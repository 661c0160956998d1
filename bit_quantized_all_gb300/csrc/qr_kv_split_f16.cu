// qr_kv_split_f16.cu -- the split attention kernel's instantiations for fp16.
#include "qr_kv_split.cuh"

namespace qrk {

cudaError_t launch_kv_split_f16(const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s) {
    return pick_kv_split<false>(a, c, group, s);
}

}  // namespace qrk
