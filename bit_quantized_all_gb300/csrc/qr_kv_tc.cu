// qr_kv_tc.cu -- the tcgen05 attention kernel's instantiations.
#include "qr_kv_tc.cuh"

namespace qrk {

cudaError_t launch_kv_tc(int dtype, const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s) {
    if (c.dim <= 64)
        return c.dim == 64 ? run_kv_tc<64, true>(dtype, a, c, group, s) : run_kv_tc<64, false>(dtype, a, c, group, s);
    return c.dim == 128 ? run_kv_tc<128, true>(dtype, a, c, group, s) : run_kv_tc<128, false>(dtype, a, c, group, s);
}

}  // namespace qrk
