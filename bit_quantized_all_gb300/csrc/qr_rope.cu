// qr_rope.cu -- rotary positions of queries and keys (qr_rope).
#include "qr_device.cuh"
#include "qr_launch.h"
#include "qr_serving.h"

namespace qrk {

constexpr int kRopeThreads = 128;

// The position of token t by a step's plan, -1 in `request` past its last one.
__device__ __forceinline__ long long plan_position(const RopeArgs &a, long long t, int &request) {
    int lo = 0, hi = a.requests;  // q_offsets[lo] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.q_offsets[mid] <= t) lo = mid; else hi = mid;
    }
    const int end = a.q_offsets[lo + 1];
    request = t < end ? lo : -1;
    return a.kv_lens[lo] - (end - t);
}

template <int DT, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
    chain_entry();
    const int pairs = a.rot / 2, heads = a.heads[0] + a.heads[1], each = pairs + a.head_dim - a.rot;
    for (long long t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        int request = 0;
        const long long p = a.positions ? a.positions[t] : plan_position(a, t, request);
        if (request < 0) continue;
        for (int i = threadIdx.x; i < heads * each; i += kRopeThreads) {
            const int which = i / each >= a.heads[0], head = i / each - (which ? a.heads[0] : 0), j = i % each;
            const uint16_t *in = a.in[which] + t * a.in_token[which] + head * a.in_head[which];
            uint16_t *out = a.out[which] + t * a.out_token[which] + head * a.out_head[which];
            if (j >= pairs) {
                out[a.rot + j - pairs] = in[a.rot + j - pairs];
                continue;
            }
            const unsigned long long turn = static_cast<unsigned long long>(p) * a.turns[j];
            float sn, cs;
            sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &sn, &cs);
            sn *= a.factor, cs *= a.factor;
            const int ia = INTERLEAVED ? 2 * j : j, ib = INTERLEAVED ? 2 * j + 1 : j + pairs;
            const float x = widen1<DT>(in[ia]), y = widen1<DT>(in[ib]);
            out[ia] = narrow1<DT>(x * cs - y * sn);
            out[ib] = narrow1<DT>(y * cs + x * sn);
        }
    }
}

cudaError_t launch_rope(int dtype, bool interleaved, const RopeArgs &a, cudaStream_t s) {
    auto kern = dtype ? (interleaved ? rope_kernel<1, true> : rope_kernel<1, false>)
                      : (interleaved ? rope_kernel<0, true> : rope_kernel<0, false>);
    return launch_chained(kern, static_cast<unsigned>(a.tokens < 65536 ? a.tokens : 65536), kRopeThreads, 0, s, a);
}

}  // namespace qrk
