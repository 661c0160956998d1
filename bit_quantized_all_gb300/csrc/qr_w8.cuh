// qr_w8.cuh -- what the kernels of the 8-bit product share.
#pragma once

#include "qr_device.cuh"
#include "qr_kv_device.cuh"
#include "qr_serving.h"

namespace qrk {

// Four packed weights (code + 128 each) of a word as two fp16 pairs, in order:
// under the high byte 0x64 they are 1024 + 128 + code, minus 1152, exact.
__device__ __forceinline__ void weights_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    lo = minus_1152(__byte_perm(w, kHigh, 0x4140));
    hi = minus_1152(__byte_perm(w, kHigh, 0x4342));
}

// The first `have` codes (at most 16; none if below 1) from a 16-byte aligned
// address, zeros after them; no byte past them is read.
__device__ __forceinline__ uint4 load16_codes(const int8_t *p, int have) {
    if (have >= 16) return *reinterpret_cast<const uint4 *>(p);
    uint32_t w[4] = {0, 0, 0, 0};
    if (have <= 0) return make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (i < have) w[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(p[i])) << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

cudaError_t launch_w8_few(int dtype, const W8Args &a, cudaStream_t s);
cudaError_t launch_w8_tc(int dtype, const W8Args &a, void *workspace, cudaStream_t s);

}  // namespace qrk
