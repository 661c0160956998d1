// qr_w4.cuh -- what the kernels of the 4-bit matrix-vector product share.
#pragma once

#include "qr_device.cuh"
#include "qr_kv_device.cuh"
#include "qr_serving.h"

namespace qrk {

struct W4MatvecArgs {
    const uint16_t *x;
    uint16_t *y;
    const uint8_t *packed;
    long long x_stride, y_stride, tokens;
    int rows, cols, group_shift;  // group = 32 << group_shift
    W4Layout l;
};

// A fragment register from a word shifted so that its pair of codes is in
// bits 0..3 and 16..19, minus the offset pair `zero` (1024 + z or 128 + z).
template <int DT>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t zero) {
    uint32_t v = (w & 0x000f000fu) | (DT == 0 ? 0x64006400u : 0x43004300u);
    if constexpr (DT == 0) {
        const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&zero));
        return *reinterpret_cast<const uint32_t *>(&r);
    } else {
        const __nv_bfloat162 r =
            __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&zero));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
}

// Eight 16-bit values from byte `off` (even) of two 16-byte words on, those
// past the first `have` zero.
__device__ __forceinline__ uint4 take8(const uint4 &a, const uint4 &b, uint32_t off, int have) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (off & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (off & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t bits = (off & 2) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = __funnelshift_r(w[i], w[i + 1], bits);
        if (2 * i + 1 >= have) w[i] = 2 * i >= have ? 0u : w[i] & 0xffffu;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The first `have` (at most 8; none if below 1) 16-bit values from a 2-byte
// aligned address, zeros after them: from the one or two aligned 16-byte words
// that hold them.
__device__ __forceinline__ uint4 load8_any(const uint16_t *p, int have) {
    if (have <= 0) return make_uint4(0, 0, 0, 0);
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint32_t off = static_cast<uint32_t>(at & 15);
    const uint4 *src = reinterpret_cast<const uint4 *>(at - off);
    const uint4 a = *src;
    uint4 b = make_uint4(0, 0, 0, 0);
    if (off + 2 * min(have, 8) > 16) b = src[1];
    return take8(a, b, off, have);
}

// The tcgen05 kernel (qr_w4_tc.cu), for more than kW4FewTokens tokens; the
// workspace holds x's rows when they are not aligned.
cudaError_t launch_w4_tc(int dtype, const W4MatvecArgs &a, bool zeros, void *workspace, cudaStream_t s);

}  // namespace qrk
