// qr_w8_matmul.cu -- y = x W^T for rows of x and weights in 8 bits
// (qr_w8_matmul); qr_w8.cu packs the weights.
#include "qr_device.cuh"
#include "qr_kv_device.cuh"
#include "qr_launch.h"
#include "qr_serving.h"

namespace qrk {

constexpr int kW8mThreads = 256, kW8mTile = 32;

// A CTA takes 32 tokens by 32 rows, a chunk of 64 columns at a time through
// shared memory; a chunk's integer sum is exact, and added in fp32.
template <int DT>
__global__ void __launch_bounds__(kW8mThreads) w8_simple_kernel(W8Args a) {
    chain_entry();
    __shared__ int s_x[kW8mTile][17], s_w[kW8mTile][17];
    const int tid = threadIdx.x, n = tid & 31, m0 = tid >> 5;
    const long long row0 = static_cast<long long>(blockIdx.x) * kW8mTile;
    for (long long token0 = blockIdx.y * static_cast<long long>(kW8mTile); token0 < a.tokens;
         token0 += gridDim.y * static_cast<long long>(kW8mTile)) {
        float acc[4] = {};
        for (int c = 0; c < a.l.chunks; ++c) {
            __syncthreads();
            for (int i = tid; i < kW8mTile * 16; i += kW8mThreads) {
                const int r = i >> 4, k = i & 15, col = c * 64 + k * 4;
                const long long row = row0 + r, token = token0 + r;
                uint32_t w = kFlip, x = 0;
                if (row < a.l.row_tiles * 16ll)
                    w = reinterpret_cast<const uint32_t *>(a.packed)[(row / 16 * a.l.chunks + c) * 256 + row % 16 * 16 + k];
                if (token < a.tokens)
                    for (int b = 0; b < 4; ++b)
                        if (col + b < a.cols) x |= static_cast<uint32_t>(static_cast<uint8_t>(a.x[token * a.x_stride + col + b])) << (8 * b);
                s_w[r][k] = static_cast<int>(w ^ kFlip);
                s_x[r][k] = static_cast<int>(x);
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                int sum = 0;
                for (int k = 0; k < 16; ++k) sum = __dp4a(s_x[m0 + 8 * e][k], s_w[n][k], sum);
                acc[e] += static_cast<float>(sum);
            }
        }
        const long long row = row0 + n;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const long long token = token0 + m0 + 8 * e;
            if (token < a.tokens && row < a.rows)
                a.y[token * a.y_stride + row] = narrow1<DT>(
                    acc[e] * a.x_scales[token] * reinterpret_cast<const float *>(a.packed + a.l.scales_at)[row]);
        }
    }
}

size_t w8_workspace(long long tokens, int cols) {
    return static_cast<size_t>((tokens + 255) / 256 * 256) * (static_cast<size_t>(cols) / 64 + (cols % 64 != 0)) * 128;
}

cudaError_t launch_w8_matmul(int dtype, const W8Args &a, void *, cudaStream_t s) {
    const long long tiles = (a.tokens + kW8mTile - 1) / kW8mTile;
    const dim3 grid((a.l.row_tiles + 1) / 2, static_cast<unsigned>(tiles < 65535 ? tiles : 65535));
    return launch_chained(dtype ? w8_simple_kernel<1> : w8_simple_kernel<0>, grid, kW8mThreads, 0, s, a);
}

}  // namespace qrk
