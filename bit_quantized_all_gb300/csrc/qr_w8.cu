// qr_w8.cu -- 8-bit weights with a scale for each row: packing and quantizing
// (qr_w8_pack, qr_w8_quantize).
#include "qr_device.cuh"
#include "qr_kv_device.cuh"
#include "qr_launch.h"
#include "qr_serving.h"
#include "qr_w8.cuh"

namespace qrk {

constexpr int kW8Threads = 256;

// A thread per 16 codes of a tile's row, then one per scale.
__global__ void __launch_bounds__(kW8Threads) w8_pack_kernel(int rows, int cols, W8Layout l, const int8_t *codes,
                                                             long long stride, const float *scales, uint8_t *packed) {
    chain_entry();
    const long long pieces = static_cast<long long>(l.row_tiles) * l.chunks * 64, all = pieces + l.row_tiles * 16ll;
    for (long long i = static_cast<long long>(blockIdx.x) * kW8Threads + threadIdx.x; i < all;
         i += static_cast<long long>(gridDim.x) * kW8Threads) {
        if (i < pieces) {
            const long long tile = i >> 6, row = tile / l.chunks * 16 + (i >> 2 & 15);
            const int col = static_cast<int>(tile % l.chunks) * 64 + static_cast<int>(i & 3) * 16;
            const int8_t *const src = codes + row * stride + col;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (row < rows) {
                if ((reinterpret_cast<uintptr_t>(src) & 15) == 0 || cols - col < 16) {
                    w = load16_codes(src, cols - col);
                } else {  // by the bytes that the address allows no more than
                    uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int b = 0; b < 16; ++b) u[b >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(src[b])) << (8 * (b & 3));
                    w = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
            reinterpret_cast<uint4 *>(packed)[i] = make_uint4(w.x ^ kFlip, w.y ^ kFlip, w.z ^ kFlip, w.w ^ kFlip);
        } else {
            const long long row = i - pieces;
            reinterpret_cast<float *>(packed + l.scales_at)[row] = row < rows ? scales[row] : 0.0f;
        }
    }
}

// A CTA takes a row: its largest magnitude, then its codes.
template <int DT>
__global__ void __launch_bounds__(kW8Threads) w8_quantize_kernel(int rows, int cols, W8Layout l, const uint16_t *w,
                                                                 long long stride, uint8_t *packed) {
    chain_entry();
    __shared__ float s_max[kW8Threads / 32];
    const int tid = threadIdx.x;
    for (long long row = blockIdx.x; row < l.row_tiles * 16ll; row += gridDim.x) {
        const uint16_t *const src = w + row * stride;
        float most = 0.0f;
        if (row < rows)
            for (int i = tid; i < cols; i += kW8Threads) most = max_nan(most, fabsf(widen1<DT>(src[i])));
#pragma unroll
        for (int d = 16; d; d >>= 1) most = max_nan(most, __shfl_xor_sync(~0u, most, d));
        __syncthreads();
        if ((tid & 31) == 0) s_max[tid >> 5] = most;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kW8Threads / 32; ++k) most = max_nan(most, s_max[k]);
        float f = __fdiv_rn(127.0f, most);
        if (!(f < INFINITY)) f = 0.0f;
        uint8_t *const to = packed + (row / 16 * l.chunks) * 1024 + row % 16 * 64;
        for (int i = tid; i < l.chunks * 64; i += kW8Threads) {
            const float x = row < rows && i < cols ? widen1<DT>(src[i]) : 0.0f;
            to[(i / 64) * 1024ll + i % 64] = static_cast<uint8_t>(__float2int_rn(__fmul_rn(x, f)) + 128);
        }
        if (tid == 0) reinterpret_cast<float *>(packed + l.scales_at)[row] = __fdiv_rn(most, 127.0f);
    }
}

cudaError_t launch_w8_pack(int rows, int cols, const int8_t *codes, long long stride, const float *scales, void *packed,
                           cudaStream_t s) {
    const W8Layout l = w8_layout(rows, cols);
    const long long units = (static_cast<long long>(l.row_tiles) * (l.chunks * 64ll + 16) + kW8Threads - 1) / kW8Threads;
    cudaError_t err = cudaSuccess;
    const int grid = grid_for(reinterpret_cast<const void *>(w8_pack_kernel), kW8Threads, units, 0, 4, &err);
    if (grid <= 0) return err;
    return launch_chained(w8_pack_kernel, grid, kW8Threads, 0, s, rows, cols, l, codes, stride, scales,
                          static_cast<uint8_t *>(packed));
}

cudaError_t launch_w8_quantize(int dtype, int rows, int cols, const void *w, long long stride, void *packed,
                               cudaStream_t s) {
    const W8Layout l = w8_layout(rows, cols);
    auto kern = dtype ? w8_quantize_kernel<1> : w8_quantize_kernel<0>;
    cudaError_t err = cudaSuccess;
    const int grid = grid_for(reinterpret_cast<const void *>(kern), kW8Threads, l.row_tiles * 16ll, 0, 4, &err);
    if (grid <= 0) return err;
    return launch_chained(kern, grid, kW8Threads, 0, s, rows, cols, l, static_cast<const uint16_t *>(w), stride,
                          static_cast<uint8_t *>(packed));
}

}  // namespace qrk
