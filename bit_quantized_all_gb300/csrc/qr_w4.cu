// qr_w4.cu -- 4-bit weights with group scales: packing and quantizing
// (qr_w4_pack, qr_w4_quantize); the product is in qr_w4_matvec.cu.
//
// Packed order.  y^T = W x^T runs on 16-bit matrix instructions with 16 weight
// rows as M and tokens as N.  A tile of 16 rows x 64 columns is 512 bytes, lane
// l = 4g + t of a warp owning 16 of them: word j (j = 0..3) is its A fragment of
// the j-th instruction of 16 columns, eight codes of rows g and g + 8 at the
// four columns 16 j + 4 t + 0..3.  Which of an instruction's sixteen columns
// stands at which of its places is free as long as x is read alike; so a lane
// reads its x values as four 8-byte pieces, and the fragments stored to
// tensor memory (qr_w4_tc.cu) have the columns in their own order.  In a word,
// nibble i and nibble i + 4 are the two codes of fragment register i, so that
// (word >> 4i) & 0x000f000f is a register's pair of codes.
#include "qr_device.cuh"
#include "qr_launch.h"
#include "qr_serving.h"

namespace qrk {

constexpr int kW4Threads = 256;

// Column (within 64) of nibble `nib` of word j of lane t; its row is
// g + 8 * (nib & 1).
__device__ __forceinline__ int w4_column(int t, int j, int nib) {
    return 16 * j + 4 * t + 2 * ((nib & 3) >> 1) + (nib >> 2);
}

// One thread per word of codes, scale pair and zero pair.
__global__ void __launch_bounds__(kW4Threads) w4_pack_kernel(int rows, int cols, int group, W4Layout l,
                                                             const uint8_t *codes, const uint16_t *scales,
                                                             const uint8_t *zeros, uint8_t *packed) {
    chain_entry();
    const long long words = static_cast<long long>(l.row_tiles) * l.chunks * 128;
    const long long pairs = static_cast<long long>(l.row_tiles) * l.groups * 8;
    const long long bytes_per_row = cols / 2 + cols % 2;
    const int groups = cols / group + (cols % group != 0);
    for (long long i = static_cast<long long>(blockIdx.x) * kW4Threads + threadIdx.x; i < words + pairs;
         i += static_cast<long long>(gridDim.x) * kW4Threads) {
        if (i < words) {
            const int j = static_cast<int>(i & 3), lane = static_cast<int>((i >> 2) & 31);
            const long long tile = i >> 7;
            const long long row0 = tile / l.chunks * 16 + (lane >> 2);
            const int col0 = static_cast<int>(tile % l.chunks) * 64;
            uint32_t w = 0;
            for (int nib = 0; nib < 8; ++nib) {
                const long long row = row0 + 8 * (nib & 1);
                const int col = col0 + w4_column(lane & 3, j, nib);
                uint32_t u = 8;
                if (row < rows && col < cols) u = (codes[row * bytes_per_row + (col >> 1)] >> (4 * (col & 1))) & 15;
                w |= u << (4 * nib);
            }
            reinterpret_cast<uint32_t *>(packed)[i] = w;
        } else {
            const long long p = i - words;
            const long long at = p >> 3;
            const long long row = at / l.groups * 16 + (p & 7);
            const int g = static_cast<int>(at % l.groups);
            for (int k = 0; k < 2; ++k) {
                const bool in = row + 8 * k < rows && g < groups;
                const long long src = (row + 8 * k) * groups + g;
                reinterpret_cast<uint16_t *>(packed + l.scales_at)[2 * p + k] = in ? scales[src] : 0;
                if (zeros) (packed + l.zeros_at)[2 * p + k] = in ? zeros[src] & 15 : 8;
            }
        }
    }
}

// A warp quantizes one group of one row, then writes the nibbles it owns;
// several lanes of one byte's two nibbles meet in a word, so the codes go
// through shared memory: a CTA of 8 warps takes 16 rows x 64 columns.
template <int DT>
__global__ void __launch_bounds__(kW4Threads) w4_quantize_kernel(int rows, int cols, int group, W4Layout l,
                                                                 const uint16_t *w, long long stride, uint8_t *packed) {
    chain_entry();
    __shared__ uint8_t code[16][64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long tiles = static_cast<long long>(l.row_tiles) * l.chunks;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const long long row0 = tile / l.chunks * 16;
        const int chunk = static_cast<int>(tile % l.chunks);
        __syncthreads();
        for (int rr = warp; rr < 16; rr += 8) {
            const long long row = row0 + rr;
            const int span = group < 64 ? group : 64;  // columns of this tile in one group
            for (int c0 = 0; c0 < 64; c0 += span) {
                const int g = (chunk * 64 + c0) / group, gc = g * group;
                float amax = 0.0f;
                for (int i = lane; i < group; i += 32)
                    if (row < rows && gc + i < cols) {
                        const uint16_t u = w[row * stride + gc + i];
                        amax = fmaxf(amax, fabsf(DT ? __uint_as_float(static_cast<uint32_t>(u) << 16)
                                                    : __half2float(__ushort_as_half(u))));
                    }
#pragma unroll
                for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
                const __half s16 = __float2half_rn(fminf(__fmul_rn(amax, 0.125f), 65504.0f));
                const float s = __half2float(s16), r = s > 0.0f ? __frcp_rn(s) : 0.0f;
                for (int i = lane; i < span; i += 32) {
                    const int col = chunk * 64 + c0 + i;
                    float x = 0.0f;
                    if (row < rows && col < cols) {
                        const uint16_t u = w[row * stride + col];
                        x = DT ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u));
                    }
                    code[rr][c0 + i] = static_cast<uint8_t>(
                        __float2int_rn(fminf(fmaxf(__fmul_rn(x, r), -8.0f), 7.0f)) + 8);
                }
                if (lane == 0 && (chunk * 64 + c0) % group == 0)
                    reinterpret_cast<__half *>(packed + l.scales_at)[((row0 / 16) * l.groups + g) * 16 +
                                                                     2 * (rr & 7) + (rr >> 3)] = s16;
            }
        }
        __syncthreads();
        if (threadIdx.x < 128) {
            const int j = threadIdx.x & 3, ln = threadIdx.x >> 2;
            uint32_t v = 0;
            for (int nib = 0; nib < 8; ++nib)
                v |= static_cast<uint32_t>(code[(ln >> 2) + 8 * (nib & 1)][w4_column(ln & 3, j, nib)]) << (4 * nib);
            reinterpret_cast<uint32_t *>(packed)[tile * 128 + threadIdx.x] = v;
        }
    }
}

cudaError_t launch_w4_pack(int rows, int cols, int group, const uint8_t *codes, const void *scales,
                           const uint8_t *zeros, void *packed, cudaStream_t s) {
    const W4Layout l = w4_layout(rows, cols, group, zeros != nullptr);
    const long long units = (static_cast<long long>(l.row_tiles) * (l.chunks * 128LL + l.groups * 8LL) + kW4Threads - 1) / kW4Threads;
    cudaError_t err = cudaSuccess;
    const int grid = grid_for(reinterpret_cast<const void *>(w4_pack_kernel), kW4Threads, units, 0, 4, &err);
    if (grid <= 0) return err;
    return launch_chained(w4_pack_kernel, grid, kW4Threads, 0, s, rows, cols, group, l, codes,
                          static_cast<const uint16_t *>(scales), zeros, static_cast<uint8_t *>(packed));
}

cudaError_t launch_w4_quantize(int dtype, int rows, int cols, int group, const void *w, long long w_stride,
                               void *packed, cudaStream_t s) {
    const W4Layout l = w4_layout(rows, cols, group, false);
    auto kern = dtype ? w4_quantize_kernel<1> : w4_quantize_kernel<0>;
    cudaError_t err = cudaSuccess;
    const int grid = grid_for(reinterpret_cast<const void *>(kern), kW4Threads,
                              static_cast<long long>(l.row_tiles) * l.chunks, 0, 4, &err);
    if (grid <= 0) return err;
    return launch_chained(kern, grid, kW4Threads, 0, s, rows, cols, group, l, static_cast<const uint16_t *>(w), w_stride,
                          static_cast<uint8_t *>(packed));
}

}  // namespace qrk
