// qr_w8_few.cu -- y = x W^T for up to 16 rows of x and weights in 8 bits
// (qr_w8_matmul); qr_w8.cu describes the packed order.
//
// y^T = W x^T on m16n8k16 with fp16 operands: 16 weight rows as M, 8 tokens as
// N, both sides' codes as exact fp16 integers.  Which of an instruction's
// columns stands at which of its places is free as long as both sides agree: a
// lane takes 16 consecutive columns of its rows, one 16-byte load of a packed
// tile's row, and of its token's row, and they serve four instructions.
//
// The eight warps of a CTA take the chunks of its slice of the columns in
// turn, for RT row tiles, and add their sums in order through shared memory;
// the CTAs of a cluster take the slices of the same rows and add theirs
// through distributed shared memory.
#include <cooperative_groups.h>

#include "qr_launch.h"
#include "qr_w8.cuh"

namespace qrk {

namespace cg = cooperative_groups;

constexpr int kW8fWarps = 8, kW8fThreads = 32 * kW8fWarps;
constexpr int kW8fDepth = 4;  // chunks in flight per warp

// NT: tiles of eight tokens; RT: tiles of 16 rows.
template <int DT, int NT, int RT>
__global__ void __launch_bounds__(kW8fThreads, 2) w8_few_kernel(W8Args a, int slice) {
    chain_entry();
    constexpr int kRows = 16 * RT, kTokens = 8 * NT, kValues = kRows * kTokens;
    __shared__ float s_part[kW8fWarps][kTokens][kRows + 4];
    __shared__ float s_sum[kValues];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int splits = static_cast<int>(cluster.num_blocks()), split = static_cast<int>(cluster.block_rank());
    const int first = split * slice, count = max(0, min(slice, a.l.chunks - first));
    const int tile0 = blockIdx.x / splits * RT;
    const int tokens = static_cast<int>(a.tokens);

    const uint4 *wp[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        wp[r] = reinterpret_cast<const uint4 *>(a.packed) +
                (static_cast<long long>(min(tile0 + r, a.l.row_tiles - 1)) * a.l.chunks + first) * 64 + lane;
    const int8_t *xp[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xp[n] = a.x + min(n * 8 + g, tokens - 1) * a.x_stride + first * 64ll + t * 16;
    const int cols = a.cols - first * 64 - t * 16;  // of this lane's part of the slice

    uint4 w[kW8fDepth][RT][2], x[kW8fDepth][NT];
    auto fetch = [&](int d, int i) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) w[d][r][h] = __ldcs(wp[r] + i * 64 + h * 32);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            x[d][n] = n * 8 + g < tokens ? load16_codes(xp[n] + i * 64, cols - i * 64) : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int d = 0; d < kW8fDepth; ++d)
        if (warp + d * kW8fWarps < count) fetch(d, warp + d * kW8fWarps);

    float acc[RT][NT][4] = {};
    for (int i0 = warp; i0 < count; i0 += kW8fDepth * kW8fWarps) {
#pragma unroll
        for (int d = 0; d < kW8fDepth; ++d) {
            const int i = i0 + d * kW8fWarps;
            if (i >= count) break;
            uint32_t b[NT][8];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint32_t u[4] = {x[d][n].x, x[d][n].y, x[d][n].z, x[d][n].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) codes_f16(u[j], b[n][2 * j], b[n][2 * j + 1]);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t up[4] = {w[d][r][0].x, w[d][r][0].y, w[d][r][0].z, w[d][r][0].w},
                               low[4] = {w[d][r][1].x, w[d][r][1].y, w[d][r][1].z, w[d][r][1].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t f[4];
                    weights_f16(up[j], f[0], f[2]);
                    weights_f16(low[j], f[1], f[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16_acc(acc[r][n], f, b[n][2 * j], b[n][2 * j + 1]);
                }
            }
            const int next = i + kW8fDepth * kW8fWarps;
            if (next < count) fetch(d, next);
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s_part[warp][n * 8 + 2 * t + (e & 1)][r * 16 + g + 8 * (e >> 1)] = acc[r][n][e];
    __syncthreads();
    const float *const scales = reinterpret_cast<const float *>(a.packed + a.l.scales_at) + tile0 * 16ll;
    auto store = [&](int i, float v) {
        const int m = i / kRows, row = i % kRows;
        if (m < tokens && tile0 * 16ll + row < a.rows)
            a.y[m * a.y_stride + tile0 * 16ll + row] = narrow1<DT>(v * a.x_scales[m] * scales[row]);
    };
    for (int i = tid; i < kValues; i += kW8fThreads) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kW8fWarps; ++k) v += s_part[k][i / kRows][i % kRows];
        if (splits == 1) store(i, v); else s_sum[i] = v;
    }
    if (splits == 1) return;
    cluster.sync();
    for (int i = kValues * split / splits + tid; i < kValues * (split + 1) / splits; i += kW8fThreads) {
        float v = 0.0f;
        for (int c = 0; c < splits; ++c) v += cluster.map_shared_rank(s_sum, c)[i];
        store(i, v);
    }
    cluster.sync();  // no CTA leaves while another reads its sums
}

template <int DT, int NT, int RT>
static cudaError_t run_w8_few(const W8Args &a, cudaStream_t s) {
    cudaError_t err = cudaSuccess;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    const long long groups = (a.l.row_tiles + RT - 1) / RT;
    int splits = 1;
    while (splits < 8 && groups * splits < 2 * sms && a.l.chunks / (2 * splits) >= kW8fWarps) splits *= 2;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(groups * splits));
    cfg.blockDim = kW8fThreads;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, w8_few_kernel<DT, NT, RT>, a, (a.l.chunks + splits - 1) / splits);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_w8_few(int dtype, const W8Args &a, cudaStream_t s) {
    if (a.tokens <= 8) return dtype ? run_w8_few<1, 1, 1>(a, s) : run_w8_few<0, 1, 1>(a, s);
    return dtype ? run_w8_few<1, 2, 2>(a, s) : run_w8_few<0, 2, 2>(a, s);
}

cudaError_t launch_w8_matmul(int dtype, const W8Args &a, void *workspace, cudaStream_t s) {
    return a.tokens <= kW8FewTokens ? launch_w8_few(dtype, a, s) : launch_w8_tc(dtype, a, workspace, s);
}

}  // namespace qrk
