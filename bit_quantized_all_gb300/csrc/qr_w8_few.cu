// qr_w8_few.cu -- y = x W^T for up to 16 rows of x and weights in 8 bits
// (qr_w8_matmul); W8Layout in qr_serving.h describes the packed order.
//
// y^T = W x^T on m16n8k16 with fp16 operands: 16 weight rows as M, 8 tokens as
// N, both sides' codes as exact fp16 integers.  Which of an instruction's
// columns stands at which of its places is free as long as both sides agree: a
// lane takes 16 consecutive columns of its rows, one 16-byte load of a packed
// tile's row, and of its token's row, and they serve four instructions.
//
// The row tiles are divided evenly among CTAs that all run at once, up to RT tiles
// each.  The warps of a CTA take the chunks of its slice of the columns in turn, for
// all of its tiles, and add their sums in order through shared memory; where there
// are few row tiles and long rows, the CTAs of a cluster take the slices of the same
// rows and add theirs through distributed shared memory.
//
// What bounds it: the weights' bytes and, with 16 tokens, x, which every CTA reads
// and converts for itself (10240 x 8192: 8 tokens 16.2 us, 5.2 TB/s, without loading x
// 14.5; 16 tokens 20 us, without loading x 16.5).  Shares of whole single rows, so
// that all SMs have the same bytes, were slower at every size (8 tokens 18.8 us):
// their tiles of eight rows use each x for half as many rows.
#include <cooperative_groups.h>

#include "qr_launch.h"
#include "qr_w8.cuh"

namespace qrk {

namespace cg = cooperative_groups;

// NT: tiles of eight tokens; RT: most tiles of 16 rows; kWarps of a CTA, with kDepth
// chunks each on their way; CTAS on an SM.  The first `more` clusters have `each` + 1
// row tiles, the others `each`.
template <int DT, int NT, int RT, int kWarps, int kDepth, int CTAS>
__global__ void __launch_bounds__(32 * kWarps, CTAS) w8_few_kernel(W8Args a, int slice, int each, int more) {
    chain_entry();
    constexpr int kThreads = 32 * kWarps;
    constexpr int kRows = 16 * RT, kTokens = 8 * NT, kValues = kRows * kTokens;
    __shared__ float s_part[kWarps][kTokens][kRows + 4];
    __shared__ float s_sum[kValues];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int splits = static_cast<int>(cluster.num_blocks()), split = static_cast<int>(cluster.block_rank());
    const int first = split * slice, count = max(0, min(slice, a.l.chunks - first));
    const int group = blockIdx.x / splits;
    const int tile0 = group * each + min(group, more), tiles = each + (group < more ? 1 : 0);
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

    uint4 w[kDepth][RT][2], x[kDepth][NT];
    auto fetch = [&](int d, int i) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
            if (r == 0 || r < tiles)
#pragma unroll
                for (int h = 0; h < 2; ++h) w[d][r][h] = __ldcs(wp[r] + i * 64ll + h * 32);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            x[d][n] = n * 8 + g < tokens ? load16_codes(xp[n] + i * 64ll, cols - i * 64) : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        if (warp + d * kWarps < count) fetch(d, warp + d * kWarps);

    float acc[RT][NT][4] = {};
    for (int i0 = warp; i0 < count; i0 += kDepth * kWarps) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            const int i = i0 + d * kWarps;
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
                if (r && r >= tiles) break;
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
            const int next = i + kDepth * kWarps;
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
        if (m < tokens && row < 16 * tiles && tile0 * 16ll + row < a.rows)
            a.y[m * a.y_stride + tile0 * 16ll + row] = narrow1<DT>(v * a.x_scales[m] * scales[row]);
    };
    for (int i = tid; i < kValues; i += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) v += s_part[k][i / kRows][i % kRows];
        if (splits == 1) store(i, v); else s_sum[i] = v;
    }
    if (splits == 1) return;
    cluster.sync();
    for (int i = kValues * split / splits + tid; i < kValues * (split + 1) / splits; i += kThreads) {
        float v = 0.0f;
        for (int c = 0; c < splits; ++c) v += cluster.map_shared_rank(s_sum, c)[i];
        store(i, v);
    }
    cluster.sync();  // no CTA leaves while another reads its sums
}

template <int DT, int NT, int RT, int kWarps, int kDepth, int CTAS>
static cudaError_t run_w8_few(const W8Args &a, int groups, int splits, cudaStream_t s) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(groups) * splits));
    cfg.blockDim = 32 * kWarps;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, w8_few_kernel<DT, NT, RT, kWarps, kDepth, CTAS>, a,
                                             (a.l.chunks + splits - 1) / splits, a.l.row_tiles / groups,
                                             a.l.row_tiles % groups);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// CTAs for at most RT row tiles each: a multiple of `wave`, the CTAs of all SMs.
template <int DT, int NT, int RT, int kWarps, int kDepth, int CTAS>
static cudaError_t run_w8_waves(const W8Args &a, long long wave, cudaStream_t s) {
    const long long waves = (a.l.row_tiles + RT * wave - 1) / (RT * wave);
    return run_w8_few<DT, NT, RT, kWarps, kDepth, CTAS>(
        a, static_cast<int>(min(wave * waves, static_cast<long long>(a.l.row_tiles))), 1, s);
}

template <int DT>
static cudaError_t pick_w8_few(const W8Args &a, cudaStream_t s) {
    cudaError_t err = cudaSuccess;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    const int tiles = a.l.row_tiles;
    // Up to three tiles an SM: each a CTA of eight warps, for many columns at once.
    // Slices cost a cluster, some 2.4 us (8 tokens through 8192 x 1024: one slice 3.5
    // us, two 5.9), and save rounds of loads (8 tokens through 1280 x 8192: one slice
    // 7.7 us, four 5.0) as long as all CTAs run at once (16 tokens through 2048 x
    // 8192: two slices 7.1 us, four 10.0).
    if (tiles <= 3ll * sms) {
        int splits = 1;
        if (a.l.chunks > 64)
            while (splits < 8 && 2ll * tiles * splits <= 3ll * sms && a.l.chunks / (2 * splits) >= 8) splits *= 2;
        if (a.tokens <= 8) return run_w8_few<DT, 1, 1, 8, 4, 3>(a, tiles, splits, s);
        // more chunks on their way where two CTAs an SM do (4096 x 4096: 6.1 and 7.3
        // us), else three CTAs (5120 x 5120: 11.4 and 8.8)
        return tiles * splits <= 2 * sms ? run_w8_few<DT, 2, 1, 8, 4, 2>(a, tiles, splits, s)
                                         : run_w8_few<DT, 2, 1, 8, 2, 3>(a, tiles, splits, s);
    }
    // More: the form in which all CTAs run at once with the most loads on their way.
    // Of tiles that share a CTA, x is read once.  In us, with 8 and 16 tokens:
    //                      8192 x 8192  10240 x 8192  14336 x 4096  20480 x 5120  28672 x 4096
    //   8: 1 tile, 8 warps    16.5          17.7          13.0          20.3          23.1
    //      2 tiles, 8 warps   13.1          18.4          13.7          21.3          23.3
    //      1 tile, 4 warps    15.9          16.6          11.7          21.1          21.0
    //      3 tiles, 4 warps   16.5          17.6          13.0          19.1          23.2
    //  16: 1 tile, 8 warps    20.2          20.9          14.4          23.7          26.6
    //      2 tiles, 8 warps   15.4          23.9          16.1          25.9          25.4
    //      2 tiles, 4 warps   19.3          20.5          13.8          25.9          25.6
    //      4 tiles, 4 warps   25.1          27.0          17.0          22.0          23.3
    if (a.tokens <= 8) {
        if (tiles <= 4ll * sms) return run_w8_waves<DT, 1, 2, 8, 4, 2>(a, 2ll * sms, s);
        if (tiles > 6ll * sms && tiles <= 9ll * sms) return run_w8_waves<DT, 1, 3, 4, 4, 3>(a, 3ll * sms, s);
        return run_w8_few<DT, 1, 1, 4, 4, 6>(a, tiles, 1, s);
    }
    if (tiles <= 4ll * sms) return run_w8_waves<DT, 2, 2, 8, 2, 2>(a, 2ll * sms, s);
    if (tiles <= 6ll * sms) return run_w8_waves<DT, 2, 2, 4, 4, 3>(a, 3ll * sms, s);
    return run_w8_waves<DT, 2, 4, 4, 2, 3>(a, 3ll * sms, s);
}

cudaError_t launch_w8_few(int dtype, const W8Args &a, cudaStream_t s) {
    return dtype ? pick_w8_few<1>(a, s) : pick_w8_few<0>(a, s);
}

cudaError_t launch_w8_matmul(int dtype, const W8Args &a, void *workspace, cudaStream_t s) {
    return a.tokens <= kW8FewTokens ? launch_w8_few(dtype, a, s) : launch_w8_tc(dtype, a, workspace, s);
}

}  // namespace qrk
