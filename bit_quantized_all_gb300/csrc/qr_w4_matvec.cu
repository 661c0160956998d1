// qr_w4_matvec.cu -- y = x W^T for few rows of x and 4-bit weights with group
// scales (qr_w4_matvec); qr_w4.cu describes the packed order.
//
// y^T = W x^T on m16n8k16: 16 weight rows as M, 8 tokens as N.  A lane's 16
// bytes of a 16 x 64 tile are its A fragments of four instructions, read
// straight from HBM into registers; a code u becomes the type's integer
// 1024 + u (bf16: 128 + u) by an or, and 1024 + z is subtracted, both exact.
// A group's products are accumulated apart and added scaled by its fp32
// scale, so the weights are never rounded.
//
// A CTA's eight warps take RT row tiles each over one slice of the columns,
// sharing the slice of x in shared memory; the CTAs of a cluster take the
// slices of the same rows and add their sums, in slice order, through
// distributed shared memory: no workspace, no second launch.
//
// What bounds it: latency.  No unit is full (16 tokens through 8192 x 8192 with
// zero points 16.9 us, 2.1 TB/s of weights: issue 44%, tensor pipe 22%, DRAM
// 22%): a CTA has some 16 chunks between its first loads and its cluster's join.
// For one token through 8192 x 1024, 4.8 us, the launch and its round trips.
#include <cooperative_groups.h>

#include "qr_launch.h"
#include "qr_w4.cuh"

namespace qrk {

namespace cg = cooperative_groups;

constexpr int kMvWarps = 8, kMvThreads = 32 * kMvWarps;
constexpr int kMvDepth = 4;  // chunks of weights in flight per warp

template <int DT>
__device__ __forceinline__ void mma_typed(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool first) {
    const float c0 = first ? 0.0f : d[0], c1 = first ? 0.0f : d[1], c2 = first ? 0.0f : d[2], c3 = first ? 0.0f : d[3];
    if constexpr (DT == 0) {
        mma_f16(d, a, b0, b1, c0, c1, c2, c3);
    } else {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    }
}

template <int NT>
struct MatvecSmem {
    static constexpr int kPanel = 16;                      // chunks of x held at a time
    static_assert(kPanel % kMvDepth == 0, "panels change between rounds of chunks");
    static constexpr int kPitch = kPanel * 128 + 32;       // bytes of a token's row: no bank conflicts
    static constexpr int kBuffer = 8 * NT * kPitch;
    static constexpr int kBytes = 2 * kBuffer;
};

// CTAs per SM: with a row tile a warp four (one token through 20480 x 5120 20.0
// us, with three 23.4), or three where zero points of groups of 32 would spill
// (8 tokens through 8192 x 8192 17.0 us, with four 19.3).
template <int RT, int NG, bool ZEROS>
constexpr int kMvCtas = RT == 2 ? 2 : NG == 2 && ZEROS ? 3 : 4;

// NG: groups of a 64-column chunk (2 for groups of 32, else 1).
template <int DT, int RT, int NT, int NG, bool ZEROS>
__global__ void __launch_bounds__(kMvThreads, kMvCtas<RT, NG, ZEROS>) w4_matvec_kernel(W4MatvecArgs a, int slice, bool vector) {
    chain_entry();
    using S = MatvecSmem<NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int splits = static_cast<int>(cluster.num_blocks()), split = static_cast<int>(cluster.block_rank());
    const int first = split * slice, count = max(0, min(slice, a.l.chunks - first));
    const long long token0 = static_cast<long long>(blockIdx.y) * (8 * NT);
    const int tokens = static_cast<int>(min(static_cast<long long>(8 * NT), a.tokens - token0));
    const int tile0 = (blockIdx.x / splits * kMvWarps + warp) * RT;
    const uint32_t base = smem_addr(smem);

    // x: panel p of the slice into buffer p % 2; rows past the tokens and
    // columns past the last are zero
    auto load_panel = [&](int p) {
        const int chunks = min(S::kPanel, count - p * S::kPanel), pieces = chunks * 8;
        const int col0 = (first + p * S::kPanel) * 64;
        uint8_t *const dst = smem + (p & 1) * S::kBuffer;
        for (int i = tid; i < tokens * pieces; i += kMvThreads) {
            const int m = i / pieces, q = i % pieces, col = col0 + q * 8;
            const uint16_t *src = a.x + (token0 + m) * a.x_stride + col;
            uint8_t *const to = dst + m * S::kPitch + q * 16;
            const int have = min(8, a.cols - col);
            if (vector && have == 8)
                copy16_async(smem_addr(to), src);
            else
                *reinterpret_cast<uint4 *>(to) = load8_any(src, have);
        }
        copy_commit();
    };

    uint4 w[kMvDepth][RT];
    uint32_t s[kMvDepth][RT][NG];
    uint16_t z[kMvDepth][RT][ZEROS ? NG : 1];
    const uint4 *wp[RT];
    const uint32_t *sp[RT];
    const uint16_t *zp[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const long long tile = min(tile0 + r, a.l.row_tiles - 1);
        wp[r] = reinterpret_cast<const uint4 *>(a.packed) + (tile * a.l.chunks + first) * 32 + lane;
        sp[r] = reinterpret_cast<const uint32_t *>(a.packed + a.l.scales_at) + tile * a.l.groups * 8 + g;
        zp[r] = reinterpret_cast<const uint16_t *>(a.packed + a.l.zeros_at) + tile * a.l.groups * 8 + g;
    }
    auto fetch = [&](int d, int i) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            w[d][r] = __ldcs(wp[r] + i * 32);
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const int gi = NG == 2 ? (first + i) * 2 + n : (first + i) >> (a.group_shift - 1);
                s[d][r][n] = sp[r][gi * 8];
                if constexpr (ZEROS) z[d][r][n] = zp[r][gi * 8];
            }
        }
    };
#pragma unroll
    for (int d = 0; d < kMvDepth; ++d)
        if (d < count) fetch(d, d);
    for (int i = tid; i < (8 * NT - tokens) * (S::kPitch / 16); i += kMvThreads) {
        const int m = tokens + i / (S::kPitch / 16), q = i % (S::kPitch / 16);
        *reinterpret_cast<uint4 *>(smem + m * S::kPitch + q * 16) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(smem + S::kBuffer + m * S::kPitch + q * 16) = make_uint4(0, 0, 0, 0);
    }
    if (count > 0) load_panel(0);

    float acc[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[r][n][k] = 0.0f;

    for (int i0 = 0; i0 < count; i0 += kMvDepth) {
        if (i0 % S::kPanel == 0) {
            const int p = i0 / S::kPanel;
            if (i0) __syncthreads();  // every warp has left the buffer that is filled next
            if (i0 + S::kPanel < count) {
                load_panel(p + 1);
                copy_wait<1>();
            } else {
                copy_wait<0>();
            }
            __syncthreads();
        }
        const uint32_t xb = base + (i0 / S::kPanel & 1) * S::kBuffer + g * S::kPitch + t * 8;
#pragma unroll
        for (int d = 0; d < kMvDepth; ++d) {
            const int i = i0 + d;
            if (i >= count) break;
            const uint32_t xa = xb + (i % S::kPanel) * 128;
            uint2 xv[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) xv[n][j] = lds64(xa + n * 8 * S::kPitch + j * 32);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t ww[4] = {w[d][r].x, w[d][r].y, w[d][r].z, w[d][r].w};
                float part[NT][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t z0 = DT == 0 ? 0x64086408u : 0x43084308u, z1 = z0;
                    if constexpr (ZEROS) {
                        const uint32_t zz = z[d][r][NG == 2 ? j >> 1 : 0];
                        z0 = ((zz & 15u) * 0x00010001u) | (DT == 0 ? 0x64006400u : 0x43004300u);
                        z1 = ((zz >> 8) * 0x00010001u) | (DT == 0 ? 0x64006400u : 0x43004300u);
                    }
                    const uint32_t af[4] = {code_pair<DT>(ww[j], z0), code_pair<DT>(ww[j] >> 4, z1),
                                            code_pair<DT>(ww[j] >> 8, z0), code_pair<DT>(ww[j] >> 12, z1)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_typed<DT>(part[n], af, xv[n][j].x, xv[n][j].y, NG == 2 ? (j & 1) == 0 : j == 0);
                    }
                    if (NG == 2 ? (j & 1) == 1 : j == 3) {
                        const float2 sc = __half22float2(*reinterpret_cast<const __half2 *>(&s[d][r][NG == 2 ? j >> 1 : 0]));
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            acc[r][n][0] = __fmaf_rn(part[n][0], sc.x, acc[r][n][0]);
                            acc[r][n][1] = __fmaf_rn(part[n][1], sc.x, acc[r][n][1]);
                            acc[r][n][2] = __fmaf_rn(part[n][2], sc.y, acc[r][n][2]);
                            acc[r][n][3] = __fmaf_rn(part[n][3], sc.y, acc[r][n][3]);
                        }
                    }
                }
            }
            if (i + kMvDepth < count) fetch(d, i + kMvDepth);
        }
    }

    // the slice's sums as [token][row] in shared memory, then every CTA of the
    // cluster adds the slices, in order, for its share of them
    constexpr int kRowsCta = 16 * RT * kMvWarps, kSumPitch = kRowsCta + 4;
    float *const sums = reinterpret_cast<float *>(smem);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int m = n * 8 + 2 * t + (k & 1);
                if (m < tokens) sums[m * kSumPitch + (warp * RT + r) * 16 + g + 8 * (k >> 1)] = acc[r][n][k];
            }
    if (splits > 1) cluster.sync(); else __syncthreads();
    const int row0 = blockIdx.x / splits * kRowsCta;
    const int mine0 = tokens * kRowsCta * split / splits, mine1 = tokens * kRowsCta * (split + 1) / splits;
    for (int i = mine0 + tid; i < mine1; i += kMvThreads) {
        const int m = i / kRowsCta, row = i % kRowsCta;
        float v = 0.0f;
        for (int c = 0; c < splits; ++c) v += cluster.map_shared_rank(sums, c)[m * kSumPitch + row];
        if (row0 + row < a.rows)
            a.y[(token0 + m) * a.y_stride + row0 + row] =
                DT ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
    }
    if (splits > 1) cluster.sync();  // no CTA leaves while another reads its sums
}

template <int DT, int RT, int NT, int NG, bool ZEROS>
static cudaError_t run_matvec(const W4MatvecArgs &a, cudaStream_t s) {
    using S = MatvecSmem<NT>;
    constexpr int kSums = 8 * NT * (16 * RT * kMvWarps + 4) * 4;
    constexpr int kBytes = S::kBytes > kSums ? S::kBytes : kSums;
    auto kern = w4_matvec_kernel<DT, RT, NT, NG, ZEROS>;
    cudaError_t err = allow_dynamic_smem(reinterpret_cast<const void *>(kern), kBytes);
    if (err != cudaSuccess) return err;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    const long long row_ctas = (a.l.row_tiles + RT * kMvWarps - 1) / (RT * kMvWarps);
    const long long token_ctas = (a.tokens + 8 * NT - 1) / (8 * NT);
    // the number of slices whose waves of CTAs, each its chunks and about three
    // more to start and end, are shortest (8192 x 8192, one token, with three CTAs
    // an SM: 6 slices 14.3 us, 4 18.0, 8, which did not fit at once, 16.8; clusters
    // of 5 and 7 leave SMs of a processing cluster idle)
    int splits = 1;
    long long best = -1;
    for (int n : {1, 2, 3, 4, 6, 8}) {
        const long long slots = static_cast<long long>(kMvCtas<RT, NG, ZEROS>) * sms, waves = (row_ctas * token_ctas * n + slots - 1) / slots;
        const long long cost = waves * ((a.l.chunks + n - 1) / n + 3);
        if (best < 0 || (n <= a.l.chunks && cost < best)) best = cost, splits = n;
    }
    const int slice = ((a.l.chunks + splits - 1) / splits);
    const bool vector = w4_x_aligned(a.x, a.tokens, a.x_stride);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(row_ctas * splits), static_cast<unsigned>(token_ctas));
    cfg.blockDim = kMvThreads;
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, kern, a, slice, vector);
    return err != cudaSuccess ? err : cudaGetLastError();
}

template <int DT, int RT, int NT>
static cudaError_t pick_group(const W4MatvecArgs &a, bool zeros, cudaStream_t s) {
    if (a.group_shift == 0)
        return zeros ? run_matvec<DT, RT, NT, 2, true>(a, s) : run_matvec<DT, RT, NT, 2, false>(a, s);
    return zeros ? run_matvec<DT, RT, NT, 1, true>(a, s) : run_matvec<DT, RT, NT, 1, false>(a, s);
}

template <int DT>
static cudaError_t pick_tokens(const W4MatvecArgs &a, bool zeros, void *workspace, cudaStream_t s) {
    if (a.tokens <= 8) return pick_group<DT, 1, 1>(a, zeros, s);
    if (a.tokens <= kW4FewTokens) {
        // two row tiles a warp read x half as often, one makes twice the CTAs.
        // 16 tokens through 8192 columns, with two and with one: 64 row tiles
        // 9.7 and 7.9 us, 96 10.2 and 9.8, 128 11.7 and 11.4, 152 13.1 and 12.8,
        // 256 14.8 and 14.3, 512 15.7 and 22.0 (9 tokens 15.3 and 21.2): near 152
        // either will do, below one is better, far above two
        if (a.l.row_tiles >= 152) return pick_group<DT, 2, 2>(a, zeros, s);
        return pick_group<DT, 1, 2>(a, zeros, s);
    }
    return launch_w4_tc(DT, a, zeros, workspace, s);
}

cudaError_t launch_w4_matvec(int dtype, long long tokens, const void *x, long long x_stride, int rows, int cols,
                             int group, bool has_zeros, const void *packed, void *y, long long y_stride,
                             void *workspace, cudaStream_t s) {
    W4MatvecArgs a;
    a.x = static_cast<const uint16_t *>(x);
    a.y = static_cast<uint16_t *>(y);
    a.packed = static_cast<const uint8_t *>(packed);
    a.x_stride = x_stride;
    a.y_stride = y_stride;
    a.tokens = tokens;
    a.rows = rows;
    a.cols = cols;
    a.group_shift = group == 32 ? 0 : group == 64 ? 1 : 2;
    a.l = w4_layout(rows, cols, group, has_zeros);
    return dtype ? pick_tokens<1>(a, has_zeros, workspace, s) : pick_tokens<0>(a, has_zeros, workspace, s);
}

}  // namespace qrk
