// qr_w8_tc.cu -- y = x W^T for 17 and more rows of x and weights in 8 bits, on
// tcgen05 (qr_w8_matmul; qr_w8.cu describes the packed order).
//
// The fast integer products of this GPU are those of 16-bit floats: codes are
// exact fp16 numbers, their products exact in fp32.  A first kernel writes x's
// codes as fp16 into the workspace, in the order and with the swizzle that the
// products read from shared memory, so that a chunk of 64 columns of a CTA's
// tokens is one bulk copy.  Then y^T = W x^T, a CTA taking 128 weight rows by N
// tokens over one slice of the columns: eight warps, a row tile each, turn packed
// codes into fp16 and store them as the A operand in tensor memory; one warp
// brings x; one warp issues the products; then the eight warps scale and store.
// The CTAs of a cluster add their slices' sums, in order, through distributed
// shared memory.
//
// A lane's 16 codes of a tile's row are consecutive columns; as fragments of the
// store to tensor memory they stand at the columns 16 j + 4 t + 0..3, so x is
// written into the workspace with its columns exchanged alike.
#include <cooperative_groups.h>

#include "qr_launch.h"
#include "qr_tcgen05.cuh"
#include "qr_w8.cuh"

namespace qrk {

namespace cg = cooperative_groups;

constexpr int kWeThreads = 256;

// x's codes as fp16: a block of N tokens x 64 columns is N * 128 bytes, swizzled.
// A thread takes 32 codes, half of a token's part of a chunk: pieces j, j + 2, ...
__global__ void __launch_bounds__(kWeThreads) w8_expand_kernel(W8Args a, uint8_t *to, int n_shift) {
    chain_entry();
    const int n = 1 << n_shift, chunks = a.l.chunks;
    // eight tokens of two chunks a warp
    const long long token = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 1 & 7);
    if (token >= a.tokens) return;
    const int j = threadIdx.x & 1, row = static_cast<int>(token & (n - 1));
    const int8_t *const src = a.x + token * a.x_stride + j * 32;
    uint8_t *const dst = to + ((token >> n_shift) * chunks << (n_shift + 7));
    for (int c = blockIdx.y * (kWeThreads / 16) + (threadIdx.x >> 4); c < chunks; c += gridDim.y * (kWeThreads / 16)) {
        const int have = a.cols - c * 64 - j * 32;
        const uint4 p = load16_codes(src + c * 64, have), q = load16_codes(src + c * 64 + 16, have - 16);
        const uint32_t u[4] = {p.x, p.y, p.z, p.w}, v[4] = {q.x, q.y, q.z, q.w};
        uint8_t *const block = dst + (static_cast<long long>(c) << (n_shift + 7));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 o;
            codes_f16(u[i], o.x, o.y);
            codes_f16(v[i], o.z, o.w);
            *reinterpret_cast<uint4 *>(block + swizzled(row, 2 * i + j)) = o;
        }
    }
}

constexpr int kWtThreads = 320;  // warps 0-7 codes and results, 8 products, 9 x
constexpr int kWtRows = 128;
constexpr int kWtStep = 4, kWtA = 2;  // chunks of a step, and buffers of codes in tensor memory, a step each
constexpr uint32_t kWtColD = kWtA * 32 * kWtStep, kWtColumns = 512;

template <int N>
struct WtSmem {
    static constexpr int kBlock = N * 128;
    static constexpr int kX = N >= 256 ? 6 : N >= 128 ? 12 : 16;  // chunks of x
    static constexpr int kPitch = kWtRows + 4;
    static_assert(N * kPitch * 4 <= kX * kBlock, "the sums fit where x was");
    uint8_t x[kX * kBlock];  // then the sums
    uint64_t a_full[kWtA], a_done[kWtA], x_full[kX], x_done[kX], d_full;
    float x_scale[N];
    uint32_t tmem;
    int fail;
};

template <int DT, int N>
__global__ void __launch_bounds__(kWtThreads, 1) w8_tc_kernel(W8Args a, const uint8_t *x16, int slice, unsigned *timeouts) {
    using S = WtSmem<N>;
    extern __shared__ uint8_t raw[];
    S &sm = *reinterpret_cast<S *>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int splits = static_cast<int>(cluster.num_blocks()), split = static_cast<int>(cluster.block_rank());
    const int first = split * slice, count = max(0, min(slice, a.l.chunks - first));
    const long long token0 = static_cast<long long>(blockIdx.y) * N;
    const int tokens = static_cast<int>(min(static_cast<long long>(N), a.tokens - token0));
    const int tile0 = blockIdx.x / splits * (kWtRows / 16);
    int *const fail = &sm.fail;
    if (tid == 0) {
        for (int i = 0; i < kWtA; ++i) {
            mbar_init(&sm.a_full[i], 8);
            mbar_init(&sm.a_done[i], 1);
        }
        for (int i = 0; i < S::kX; ++i) {
            mbar_init(&sm.x_full[i], 1);
            mbar_init(&sm.x_done[i], 1);
        }
        mbar_init(&sm.d_full, 1);
        mbar_init_fence();
        sm.fail = 0;
    }
    if (warp == 8) tc_alloc(&sm.tmem, kWtColumns);
    chain_entry();
    for (int i = tid; i < tokens; i += kWtThreads) sm.x_scale[i] = a.x_scales[token0 + i];
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const int steps = (count + kWtStep - 1) / kWtStep;
    const int quarter = warp & 3;  // of tensor memory's lanes, that this warp reaches

    if (warp < 8) {
        // ---- codes: a row tile of 16, two steps of them on their way in registers
        const long long tile = min(tile0 + 2 * quarter + (warp >> 2), a.l.row_tiles - 1);
        const uint4 *const src = reinterpret_cast<const uint4 *>(a.packed) + (tile * a.l.chunks + first) * 64 + lane;
        uint4 w[2][kWtStep][2];
        auto fetch = [&](int b, int p) {
#pragma unroll
            for (int u = 0; u < kWtStep; ++u)
                if (kWtStep * p + u < count) {
                    w[b][u][0] = __ldg(src + (kWtStep * p + u) * 64);
                    w[b][u][1] = __ldg(src + (kWtStep * p + u) * 64 + 32);
                }
        };
        fetch(0, 0);
        fetch(1, 1);
        const uint32_t to = tmem + (static_cast<uint32_t>(quarter * 32 + (warp >> 2) * 16) << 16);
        bool ok = true;
        for (int p0 = 0; p0 < steps && ok; p0 += 2) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int p = p0 + b;
                if (p >= steps) break;
                if (p >= kWtA) ok = tc_wait_warp(&sm.a_done[b], (p / kWtA - 1) & 1, fail, timeouts);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int u = 0; u < kWtStep; ++u) {
                    const uint32_t up[4] = {w[b][u][0].x, w[b][u][0].y, w[b][u][0].z, w[b][u][0].w},
                                   low[4] = {w[b][u][1].x, w[b][u][1].y, w[b][u][1].z, w[b][u][1].w};
                    uint32_t v[16];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        weights_f16(up[j], v[4 * j], v[4 * j + 1]);
                        weights_f16(low[j], v[4 * j + 2], v[4 * j + 3]);
                    }
                    tc_st_fragments(to + b * (32 * kWtStep) + u * 32, v);  // (past the last chunk: unused)
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.a_full[b]);
                fetch(b, p + 2);
            }
        }
    } else if (warp == 8) {
        // ---- products
        const bool leader = elect_lane();
        constexpr uint32_t kDesc = mma_desc(N, false);
        bool ok = true;
        for (int p = 0; p < steps && ok; ++p) {
            const int s = p % kWtA, chunks = min(kWtStep, count - kWtStep * p);
            ok = tc_wait_warp(&sm.a_full[s], (p / kWtA) & 1, fail, timeouts);
            for (int u = 0; u < chunks && ok; ++u) {
                const int i = kWtStep * p + u, xs = i % S::kX;
                ok = tc_wait_warp(&sm.x_full[xs], (i / S::kX) & 1, fail, timeouts);
                if (!ok) break;
                tc_fence_after();
                const uint32_t x = smem_addr(sm.x) + xs * S::kBlock, codes = tmem + s * (32 * kWtStep) + u * 32;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    tc_mma_ts(leader, tmem + kWtColD, codes + j * 8, smem_desc(x + j * 32, 16, 1024), kDesc, i + j > 0);
                tc_commit(leader, &sm.x_done[xs]);
            }
            if (ok) tc_commit(leader, &sm.a_done[s]);
        }
        tc_commit(leader, &sm.d_full);
    } else if (lane == 0) {
        // ---- x: a chunk's block is one copy
        const uint8_t *const src = x16 + (blockIdx.y * static_cast<long long>(a.l.chunks) + first) * S::kBlock;
        bool ok = true;
        int i = 0;
        for (; i < count; ++i) {
            const int xs = i % S::kX;
            if (i >= S::kX) ok = tc_wait(&sm.x_done[xs], (i / S::kX - 1) & 1, fail, timeouts);
            if (!ok) break;
            mbar_arrive_expect_tx(&sm.x_full[xs], S::kBlock);
            bulk_copy_g2s(sm.x + xs * S::kBlock, src + static_cast<long long>(i) * S::kBlock, S::kBlock, &sm.x_full[xs]);
        }
        // none of the copies is on its way when the CTA leaves
        for (int k = max(0, i - S::kX); k < i; ++k) mbar_wait(&sm.x_full[k % S::kX], (k / S::kX) & 1);
    }
    __syncwarp();

    // the slice's sums as [token][row], then every CTA of the cluster adds the
    // slices, in order, for its share of them
    const bool done = tc_wait_warp(&sm.d_full, 0, fail, timeouts);
    tc_fence_after();
    __syncthreads();  // (x's buffers are free)
    float *const sums = reinterpret_cast<float *>(sm.x);
    if (warp < 8) {
        constexpr int kMine = N / 2;
        const int from = (warp >> 2) * kMine;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kWtColD + from;
#pragma unroll
        for (int h = 0; h < kMine / 16; ++h) {
            uint32_t v[16];
            tc_ld16(lanes + h * 16, v);
            tc_wait_ld(v);
#pragma unroll
            for (int e = 0; e < 16; ++e)
                sums[(from + h * 16 + e) * S::kPitch + quarter * 32 + lane] = count > 0 && done ? __uint_as_float(v[e]) : 0.0f;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tc_free(tmem, kWtColumns);
    if (splits > 1) cluster.sync();
    const long long row0 = tile0 * 16ll;
    const int mine0 = tokens * kWtRows * split / splits, mine1 = tokens * kWtRows * (split + 1) / splits;
    const float *const scales = reinterpret_cast<const float *>(a.packed + a.l.scales_at) + row0;
    for (int i = mine0 + tid; i < mine1; i += kWtThreads) {
        const int m = i / kWtRows, row = i % kWtRows;
        float v = 0.0f;
        if (splits > 1)
            for (int c = 0; c < splits; ++c) v += cluster.map_shared_rank(sums, c)[m * S::kPitch + row];
        else
            v = sums[m * S::kPitch + row];
        if (row0 + row < a.rows) a.y[(token0 + m) * a.y_stride + row0 + row] = narrow1<DT>(v * sm.x_scale[m] * scales[row]);
    }
    if (splits > 1) cluster.sync();  // no CTA leaves while another reads its sums
}

template <int DT, int N>
static cudaError_t run_w8_tc(const W8Args &a, const uint8_t *x16, cudaStream_t s) {
    auto kern = w8_tc_kernel<DT, N>;
    const int bytes = sizeof(WtSmem<N>) + 1024;
    cudaError_t err = allow_dynamic_smem(reinterpret_cast<const void *>(kern), bytes);
    if (err != cudaSuccess) return err;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    unsigned *timeouts = wait_timeout_counter(&err);
    if (!timeouts) return err;
    const long long row_ctas = (a.l.row_tiles + 7) / 8, token_ctas = (a.tokens + N - 1) / N;
    int splits = 1;
    long long best = -1;
    for (int n = 1; n <= 8; n *= 2) {
        const long long waves = (row_ctas * token_ctas * n + sms - 1) / sms, cost = waves * ((a.l.chunks + n - 1) / n + 12);
        if (best < 0 || cost < best) best = cost, splits = n;
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = kWtThreads;
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    // a grid's second dimension, the tokens' tiles, ends at 65535: more tokens are more launches
    for (long long done = 0; done < token_ctas; done += 65535) {
        const long long now = token_ctas - done < 65535 ? token_ctas - done : 65535;
        W8Args part = a;
        part.tokens = a.tokens - done * N < now * N ? a.tokens - done * N : now * N;
        part.x_scales += done * N;
        part.y += done * N * a.y_stride;
        cfg.gridDim = dim3(static_cast<unsigned>(row_ctas * splits), static_cast<unsigned>(now));
        err = cudaLaunchKernelEx(&cfg, kern, part, x16 + done * a.l.chunks * WtSmem<N>::kBlock,
                                 (a.l.chunks + splits - 1) / splits, timeouts);
        if (err == cudaSuccess) err = cudaGetLastError();
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

// Tokens of a CTA: the fewest that take them all, 256 at most.
static int w8_token_shift(long long tokens) { return tokens <= 32 ? 5 : tokens <= 64 ? 6 : tokens <= 128 ? 7 : 8; }

size_t w8_workspace(long long tokens, int cols) {
    const long long n = 1ll << w8_token_shift(tokens);
    return static_cast<size_t>((tokens + n - 1) / n * n) * (static_cast<size_t>(cols) / 64 + (cols % 64 != 0)) * 128;
}

template <int DT>
static cudaError_t pick_tokens(int shift, const W8Args &a, const uint8_t *x16, cudaStream_t s) {
    switch (shift) {
        case 5: return run_w8_tc<DT, 32>(a, x16, s);
        case 6: return run_w8_tc<DT, 64>(a, x16, s);
        case 7: return run_w8_tc<DT, 128>(a, x16, s);
        default: return run_w8_tc<DT, 256>(a, x16, s);
    }
}

cudaError_t launch_w8_tc(int dtype, const W8Args &a, void *workspace, cudaStream_t s) {
    const int shift = w8_token_shift(a.tokens);
    uint8_t *const x16 = static_cast<uint8_t *>(workspace);
    const int sweep = (a.l.chunks + kWeThreads / 16 - 1) / (kWeThreads / 16);
    const dim3 grid(static_cast<unsigned>((a.tokens + 7) / 8), static_cast<unsigned>(sweep < 65535 ? sweep : 65535));
    const cudaError_t err = launch_chained(w8_expand_kernel, grid, kWeThreads, 0, s, a, x16, shift);
    if (err != cudaSuccess) return err;
    return dtype ? pick_tokens<1>(shift, a, x16, s) : pick_tokens<0>(shift, a, x16, s);
}

}  // namespace qrk
