// qr_w4_tc.cu -- y = x W^T for 17 and more rows of x and 4-bit weights with
// group scales, on tcgen05 (qr_w4_matvec; qr_w4.cu describes the packed order).
//
// y^T = W x^T, a CTA taking 128 weight rows by up to 64 tokens over one slice of
// the columns, a step of four chunks of 64 columns at a time.  Eight warps, a row tile each,
// turn codes into the type's exact integers u - z and store them as the A operand
// in tensor memory: the packed words are the fragments of that store, so nothing
// is exchanged.  Four warps bring x into shared memory.  One warp issues the
// products.  As scales differ from group to group, each group's (or chunk's, for
// groups of 64 and 128) products go to a ring of accumulators of their own, and
// eight warps, a thread per row and half of the tokens, add them scaled in fp32:
// the weights are never rounded.  The CTAs of a cluster add their slices' sums,
// in order, through distributed shared memory.
//
// What bounds it: the warps' latencies, of which two a scheduler hide each
// other's in the conversion and in the sums, above the codes from HBM (4 KB a
// chunk, 178 cycles of an SM's share): some 700 cycles a chunk (64 tokens
// through 20481 x 5123 52.7 us, 1.1 TB/s of weights, 255 TFLOP/s).
#include <cooperative_groups.h>

#include "qr_launch.h"
#include "qr_tcgen05.cuh"
#include "qr_w4.cuh"

namespace qrk {

namespace cg = cooperative_groups;

constexpr int kWtThreads = 672;  // warps 0-7 codes, 8-15 sums, 16 products, 17-20 x
constexpr int kWtRows = 128;
// A barrier's arrival and wait cost about as much as a chunk's work, so buffers
// are handed on by the step, and accumulators two at a time.
constexpr int kWtStep = 4;             // chunks
constexpr int kWtA = 2, kWtD = 2;      // buffers of codes (a step each) and of accumulators (two each)
constexpr int kWtAhead = 4;            // steps of codes on their way
constexpr uint32_t kWtColD = kWtA * 32 * kWtStep, kWtColumns = 512;
constexpr int kWtX = 4, kWtXAhead = 2;  // buffers of x, a step each; of them on their way

template <int N>
struct WtSmem {
    uint8_t x[kWtX * kWtStep * N * 128];        // then the sums
    uint8_t codes[8][kWtAhead][kWtStep][512];   // by warp: its row tile
    uint8_t zeros[8][kWtAhead][kWtStep][32];
    uint8_t scales[8][kWtAhead][kWtStep][128];  // by warp: its quarter's two row tiles
    uint64_t a_full[kWtA], a_done[kWtA], x_full[kWtX], x_done[kWtX], d_full[kWtD], d_done[kWtD];
    uint32_t tmem;
    int fail;
};

// N: tokens of a CTA; NG: groups of a 64-column chunk (2 for groups of 32, else 1).
template <int DT, int N, int NG, bool ZEROS>
__global__ void __launch_bounds__(kWtThreads, 1) w4_tc_kernel(W4MatvecArgs a, int slice, unsigned *timeouts) {
    chain_entry();
    using S = WtSmem<N>;
    extern __shared__ uint8_t raw[];
    S &sm = *reinterpret_cast<S *>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2;
    const int splits = static_cast<int>(cluster.num_blocks()), split = static_cast<int>(cluster.block_rank());
    const int first = split * slice, count = max(0, min(slice, a.l.chunks - first));
    const long long token0 = static_cast<long long>(blockIdx.y) * N;
    const int tokens = static_cast<int>(min(static_cast<long long>(N), a.tokens - token0));
    const int tile0 = blockIdx.x / splits * (kWtRows / 16);
    int *const fail = &sm.fail;

    constexpr int kXStep = kWtStep * N * 128;
    if (tid == 0) {
        for (int i = 0; i < kWtA; ++i) {
            mbar_init(&sm.a_full[i], 256);
            mbar_init(&sm.a_done[i], 1);
        }
        for (int i = 0; i < kWtX; ++i) {
            mbar_init(&sm.x_full[i], 128);
            mbar_init(&sm.x_done[i], 1);
        }
        for (int i = 0; i < kWtD; ++i) {
            mbar_init(&sm.d_full[i], 1);
            mbar_init(&sm.d_done[i], 256);
        }
        mbar_init_fence();
        sm.fail = 0;
    }
    if (warp == 16) tc_alloc(&sm.tmem, kWtColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const int steps = (count + kWtStep - 1) / kWtStep;
    const int quarter = warp & 3;  // of tensor memory's lanes, that this warp reaches
    constexpr int kMine = N / 2;
    float acc[kMine];  // of the sums' threads: this row's, half of the tokens
    auto group_of = [&](int i, int n) { return NG == 2 ? (first + i) * 2 + n : (first + i) >> (a.group_shift - 1); };

    if (warp < 8) {
        // ---- codes: a row tile of 16
        const uint32_t codes = smem_addr(sm.codes[warp]);
        const long long tile = min(tile0 + 2 * quarter + (warp >> 2), a.l.row_tiles - 1);
        const uint8_t *const src = a.packed + (tile * a.l.chunks + first) * 512 + lane * 16;
        const uint8_t *const zsrc = a.packed + a.l.zeros_at + tile * a.l.groups * 16;
        auto fetch = [&](int p) {
            const uint32_t slot = p % kWtAhead;
#pragma unroll
            for (int u = 0; u < kWtStep; ++u)
                if (kWtStep * p + u < count)
                    copy16_async(codes + (slot * kWtStep + u) * 512 + lane * 16, src + (kWtStep * p + u) * 512ll);
            if (ZEROS && lane < kWtStep * NG && kWtStep * p + lane / NG < count)
                copy16_async(smem_addr(sm.zeros[warp][slot][lane / NG]) + lane % NG * 16,
                             zsrc + group_of(kWtStep * p + lane / NG, lane % NG) * 16);
            copy_commit();
        };
        for (int p = 0; p < kWtAhead - 1; ++p) fetch(p);
        const uint32_t to = tmem + (static_cast<uint32_t>(quarter * 32 + (warp >> 2) * 16) << 16);
        for (int p = 0; p < steps; ++p) {
            copy_wait<kWtAhead - 2>();
            __syncwarp();
            const uint32_t slot = p % kWtAhead;
            uint4 w4[kWtStep];
#pragma unroll
            for (int u = 0; u < kWtStep; ++u) w4[u] = lds128(codes + (slot * kWtStep + u) * 512 + lane * 16);
            const int s = p % kWtA;
            if (p >= kWtA && !tc_wait_warp(&sm.a_done[s], (p / kWtA - 1) & 1, fail, timeouts)) break;
            tc_fence_after();
#pragma unroll
            for (int u = 0; u < kWtStep; ++u) {
                const uint32_t w[4] = {w4[u].x, w4[u].y, w4[u].z, w4[u].w};
                uint32_t v[16];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t z0 = DT == 0 ? 0x64086408u : 0x43084308u, z1 = z0;
                    if constexpr (ZEROS) {
                        const uint32_t zz =
                            *reinterpret_cast<const uint16_t *>(&sm.zeros[warp][slot][u][(NG == 2 ? j >> 1 : 0) * 16 + g * 2]);
                        z0 = ((zz & 15u) * 0x00010001u) | (DT == 0 ? 0x64006400u : 0x43004300u);
                        z1 = ((zz >> 8) * 0x00010001u) | (DT == 0 ? 0x64006400u : 0x43004300u);
                    }
                    v[4 * j] = code_pair<DT>(w[j], z0);
                    v[4 * j + 1] = code_pair<DT>(w[j] >> 8, z0);
                    v[4 * j + 2] = code_pair<DT>(w[j] >> 4, z1);
                    v[4 * j + 3] = code_pair<DT>(w[j] >> 12, z1);
                }
                tc_st_fragments(to + s * (32 * kWtStep) + u * 32, v);  // (past the last chunk: unused)
            }
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(&sm.a_full[s]);
            __syncwarp();
            fetch(p + kWtAhead - 1);
        }
        copy_wait<0>();
    } else if (warp < 16) {
        // ---- sums: a thread per row, half of the tokens
        const int mine = warp - 8, from = (mine >> 2) * kMine;
#pragma unroll
        for (int n = 0; n < kMine; ++n) acc[n] = 0.0f;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kWtColD + from;
        // a row tile's scales of one group are 32 bytes, two pieces
        const uint8_t *const src = a.packed + a.l.scales_at;
        auto fetch = [&](int p) {
#pragma unroll
            for (int i = lane; i < kWtStep * 4 * NG; i += 32) {
                const int u = i / (4 * NG), at = i % (4 * NG), r = at / (2 * NG), n = at / 2 % NG;
                if (kWtStep * p + u < count) {
                    const long long tile = min(tile0 + 2 * quarter + r, a.l.row_tiles - 1);
                    copy16_async(smem_addr(sm.scales[mine][p % kWtAhead][u]) + at * 16,
                                 src + (tile * a.l.groups + group_of(kWtStep * p + u, n)) * 32 + (at & 1) * 16);
                }
            }
            copy_commit();
        };
        for (int p = 0; p < kWtAhead - 1; ++p) fetch(p);
        bool ok = true;
        for (int p = 0; p < steps && ok; ++p) {
            copy_wait<kWtAhead - 2>();
            __syncwarp();
#pragma unroll
            for (int un = 0; un < kWtStep * NG; un += 2) {
                // the unit of accumulators un and un + 1 of the step
                const int use = p * (kWtStep * NG / 2) + un / 2, d = use % kWtD;
                if (kWtStep * p + un / NG >= count || !ok) break;
                float scale[2];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    scale[k] = __half2float(*reinterpret_cast<const __half *>(
                        &sm.scales[mine][p % kWtAhead][(un + k) / NG][((lane >> 4) * NG + (un + k) % NG) * 32 + (lane & 7) * 4 +
                                                                       (lane >> 3 & 1) * 2]));
                const bool both = kWtStep * p + (un + 1) / NG < count;
                ok = tc_wait_warp(&sm.d_full[d], (use / kWtD) & 1, fail, timeouts);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t v[kMine / 16][16];
#pragma unroll
                    for (int h = 0; h < kMine / 16; ++h) tc_ld16(lanes + (2 * d + k) * N + h * 16, v[h]);
#pragma unroll
                    for (int h = 0; h < kMine / 16; ++h) tc_wait_ld(v[h]);
                    if (k == 1) {
                        tc_fence_before();
                        mbar_arrive(&sm.d_done[d]);
                        if (!both) break;  // (an accumulator that no product wrote)
                    }
#pragma unroll
                    for (int h = 0; h < kMine / 16; ++h)
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 y = fma2(make_float2(__uint_as_float(v[h][e]), __uint_as_float(v[h][e + 1])),
                                                  make_float2(scale[k], scale[k]),
                                                  make_float2(acc[h * 16 + e], acc[h * 16 + e + 1]));
                            acc[h * 16 + e] = y.x;
                            acc[h * 16 + e + 1] = y.y;
                        }
                }
            }
            __syncwarp();
            fetch(p + kWtAhead - 1);
        }
        copy_wait<0>();
    } else if (warp == 16) {
        // ---- products
        const bool leader = elect_lane();
        constexpr uint32_t kDesc = mma_desc(N, false, DT == 1);
        bool ok = true;
        for (int p = 0; p < steps && ok; ++p) {
            const int s = p % kWtA, xs = p % kWtX, chunks = min(kWtStep, count - kWtStep * p);
            ok = tc_wait_warp(&sm.a_full[s], (p / kWtA) & 1, fail, timeouts) &&
                 tc_wait_warp(&sm.x_full[xs], (p / kWtX) & 1, fail, timeouts);
            const uint32_t x = smem_addr(sm.x) + xs * kXStep, codes = tmem + s * (32 * kWtStep);
#pragma unroll
            for (int un = 0; un < kWtStep * NG; un += 2) {
                const int use = p * (kWtStep * NG / 2) + un / 2, d = use % kWtD;
                if (un / NG >= chunks) break;
                if (ok && use >= kWtD) ok = tc_wait_warp(&sm.d_done[d], (use / kWtD - 1) & 1, fail, timeouts);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int u = (un + k) / NG, n = (un + k) % NG;
                    if (u >= chunks) break;
#pragma unroll
                    for (int j = n * (4 / NG); j < (n + 1) * (4 / NG); ++j)
                        tc_mma_ts(leader, tmem + kWtColD + (2 * d + k) * N, codes + u * 32 + j * 8,
                                  smem_desc(x + u * (N * 128) + j * 32, 16, 1024), kDesc, j > n * (4 / NG));
                }
                tc_commit(leader, &sm.d_full[d]);
            }
            if (ok) {
                tc_commit(leader, &sm.a_done[s]);
                tc_commit(leader, &sm.x_done[xs]);
            }
        }
    } else {
        // ---- x: [token][64 columns]
        const int xt = tid - 544;
        const uint32_t x0 = smem_addr(sm.x);
        for (int i = xt; i < kWtX * kWtStep * (N - tokens) * 8; i += 128) {  // rows past the tokens stay zero
            const int buf = i / ((N - tokens) * 8), row = tokens + i / 8 % (N - tokens);
            reinterpret_cast<uint4 *>(sm.x + buf * (N * 128))[row * 8 + i % 8] = make_uint4(0, 0, 0, 0);
        }
        // this thread's pieces of a chunk: 16 bytes of rows m0, m0 + 16, ...
        constexpr int kEach = N / 16;
        const int m0 = xt >> 3, q = xt & 7;
        const uint16_t *const src = a.x + (token0 + m0) * a.x_stride + static_cast<long long>(first) * 64 + q * 8;
        for (int p = 0; p < steps + kWtXAhead; ++p) {
            if (p < steps) {
                if (p >= kWtX && !tc_wait_warp(&sm.x_done[p % kWtX], (p / kWtX - 1) & 1, fail, timeouts)) break;
#pragma unroll
                for (int u = 0; u < kWtStep; ++u) {
                    const int i = kWtStep * p + u;
                    const uint32_t buf = x0 + (p % kWtX) * kXStep + u * (N * 128);
                    const int have = i < count ? a.cols - (first + i) * 64 - q * 8 : 0;
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        const int m = m0 + 16 * e;
                        if (m >= tokens) break;
                        const uint16_t *const at = src + 16ll * e * a.x_stride + i * 64;
                        if (have >= 8) {
                            copy16_async(buf + swizzled(m, q), at);
                        } else {
                            const uint4 w = load8_any(at, have);
                            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(buf + swizzled(m, q)), "r"(w.x),
                                         "r"(w.y), "r"(w.z), "r"(w.w)
                                         : "memory");
                        }
                    }
                }
            }
            copy_commit();
            if (p >= kWtXAhead) {
                copy_wait<kWtXAhead>();
                smem_to_tensor_fence();
                mbar_arrive(&sm.x_full[(p - kWtXAhead) % kWtX]);
            }
        }
        copy_wait<0>();
    }

    // the slice's sums as [token][row], then every CTA of the cluster adds the
    // slices, in order, for its share of them
    constexpr int kPitch = kWtRows + 4;
    static_assert(N * kPitch * 4 <= kWtX * kWtStep * N * 128, "the sums fit where x was");
    float *const sums = reinterpret_cast<float *>(sm.x);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 16) tc_free(tmem, kWtColumns);
    if (warp >= 8 && warp < 16) {
        const int from = (warp - 8 >> 2) * kMine;
#pragma unroll
        for (int n = 0; n < kMine; ++n)
            if (from + n < tokens) sums[(from + n) * kPitch + quarter * 32 + lane] = acc[n];
    }
    if (splits > 1) cluster.sync(); else __syncthreads();
    const int row0 = tile0 * 16;
    const int mine0 = tokens * kWtRows * split / splits, mine1 = tokens * kWtRows * (split + 1) / splits;
    for (int i = mine0 + tid; i < mine1; i += kWtThreads) {
        const int m = i / kWtRows, row = i % kWtRows;
        float v = 0.0f;
        for (int c = 0; c < splits; ++c) v += cluster.map_shared_rank(sums, c)[m * kPitch + row];
        if (row0 + row < a.rows)
            a.y[(token0 + m) * a.y_stride + row0 + row] =
                DT ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
    }
    if (splits > 1) cluster.sync();  // no CTA leaves while another reads its sums
}

template <int DT, int N, int NG, bool ZEROS>
static cudaError_t run_w4_tc(const W4MatvecArgs &a, cudaStream_t s) {
    auto kern = w4_tc_kernel<DT, N, NG, ZEROS>;
    const int bytes = sizeof(WtSmem<N>) + 1024;
    cudaError_t err = allow_dynamic_smem(reinterpret_cast<const void *>(kern), bytes);
    if (err != cudaSuccess) return err;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    unsigned *timeouts = wait_timeout_counter(&err);
    if (!timeouts) return err;
    const long long row_ctas = (a.l.row_tiles + 7) / 8, token_ctas = (a.tokens + N - 1) / N;
    // The number of slices whose waves of CTAs, each its chunks and about twelve
    // more to start and end, are shortest; or whole waves of one number, and a
    // second launch, which costs about eight, for the rest of the rows in as many
    // slices as make that short (64 tokens through 20481 x 5123: two slices in
    // three waves 68.5 us, one wave whole and nine row tiles in eight slices 52.7;
    // 32 through 10240 x 8192: 39.2 and 31.1).
    struct Slices {
        int splits;
        long long cost;
    };
    auto slices_of = [&](long long rows) {
        Slices x = {1, -1};
        for (int n = 1; n <= 8; n *= 2) {
            const long long waves = (rows * token_ctas * n + sms - 1) / sms, cost = waves * ((a.l.chunks + n - 1) / n + 12);
            if (x.cost < 0 || cost < x.cost) x = {n, cost};
        }
        return x;
    };
    Slices first = slices_of(row_ctas), rest = {1, 0};
    long long first_rows = row_ctas;
    for (int n = 1; n <= 8; n *= 2) {
        const long long a_wave = sms / (n * token_ctas), waves = a_wave ? row_ctas / a_wave : 0, rows = waves * a_wave;
        if (rows == 0 || rows == row_ctas) continue;
        const Slices x = slices_of(row_ctas - rows);
        const long long cost = waves * ((a.l.chunks + n - 1) / n + 12);
        if (cost + x.cost + 8 < first.cost + rest.cost) first = {n, cost}, rest = {x.splits, x.cost + 8}, first_rows = rows;
    }
    auto launch = [&](const W4MatvecArgs &part, int splits, long long rows) {
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = splits;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(rows * splits), static_cast<unsigned>(token_ctas));
        cfg.blockDim = kWtThreads;
        cfg.dynamicSmemBytes = bytes;
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, part, (a.l.chunks + splits - 1) / splits, timeouts);
        return e != cudaSuccess ? e : cudaGetLastError();
    };
    W4MatvecArgs part = a;
    if (first_rows < row_ctas) part.rows = static_cast<int>(first_rows * kWtRows);
    err = launch(part, first.splits, first_rows);
    if (err != cudaSuccess || first_rows == row_ctas) return err;
    // the rest: everything that a row tile indexes begins first_rows later
    const long long tiles = first_rows * (kWtRows / 16), codes = tiles * a.l.chunks * 512;
    part.rows = static_cast<int>(a.rows - first_rows * kWtRows);
    part.y = a.y + first_rows * kWtRows;
    part.packed = a.packed + codes;
    part.l.row_tiles = static_cast<int>(a.l.row_tiles - tiles);
    part.l.scales_at = a.l.scales_at + tiles * a.l.groups * 32 - codes;
    part.l.zeros_at = a.l.zeros_at + tiles * a.l.groups * 16 - codes;
    return launch(part, rest.splits, row_ctas - first_rows);
}

template <int DT, int N>
static cudaError_t pick_group(const W4MatvecArgs &a, bool zeros, cudaStream_t s) {
    if (a.group_shift == 0) return zeros ? run_w4_tc<DT, N, 2, true>(a, s) : run_w4_tc<DT, N, 2, false>(a, s);
    return zeros ? run_w4_tc<DT, N, 1, true>(a, s) : run_w4_tc<DT, N, 1, false>(a, s);
}

// Rows of x on 16-byte boundaries, columns padded with zeros to whole chunks.
__global__ void __launch_bounds__(256) w4_align_kernel(W4MatvecArgs a, uint4 *to, int pieces) {
    chain_entry();
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < a.tokens * pieces; i += gridDim.x * 256ll) {
        const long long m = i / pieces;
        const int col = static_cast<int>(i - m * pieces) * 8;
        to[i] = load8_any(a.x + m * a.x_stride + col, a.cols - col);
    }
}

cudaError_t launch_w4_tc(int dtype, const W4MatvecArgs &given, bool zeros, void *workspace, cudaStream_t s) {
    W4MatvecArgs a = given;
    if (!w4_x_aligned(a.x, a.tokens, a.x_stride)) {
        // copied once rather than shifted into place by every CTA: the copy of 64
        // rows of 5123 is 0.7 MB, which each of 161 CTAs along the rows would read
        const int pieces = a.l.chunks * 8;
        const long long blocks = (a.tokens * pieces + 255) / 256;
        const cudaError_t err = launch_chained(w4_align_kernel, static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, s,
                                               given, static_cast<uint4 *>(workspace), pieces);
        if (err != cudaSuccess) return err;
        a.x = static_cast<const uint16_t *>(workspace);
        a.x_stride = a.l.chunks * 64;
        a.cols = a.l.chunks * 64;
    }
    // a grid's second dimension, the tokens' tiles, ends at 65535: more tokens
    // are more launches
    constexpr long long kMost = 65535ll * 64;
    for (long long done = 0; done < given.tokens; done += kMost) {
        W4MatvecArgs part = a;
        part.tokens = given.tokens - done < kMost ? given.tokens - done : kMost;
        part.x += done * a.x_stride;
        part.y += done * a.y_stride;
        // up to 32 tokens half the columns: 32 tokens through 8192 x 8192 22 us, as
        // half of a tile of 64 26 us
        const cudaError_t err = part.tokens <= 32 ? (dtype ? pick_group<1, 32>(part, zeros, s) : pick_group<0, 32>(part, zeros, s))
                                                  : (dtype ? pick_group<1, 64>(part, zeros, s) : pick_group<0, 64>(part, zeros, s));
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace qrk
