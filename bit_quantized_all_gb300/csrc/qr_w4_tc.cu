// qr_w4_tc.cu -- y = x W^T for 17 and more rows of x and 4-bit weights with
// group scales, on tcgen05 (qr_w4_matvec; qr_w4.cu describes the packed order).
//
// y^T = W x^T, a CTA taking 128 weight rows by up to 64 tokens over one slice of
// the columns, 64 columns (a chunk) at a time.  Four warps turn codes into the
// type's exact integers u - z and store them as the A operand in tensor memory:
// the packed words are the fragments of that store, so nothing is exchanged.
// Four warps bring x into shared memory.  One warp issues the products.  As scales differ from group
// to group, each group's (or chunk's, for groups of 128) products go to a ring
// of accumulators of their own, and four warps, a thread per row, add them
// scaled in fp32: the weights are never rounded.  The CTAs of a cluster add
// their slices' sums, in order, through distributed shared memory.
//
// What bounds it: HBM for the codes (4 KB a chunk: 178 cycles of an SM's
// share), closely followed by issue (conversion and scaling, about 190 slots a
// scheduler and chunk).
#include <cooperative_groups.h>

#include "qr_launch.h"
#include "qr_tcgen05.cuh"
#include "qr_w4.cuh"

namespace qrk {

namespace cg = cooperative_groups;

constexpr int kWtThreads = 416;  // warps 0-3 codes, 4-7 sums, 8 products, 9-12 x
constexpr int kWtRows = 128;
constexpr int kWtA = 4, kWtD = 4, kWtX = 8;  // buffers of codes, accumulators, x chunks
constexpr int kWtAhead = 16;                 // chunks of codes on their way
constexpr int kWtRaw = 6;                    // chunks of unaligned x on their way
constexpr uint32_t kWtColD = kWtA * 32, kWtColumns = 512;

template <int N>
struct WtSmem {
    uint8_t x[kWtX][N * 128];                       // then the sums
    uint8_t codes[4][kWtAhead][1024];               // by warp: its two row tiles
    uint8_t zeros[4][kWtAhead][64];
    uint8_t scales[4][kWtAhead][128];
    uint8_t raw[kWtRaw][N][160];                    // chunks of unaligned x as they lie in memory
    uint64_t a_full[kWtA], a_done[kWtA], x_full[kWtX], x_done[kWtX], d_full[kWtD], d_done[kWtD];
    uint32_t tmem;
    int fail;
};

// N: tokens of a CTA; NG: groups of a 64-column chunk (2 for groups of 32, else 1).
template <int DT, int N, int NG, bool ZEROS>
__global__ void __launch_bounds__(kWtThreads, 1) w4_tc_kernel(W4MatvecArgs a, int slice, bool vector, unsigned *timeouts) {
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

    if (tid == 0) {
        for (int i = 0; i < kWtA; ++i) {
            mbar_init(&sm.a_full[i], 128);
            mbar_init(&sm.a_done[i], 1);
        }
        for (int i = 0; i < kWtX; ++i) {
            mbar_init(&sm.x_full[i], 128);
            mbar_init(&sm.x_done[i], 1);
        }
        for (int i = 0; i < kWtD; ++i) {
            mbar_init(&sm.d_full[i], 1);
            mbar_init(&sm.d_done[i], 128);
        }
        mbar_init_fence();
        sm.fail = 0;
    }
    if (warp == 8) tc_alloc(&sm.tmem, kWtColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    float acc[N];  // of the sums' threads: this row's

    if (warp < 4) {
        // ---- codes: a warp's two row tiles of 16 x 64
        const uint32_t codes = smem_addr(sm.codes[warp]), zeros = smem_addr(sm.zeros[warp]);
        const uint8_t *src[2], *zsrc[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const long long tile = min(tile0 + 2 * warp + r, a.l.row_tiles - 1);
            src[r] = a.packed + (tile * a.l.chunks + first) * 512 + lane * 16;
            zsrc[r] = a.packed + a.l.zeros_at + tile * a.l.groups * 16;
        }
        auto group_of = [&](int i, int n) { return NG == 2 ? (first + i) * 2 + n : (first + i) >> (a.group_shift - 1); };
        auto fetch = [&](int i) {
            if (i < count) {
                const uint32_t slot = i % kWtAhead;
#pragma unroll
                for (int r = 0; r < 2; ++r) copy16_async(codes + slot * 1024 + r * 512 + lane * 16, src[r] + i * 512ll);
                if (ZEROS && lane < 2 * NG)
                    copy16_async(zeros + slot * 64 + lane * 16, zsrc[lane / NG] + group_of(i, lane % NG) * 16);
            }
            copy_commit();
        };
        for (int i = 0; i < kWtAhead - 1; ++i) fetch(i);
        for (int i = 0; i < count; ++i) {
            copy_wait<kWtAhead - 2>();
            __syncwarp();
            const uint32_t slot = i % kWtAhead;
            uint32_t v[2][16];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint4 w4 = lds128(codes + slot * 1024 + r * 512 + lane * 16);
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t z0 = DT == 0 ? 0x64086408u : 0x43084308u, z1 = z0;
                    if constexpr (ZEROS) {
                        const uint32_t zz = *reinterpret_cast<const uint16_t *>(
                            &sm.zeros[warp][slot][(r * NG + (NG == 2 ? j >> 1 : 0)) * 16 + g * 2]);
                        z0 = ((zz & 15u) * 0x00010001u) | (DT == 0 ? 0x64006400u : 0x43004300u);
                        z1 = ((zz >> 8) * 0x00010001u) | (DT == 0 ? 0x64006400u : 0x43004300u);
                    }
                    v[r][4 * j] = code_pair<DT>(w[j], z0);
                    v[r][4 * j + 1] = code_pair<DT>(w[j] >> 8, z0);
                    v[r][4 * j + 2] = code_pair<DT>(w[j] >> 4, z1);
                    v[r][4 * j + 3] = code_pair<DT>(w[j] >> 12, z1);
                }
            }
            __syncwarp();
            fetch(i + kWtAhead - 1);
            const int s = i % kWtA;
            if (i >= kWtA && !tc_wait_warp(&sm.a_done[s], (i / kWtA - 1) & 1, fail, timeouts)) break;
            tc_fence_after();
#pragma unroll
            for (int r = 0; r < 2; ++r) tc_st_fragments(tmem + (static_cast<uint32_t>(warp * 32 + r * 16) << 16) + s * 32, v[r]);
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(&sm.a_full[s]);
        }
        copy_wait<0>();
    } else if (warp < 8) {
        // ---- sums: a thread per row
        const int q = warp - 4;
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] = 0.0f;
        const uint32_t scales = smem_addr(sm.scales[q]), lanes = tmem + (static_cast<uint32_t>(q * 32) << 16) + kWtColD;
        // a row tile's scales of one group are 32 bytes, two pieces
        const uint8_t *const src = a.packed + a.l.scales_at;
        auto fetch = [&](int i) {
            if (i < count && lane < 4 * NG) {
                const int r = lane / (2 * NG), n = lane / 2 % NG;
                const long long tile = min(tile0 + 2 * q + r, a.l.row_tiles - 1);
                const int gi = NG == 2 ? (first + i) * 2 + n : (first + i) >> (a.group_shift - 1);
                copy16_async(scales + (i % kWtAhead) * 128 + lane * 16, src + (tile * a.l.groups + gi) * 32 + (lane & 1) * 16);
            }
            copy_commit();
        };
        for (int i = 0; i < kWtAhead - 1; ++i) fetch(i);
        bool ok = true;
        for (int i = 0; i < count && ok; ++i) {
            copy_wait<kWtAhead - 2>();
            __syncwarp();
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const int use = i * NG + n, d = use % kWtD;
                const float scale = __half2float(*reinterpret_cast<const __half *>(
                    &sm.scales[q][i % kWtAhead][((lane >> 4) * NG + n) * 32 + (lane & 7) * 4 + (lane >> 3 & 1) * 2]));
                if (!tc_wait_warp(&sm.d_full[d], (use / kWtD) & 1, fail, timeouts)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < N / 32; ++h) {
                    uint32_t v[32];
                    tc_ld32(lanes + d * N + h * 32, v);
                    tc_wait_ld(v);
                    if (h == N / 32 - 1) {
                        tc_fence_before();
                        mbar_arrive(&sm.d_done[d]);
                    }
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float2 y = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])),
                                              make_float2(scale, scale), make_float2(acc[h * 32 + k], acc[h * 32 + k + 1]));
                        acc[h * 32 + k] = y.x;
                        acc[h * 32 + k + 1] = y.y;
                    }
                }
            }
            __syncwarp();
            fetch(i + kWtAhead - 1);
        }
        copy_wait<0>();
    } else if (warp == 8) {
        // ---- products
        const bool leader = elect_lane();
        constexpr uint32_t kDesc = mma_desc(N, false, DT == 1);
        bool ok = true;
        for (int i = 0; i < count && ok; ++i) {
            const int s = i % kWtA, xs = i % kWtX;
            ok = tc_wait_warp(&sm.a_full[s], (i / kWtA) & 1, fail, timeouts) &&
                 tc_wait_warp(&sm.x_full[xs], (i / kWtX) & 1, fail, timeouts);
            const uint32_t x = smem_addr(sm.x[xs]);
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const int use = i * NG + n, d = use % kWtD;
                if (ok && use >= kWtD) ok = tc_wait_warp(&sm.d_done[d], (use / kWtD - 1) & 1, fail, timeouts);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int j = n * (4 / NG); j < (n + 1) * (4 / NG); ++j)
                    tc_mma_ts(leader, tmem + kWtColD + d * N, tmem + s * 32 + j * 8, smem_desc(x + j * 32, 16, 1024), kDesc,
                              j > n * (4 / NG));
                tc_commit(leader, &sm.d_full[d]);
            }
            if (ok) {
                tc_commit(leader, &sm.a_done[s]);
                tc_commit(leader, &sm.x_done[xs]);
            }
        }
    } else {
        // ---- x: [token][64 columns]
        const int xt = tid - 288;
        for (int i = xt; i < kWtX * (N - tokens) * 8; i += 128) {  // rows past the tokens stay zero
            const int buf = i / ((N - tokens) * 8), row = tokens + i / 8 % (N - tokens);
            reinterpret_cast<uint4 *>(sm.x[buf])[row * 8 + i % 8] = make_uint4(0, 0, 0, 0);
        }
        // this thread's pieces of a chunk: 16 bytes of rows m0, m0 + 16, ...
        constexpr int kEach = N / 16;
        const int m0 = xt >> 3, q = xt & 7;
        const uint16_t *const src = a.x + (token0 + m0) * a.x_stride + static_cast<long long>(first) * 64 + q * 8;
        auto tc_wait_if = [&](bool wanted, uint64_t *bar, uint32_t parity, int *f, unsigned *t) {
            if (wanted) tc_wait_warp(bar, parity, f, t);
        };
        auto ready = [&](int i) {
            return i < kWtX || tc_wait_warp(&sm.x_done[i % kWtX], (i / kWtX - 1) & 1, fail, timeouts);
        };
        auto announce = [&](int i) {
            smem_to_tensor_fence();
            mbar_arrive(&sm.x_full[i % kWtX]);
        };
        if (vector) {
            constexpr int kLag = kWtX - 2;  // chunks on their way
            for (int i = 0; i < count + kLag; ++i) {
                if (i < count) {
                    if (!ready(i)) break;
                    const uint32_t buf = smem_addr(sm.x[i % kWtX]);
                    const int have = a.cols - (first + i) * 64 - q * 8;
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        const int m = m0 + 16 * e;
                        if (m >= tokens) break;
                        const uint16_t *const at = src + 16ll * e * a.x_stride + i * 64;
                        if (have >= 8) {
                            copy16_async(buf + swizzled(m, q), at);
                        } else {
                            const uint4 w = load8_any(at, have);
                            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(buf + swizzled(m, q)), "r"(w.x), "r"(w.y),
                                         "r"(w.z), "r"(w.w)
                                         : "memory");
                        }
                    }
                }
                copy_commit();
                if (i >= kLag) {
                    copy_wait<kLag>();
                    announce(i - kLag);
                }
            }
            copy_wait<0>();
        } else {
            // rows that are not 16-byte aligned: the aligned pieces that hold a
            // chunk of one (nine at most, of 16 bytes) are copied as they are,
            // then shifted into place
            auto fetch = [&](int i) {
                if (i < count) {
                    const uint32_t buf = smem_addr(sm.raw[i % kWtRaw]);
                    const int bytes = 2 * min(64, a.cols - (first + i) * 64);
                    for (int p = xt; p < tokens * 9; p += 128) {
                        const int m = p / 9, k = p - m * 9;
                        const uintptr_t row = reinterpret_cast<uintptr_t>(a.x + (token0 + m) * a.x_stride + (first + i) * 64ll);
                        const int off = static_cast<int>(row & 15);
                        if (k * 16 < off + bytes) copy16_async(buf + m * 160 + k * 16, reinterpret_cast<const void *>(row - off + k * 16));
                    }
                }
                copy_commit();
            };
            for (int i = 0; i < kWtRaw - 1; ++i) fetch(i);
            for (int i = 0; i < count; ++i) {
                copy_wait<kWtRaw - 2>();
                asm volatile("bar.sync 1, 128;" ::: "memory");  // the four warps' pieces; the buffer filled next is left
                fetch(i + kWtRaw - 1);
                // (after a wait that ran out the four warps go on together)
                tc_wait_if(i >= kWtX, &sm.x_done[i % kWtX], (i / kWtX - 1) & 1, fail, timeouts);
                const uint32_t buf = smem_addr(sm.x[i % kWtX]), raw_buf = smem_addr(sm.raw[i % kWtRaw]);
                const int have = a.cols - (first + i) * 64 - q * 8;
#pragma unroll 2
                for (int e = 0; e < kEach; ++e) {
                    const int m = m0 + 16 * e;
                    if (m >= tokens) break;
                    const uint32_t off = reinterpret_cast<uintptr_t>(src + 16ll * e * a.x_stride) & 15;
                    const uint4 lo = lds128(raw_buf + m * 160 + q * 16), hi = lds128(raw_buf + m * 160 + q * 16 + 16);
                    const uint4 w = take8(lo, hi, off, have);
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(buf + swizzled(m, q)), "r"(w.x), "r"(w.y), "r"(w.z),
                                 "r"(w.w)
                                 : "memory");
                }
                announce(i);
            }
            copy_wait<0>();
        }
    }

    // the slice's sums as [token][row], then every CTA of the cluster adds the
    // slices, in order, for its share of them
    constexpr int kPitch = kWtRows + 4;
    static_assert(N * kPitch * 4 <= kWtX * N * 128, "the sums fit where x was");
    float *const sums = reinterpret_cast<float *>(sm.x[0]);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tc_free(tmem, kWtColumns);
    if (warp >= 4 && warp < 8) {
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (n < tokens) sums[n * kPitch + tid - 128] = acc[n];
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
    // the number of slices whose waves of CTAs, each its chunks and about twelve
    // more to start and end, are shortest
    int splits = 1;
    long long best = -1;
    for (int n = 1; n <= 8; n *= 2) {
        const long long waves = (row_ctas * token_ctas * n + sms - 1) / sms, cost = waves * ((a.l.chunks + n - 1) / n + 12);
        if (best < 0 || cost < best) best = cost, splits = n;
    }
    const int slice = (a.l.chunks + splits - 1) / splits;
    const bool vector = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && (a.tokens == 1 || a.x_stride % 8 == 0);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(row_ctas * splits), static_cast<unsigned>(token_ctas));
    cfg.blockDim = kWtThreads;
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, kern, a, slice, vector, timeouts);
    return err != cudaSuccess ? err : cudaGetLastError();
}

template <int DT, int N>
static cudaError_t pick_group(const W4MatvecArgs &a, bool zeros, cudaStream_t s) {
    if (a.group_shift == 0) return zeros ? run_w4_tc<DT, N, 2, true>(a, s) : run_w4_tc<DT, N, 2, false>(a, s);
    return zeros ? run_w4_tc<DT, N, 1, true>(a, s) : run_w4_tc<DT, N, 1, false>(a, s);
}

cudaError_t launch_w4_tc(int dtype, const W4MatvecArgs &a, bool zeros, cudaStream_t s) {
    if (a.tokens <= 32) return dtype ? pick_group<1, 32>(a, zeros, s) : pick_group<0, 32>(a, zeros, s);
    return dtype ? pick_group<1, 64>(a, zeros, s) : pick_group<0, 64>(a, zeros, s);
}

}  // namespace qrk
