// qr_w8_tc.cu -- y = x W^T for 17 and more rows of x and weights in 8 bits, on
// tcgen05 (qr_w8_matmul; qr_w8.cu describes the packed order).
//
// The fast integer products of this GPU are those of 16-bit floats: codes are
// exact fp16 numbers, their products exact in fp32.  A first kernel writes x's
// codes as fp16 into the workspace, in the order and with the swizzle that the
// products read from shared memory, so that a chunk of 64 columns of a CTA's
// tokens is one bulk copy.  Then y^T = W x^T in tiles of 128 weight rows by N
// tokens: eight warps, a row tile of 16 each, turn packed codes into fp16 and store
// them as the A operand in tensor memory, one warp brings x, one issues the
// products, and four scale and store a finished tile while the next one runs.
//
// The chunks of all tiles, one tile after the other, are divided evenly among
// the CTAs, one an SM.  A tile that one CTA has whole is stored by it; the parts
// of the others go to the workspace as fp32 sums, and a last kernel adds them in
// order, so that the result has the same bits every time.
//
// A lane's 16 codes of a tile's row are consecutive columns; as fragments of the
// store to tensor memory they stand at the columns 16 j + 4 t + 0..3, so x is
// written into the workspace with its columns exchanged alike.
#include "qr_launch.h"
#include "qr_tcgen05.cuh"
#include "qr_w8.cuh"

namespace qrk {

constexpr int kWeThreads = 256;

// x's codes as fp16: a block of N tokens x 64 columns is N * 128 bytes, swizzled.
// A thread takes 32 codes, half of a token's part of a chunk: pieces j, j + 2, ...
__global__ void __launch_bounds__(kWeThreads) w8_expand_kernel(W8Args a, uint8_t *to, int n_shift) {
    // the product may start once everything before this kernel is complete: until
    // its own wait it reads the weights only
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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

// warps 0-7 codes, 8 products, 9 x, 10-13 results, and up to 128 tokens 14 the
// packed codes' way in
template <int N>
constexpr int kWtThreads = N >= 256 ? 448 : 480;
constexpr int kWtRows = 128;
constexpr int kWtStep = 4, kWtA = 2;  // chunks of a step, and buffers of codes in tensor memory, a step each
constexpr uint32_t kWtColD = kWtA * 32 * kWtStep, kWtColumns = 512;
constexpr int kWtMostCtas = 152;  // the workspace has two parts for each

template <int N>
struct WtSmem {
    static constexpr int kBlock = N * 128;
    // Up to 128 tokens the weights' bytes bound the kernel, and their way in is deep,
    // through shared memory; with 256 tokens x fills that, and the products leave
    // time for two steps in registers (64 tokens through 10240 x 8192: XX).
    static constexpr bool kStaged = N < 256;
    static constexpr int kW = kStaged ? (N >= 128 ? 2 : N >= 64 ? 3 : 4) : 1;  // steps of packed codes
    // x: chunks that are handed on together (a wait and a commit take the products'
    // warp some 150 cycles, four chunks' products of 64 tokens run for 512), and
    // buffers of them
    static constexpr int kXc = N >= 256 ? 1 : N >= 128 ? 2 : 4;
    static constexpr int kX = N >= 256 ? 6 : N >= 128 ? 4 : N >= 64 ? 3 : 4;
    static constexpr int kD = N >= 256 ? 1 : 2;  // accumulators
    uint8_t x[kX * kXc * kBlock];
    uint8_t codes[kStaged ? kW : 1][8][kStaged ? kWtStep * 1024 : 16];  // by warp: its row tile
    uint8_t out[4][32 * 80];  // by warp: 32 tokens of 32 rows
    float x_scale[4][N];      // by warp
    uint64_t a_full[kWtA], a_done[kWtA], x_full[kX], x_done[kX], d_full[kD], d_done[kD], w_full[kW], w_done[kW];
    uint32_t tmem;
    int fail;
};

// The division of the chunks: all = tiles * chunks of them over `ctas`.
struct W8Shares {
    long long all;
    int chunks, row_ctas, ctas;

    __host__ __device__ __forceinline__ long long begin(long long cta) const { return all * cta / ctas; }
    // the CTA that has chunk `u`
    __device__ __forceinline__ int owner(long long u) const { return static_cast<int>(((u + 1) * ctas - 1) / all); }
};

// Walks a CTA's chunks, a step of up to kWtStep chunks of one tile at a time.
struct W8Walk {
    long long left;
    int chunk, chunks, row_tile, row_ctas;
    long long token_tile;

    __device__ __forceinline__ W8Walk(const W8Shares &s, int cta) {
        const long long u = s.begin(cta), tile = u / s.chunks;
        left = s.begin(cta + 1) - u;
        chunk = static_cast<int>(u - tile * s.chunks);
        chunks = s.chunks;
        row_ctas = s.row_ctas;
        token_tile = tile / row_ctas;
        row_tile = static_cast<int>(tile - token_tile * row_ctas);
    }
    __device__ __forceinline__ int step() const {
        return static_cast<int>(min(static_cast<long long>(min(kWtStep, chunks - chunk)), left));
    }
    // Chunks of this tile that are the CTA's, from here on.
    __device__ __forceinline__ int segment() const {
        return static_cast<int>(min(static_cast<long long>(chunks - chunk), left));
    }
    __device__ __forceinline__ void advance(int n) {
        left -= n;
        chunk += n;
        if (chunk == chunks) {
            chunk = 0;
            if (++row_tile == row_ctas) row_tile = 0, ++token_tile;
        }
    }
};

template <int DT, int N>
__global__ void __launch_bounds__(kWtThreads<N>, 1)
    w8_tc_kernel(W8Args a, W8Shares shares, const uint8_t *x16, float *parts, unsigned *timeouts) {
    using S = WtSmem<N>;
    extern __shared__ uint8_t raw[];
    S &sm = *reinterpret_cast<S *>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *const fail = &sm.fail;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        for (int i = 0; i < kWtA; ++i) {
            mbar_init(&sm.a_full[i], 8);
            mbar_init(&sm.a_done[i], 1);
        }
        for (int i = 0; i < S::kX; ++i) {
            mbar_init(&sm.x_full[i], 1);
            mbar_init(&sm.x_done[i], 1);
        }
        for (int i = 0; i < S::kD; ++i) {
            mbar_init(&sm.d_full[i], 1);
            mbar_init(&sm.d_done[i], 4);
        }
        for (int i = 0; i < S::kW; ++i) {
            mbar_init(&sm.w_full[i], 1);
            mbar_init(&sm.w_done[i], 8);
        }
        mbar_init_fence();
        sm.fail = 0;
    }
    if (warp == 8) tc_alloc(&sm.tmem, kWtColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const int quarter = warp & 3;  // of tensor memory's lanes, that this warp reaches
    W8Walk at(shares, blockIdx.x);

    if (warp < 8) {
        // ---- codes: a row tile of 16
        const uint32_t to = tmem + (static_cast<uint32_t>(quarter * 32 + (warp >> 2) * 16) << 16);
        // a chunk's packed codes to its place as the A operand
        auto convert = [&](const uint4 &u, const uint4 &l, int b, int k) {
            const uint32_t up[4] = {u.x, u.y, u.z, u.w}, low[4] = {l.x, l.y, l.z, l.w};
            uint32_t v[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                weights_f16(up[j], v[4 * j], v[4 * j + 1]);
                weights_f16(low[j], v[4 * j + 2], v[4 * j + 3]);
            }
            tc_st_fragments(to + b * (32 * kWtStep) + k * 32, v);  // (past the step's last chunk: unused)
        };
        auto hand_on = [&](int b) {
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.a_full[b]);
        };
        bool ok = true;
        if constexpr (S::kStaged) {
            for (unsigned p = 0; at.left > 0; ++p) {
                const unsigned b = p % kWtA, ws = p % S::kW;
                ok = tc_wait_warp(&sm.w_full[ws], (p / S::kW) & 1, fail, timeouts);
                const uint32_t from = smem_addr(sm.codes[ws][2 * quarter + (warp >> 2)]) + lane * 16;
                uint4 w[kWtStep][2];
#pragma unroll
                for (int u = 0; u < kWtStep; ++u) w[u][0] = lds128(from + u * 1024), w[u][1] = lds128(from + u * 1024 + 512);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.w_done[ws]);
                if (ok && p >= kWtA) ok = tc_wait_warp(&sm.a_done[b], (p / kWtA - 1) & 1, fail, timeouts);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int u = 0; u < kWtStep; ++u) convert(w[u][0], w[u][1], b, u);
                hand_on(b);
                at.advance(at.step());
            }
        } else {
            // two steps on their way in registers
            W8Walk ahead = at;
            const int mine = 2 * quarter + (warp >> 2);
            uint4 w[2][kWtStep][2];
            auto fetch = [&](int b) {
                if (ahead.left <= 0) return;
                const int n = ahead.step();
                const long long tile = min(ahead.row_tile * (kWtRows / 16) + mine, a.l.row_tiles - 1);
                const uint4 *const src = reinterpret_cast<const uint4 *>(a.packed) + (tile * a.l.chunks + ahead.chunk) * 64 + lane;
#pragma unroll
                for (int u = 0; u < kWtStep; ++u)
                    if (u < n) {
                        w[b][u][0] = __ldg(src + u * 64);
                        w[b][u][1] = __ldg(src + u * 64 + 32);
                    }
                ahead.advance(n);
            };
            fetch(0);
            fetch(1);
            for (int round = 0; at.left > 0 && ok; ++round) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (at.left <= 0) break;
                    if (round > 0) ok = tc_wait_warp(&sm.a_done[b], (round - 1) & 1, fail, timeouts);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int u = 0; u < kWtStep; ++u) convert(w[b][u][0], w[b][u][1], b, u);
                    hand_on(b);
                    at.advance(at.step());
                    fetch(b);
                }
            }
        }
    } else if (warp == 8) {
        // ---- products
        const bool leader = elect_lane();
        constexpr uint32_t kDesc = mma_desc(N, false);
        bool ok = true;
        unsigned p = 0, i = 0;
        for (unsigned g = 0; at.left > 0 && ok; ++g) {
            const unsigned d = g % S::kD;
            int n = at.segment();
            if (g >= S::kD) ok = tc_wait_warp(&sm.d_done[d], (g / S::kD - 1) & 1, fail, timeouts);
            bool add = false;
            while (n > 0 && ok) {
                const int s = p % kWtA, chunks = at.step();
                ok = tc_wait_warp(&sm.a_full[s], (p / kWtA) & 1, fail, timeouts);
                for (int u0 = 0; u0 < chunks && ok; u0 += S::kXc, ++i) {
                    const int xs = i % S::kX;
                    ok = tc_wait_warp(&sm.x_full[xs], (i / S::kX) & 1, fail, timeouts);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t x = smem_addr(sm.x) + xs * (S::kXc * S::kBlock), codes = tmem + s * (32 * kWtStep) + u0 * 32;
#pragma unroll
                    for (int k = 0; k < S::kXc; ++k) {
                        if (u0 + k >= chunks) break;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            tc_mma_ts(leader, tmem + kWtColD + d * N, codes + k * 32 + j * 8,
                                      smem_desc(x + k * S::kBlock + j * 32, 16, 1024), kDesc, add || k + j > 0);
                    }
                    add = true;
                    tc_commit(leader, &sm.x_done[xs]);
                }
                if (!ok) break;
                tc_commit(leader, &sm.a_done[s]);
                ++p;
                n -= chunks;
                at.advance(chunks);
            }
            tc_commit(leader, &sm.d_full[d]);
            // (after a wait that ran out: nothing is under way when tensor memory is freed)
            if (!ok) mbar_wait(&sm.d_full[d], (g / S::kD) & 1);
        }
    } else if (warp == 9) {
        // ---- x: the blocks of consecutive chunks are one copy
        if (lane == 0) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            unsigned i = 0;
            for (bool ok = true; at.left > 0 && ok;) {
                const int chunks = at.step();
                for (int u0 = 0; u0 < chunks; u0 += S::kXc, ++i) {
                    const int xs = i % S::kX;
                    if (i >= S::kX) ok = tc_wait(&sm.x_done[xs], (i / S::kX - 1) & 1, fail, timeouts);
                    if (!ok) break;
                    const uint32_t bytes = min(S::kXc, chunks - u0) * S::kBlock;
                    mbar_arrive_expect_tx(&sm.x_full[xs], bytes);
                    bulk_copy_g2s(sm.x + xs * (S::kXc * S::kBlock), x16 + (at.token_tile * at.chunks + at.chunk + u0) * S::kBlock,
                                  bytes, &sm.x_full[xs]);
                }
                at.advance(chunks);
            }
            // none of the copies is on its way when the CTA leaves
            for (unsigned k = i < S::kX ? 0 : i - S::kX; k < i; ++k) mbar_wait(&sm.x_full[k % S::kX], (k / S::kX) & 1);
        }
        __syncwarp();
    } else if (warp == 14) {
        // ---- the packed codes' way in: a step of a row tile is one copy
        if constexpr (S::kStaged) {
            if (lane == 0) {
                unsigned p = 0;
                for (; at.left > 0; ++p) {
                    const unsigned ws = p % S::kW;
                    if (p >= S::kW && !tc_wait(&sm.w_done[ws], (p / S::kW - 1) & 1, fail, timeouts)) break;
                    const int n = at.step();
                    mbar_arrive_expect_tx(&sm.w_full[ws], 8 * n * 1024);
                    for (int k = 0; k < 8; ++k) {
                        const long long tile = min(at.row_tile * (kWtRows / 16) + k, a.l.row_tiles - 1);
                        bulk_copy_g2s(sm.codes[ws][k], a.packed + (tile * a.l.chunks + at.chunk) * 1024, n * 1024, &sm.w_full[ws]);
                    }
                    at.advance(n);
                }
                for (unsigned k = p < S::kW ? 0 : p - S::kW; k < p; ++k) mbar_wait(&sm.w_full[k % S::kW], (k / S::kW) & 1);
            }
            __syncwarp();
        }
    } else {
        // ---- results: a thread per row
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int mine = warp - 10;
        uint8_t *const stage = sm.out[mine];
        float *const x_scale = sm.x_scale[mine];
        const bool vector = (reinterpret_cast<uintptr_t>(a.y) & 15) == 0 && a.y_stride % 8 == 0;
        long long held = -1;  // the tokens whose scales are in shared memory
        bool ok = true;
        for (unsigned g = 0; at.left > 0; ++g) {
            const unsigned d = g % S::kD;
            const int n = at.segment();
            const bool whole = n == at.chunks;
            const long long token0 = at.token_tile * N, row0 = static_cast<long long>(at.row_tile) * kWtRows + quarter * 32;
            const int tokens = static_cast<int>(min(static_cast<long long>(N), a.tokens - token0));
            if (whole && held != at.token_tile) {
                held = at.token_tile;
                __syncwarp();
                for (int m = lane; m < N; m += 32) x_scale[m] = m < tokens ? a.x_scales[token0 + m] : 0.0f;
                __syncwarp();
            }
            const float scale = row0 + lane < a.rows ? reinterpret_cast<const float *>(a.packed + a.l.scales_at)[row0 + lane] : 0.0f;
            float *const part = parts + (2ll * blockIdx.x + (at.chunk == 0)) * (kWtRows * N) + quarter * 32 + lane;
            ok = tc_wait_warp(&sm.d_full[d], (g / S::kD) & 1, fail, timeouts);
            if (!ok) break;
            tc_fence_after();
            const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kWtColD + d * N;
#pragma unroll 1
            for (int h = 0; h < N / 32; ++h) {
                uint32_t v[32];
                tc_ld32(lanes + h * 32, v);
                tc_wait_ld(v);
                if (h == N / 32 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.d_done[d]);
                }
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) part[(h * 32 + e) * kWtRows] = __uint_as_float(v[e]);
                    continue;
                }
                if (h * 32 >= tokens) continue;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    *reinterpret_cast<uint16_t *>(stage + e * 80 + lane * 2) =
                        narrow1<DT>(__uint_as_float(v[e]) * x_scale[h * 32 + e] * scale);
                __syncwarp();
                if (vector && row0 + 32 <= a.rows) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int m = e * 8 + (lane >> 2);
                        const uint4 o = *reinterpret_cast<const uint4 *>(stage + m * 80 + (lane & 3) * 16);
                        if (h * 32 + m < tokens)
                            *reinterpret_cast<uint4 *>(a.y + (token0 + h * 32 + m) * a.y_stride + row0 + (lane & 3) * 8) = o;
                    }
                } else if (row0 + lane < a.rows) {
                    for (int m = 0; m < 32 && h * 32 + m < tokens; ++m)
                        a.y[(token0 + h * 32 + m) * a.y_stride + row0 + lane] =
                            *reinterpret_cast<const uint16_t *>(stage + m * 80 + lane * 2);
                }
                __syncwarp();
            }
            at.advance(n);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tc_free(tmem, kWtColumns);
    // (a kernel is complete for the next one only when all of its threads have
    // waited for the one before, or left)
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Adds the parts of the tiles that several CTAs share: block x is the tile in
// which CTA x's share ends, y a group of 32 tokens of it.  What is not a part (the
// scales) was there before the product began, and is read before its end.
template <int DT>
__global__ void __launch_bounds__(256) w8_join_kernel(W8Args a, W8Shares shares, const float *parts, int n) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long end = shares.begin(blockIdx.x + 1), tile = (end - 1) / shares.chunks;
    const long long from = tile * shares.chunks, to = from + shares.chunks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long token0 = tile / shares.row_ctas * n + blockIdx.y * 32 + warp;  // and every eighth from there
    const long long row = tile % shares.row_ctas * kWtRows + lane * 4;
    // nothing where the tile is whole, or another block's to add
    const bool mine = end != to && shares.owner(from) == static_cast<int>(blockIdx.x) && token0 < a.tokens && row < a.rows;
    const int last = shares.owner(to - 1);
    float4 scale = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float x_scale[4];
    if (mine) scale = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(a.packed + a.l.scales_at) + row);
#pragma unroll
    for (int k = 0; k < 4; ++k) x_scale[k] = mine && token0 + 8 * k < a.tokens ? a.x_scales[token0 + 8 * k] : 0.0f;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!mine) return;
    const float4 *const p = reinterpret_cast<const float4 *>(parts) + (blockIdx.y * 32 + warp) * (kWtRows / 4) + lane;
    const long long pitch = static_cast<long long>(kWtRows / 4) * n;  // of a part; CTA c's are 2 c and 2 c + 1
    float4 sum[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] = __ldcg(p + (2ll * blockIdx.x + 1) * pitch + k * 8 * (kWtRows / 4));
#pragma unroll 4
    for (int c = blockIdx.x + 1; c <= last; ++c) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 v = __ldcg(p + 2ll * c * pitch + k * 8 * (kWtRows / 4));
            sum[k].x += v.x, sum[k].y += v.y, sum[k].z += v.z, sum[k].w += v.w;
        }
    }
    const bool vector = (reinterpret_cast<uintptr_t>(a.y) & 7) == 0 && a.y_stride % 4 == 0 && row + 4 <= a.rows;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const long long token = token0 + 8 * k;
        if (token >= a.tokens) break;
        const float s = x_scale[k];
        const float y[4] = {sum[k].x * s * scale.x, sum[k].y * s * scale.y, sum[k].z * s * scale.z, sum[k].w * s * scale.w};
        uint16_t *const to_y = a.y + token * a.y_stride + row;
        if (vector)
            *reinterpret_cast<uint2 *>(to_y) = make_uint2(narrow2<DT>(y[0], y[1]), narrow2<DT>(y[2], y[3]));
        else
            for (int e = 0; e < 4 && row + e < a.rows; ++e) to_y[e] = narrow1<DT>(y[e]);
    }
}

// Tokens of a tile: the fewest that take them all, 256 at most.
static int w8_token_shift(long long tokens) { return tokens <= 32 ? 5 : tokens <= 64 ? 6 : tokens <= 128 ? 7 : 8; }

static size_t w8_x16_bytes(long long tokens, int chunks, int shift) {
    return static_cast<size_t>((tokens + (1 << shift) - 1) >> shift << shift) * chunks * 128;
}

size_t w8_workspace(long long tokens, int cols) {
    const int shift = w8_token_shift(tokens);
    return w8_x16_bytes(tokens, cols / 64 + (cols % 64 != 0), shift) + (size_t(2) * kWtMostCtas * kWtRows * 4 << shift);
}

template <int DT, int N>
static cudaError_t run_w8_tc(const W8Args &a, uint8_t *workspace, int shift, cudaStream_t s) {
    auto kern = w8_tc_kernel<DT, N>;
    const int bytes = sizeof(WtSmem<N>) + 1024;
    cudaError_t err = allow_dynamic_smem(reinterpret_cast<const void *>(kern), bytes);
    if (err != cudaSuccess) return err;
    int sms = sm_count(&err);
    if (sms <= 0) return err;
    if (sms > kWtMostCtas) sms = kWtMostCtas;
    unsigned *timeouts = wait_timeout_counter(&err);
    if (!timeouts) return err;
    const long long tiles = (a.l.row_tiles + 7) / 8 * ((a.tokens + N - 1) / N);
    W8Shares shares = {tiles * a.l.chunks, a.l.chunks, (a.l.row_tiles + 7) / 8, sms};
    // at least eight chunks a CTA, or a tile where that is less
    const long long few = a.l.chunks < 8 ? tiles : shares.all / 8;
    if (few < sms) shares.ctas = static_cast<int>(few > 1 ? few : 1);
    float *const parts = reinterpret_cast<float *>(workspace + w8_x16_bytes(a.tokens, a.l.chunks, shift));
    err = launch_chained(kern, shares.ctas, kWtThreads<N>, bytes, s, a, shares, static_cast<const uint8_t *>(workspace), parts,
                         timeouts);
    if (err != cudaSuccess) return err;
    bool joined = false;
    for (int c = 1; c < shares.ctas && !joined; ++c) joined = shares.begin(c) % a.l.chunks != 0;
    if (!joined) return cudaSuccess;
    return launch_chained(w8_join_kernel<DT>, dim3(shares.ctas - 1, N / 32), 256, 0, s, a, shares, static_cast<const float *>(parts), N);
}

template <int DT>
static cudaError_t pick_tokens(int shift, const W8Args &a, uint8_t *workspace, cudaStream_t s) {
    switch (shift) {
        case 5: return run_w8_tc<DT, 32>(a, workspace, shift, s);
        case 6: return run_w8_tc<DT, 64>(a, workspace, shift, s);
        case 7: return run_w8_tc<DT, 128>(a, workspace, shift, s);
        default: return run_w8_tc<DT, 256>(a, workspace, shift, s);
    }
}

cudaError_t launch_w8_tc(int dtype, const W8Args &a, void *workspace, cudaStream_t s) {
    const int shift = w8_token_shift(a.tokens);
    uint8_t *const to = static_cast<uint8_t *>(workspace);
    const int sweep = (a.l.chunks + kWeThreads / 16 - 1) / (kWeThreads / 16);
    const dim3 grid(static_cast<unsigned>((a.tokens + 7) / 8), static_cast<unsigned>(sweep < 65535 ? sweep : 65535));
    const cudaError_t err = launch_chained(w8_expand_kernel, grid, kWeThreads, 0, s, a, to, shift);
    if (err != cudaSuccess) return err;
    return dtype ? pick_tokens<1>(shift, a, to, s) : pick_tokens<0>(shift, a, to, s);
}

}  // namespace qrk
