// qr_w8_tc.cu -- y = x W^T for 17 and more rows of x and weights in 8 bits, on
// tcgen05 (qr_w8_matmul; W8Layout in qr_serving.h describes the packed order).
//
// The fast integer products of this GPU are those of 16-bit floats: codes are
// exact fp16 numbers, their products exact in fp32.  A first kernel writes x's
// codes as fp16 into the workspace, in the order and with the swizzle that the
// products read from shared memory, so that a chunk of 64 columns of a CTA's
// tokens is one bulk copy.  Then y^T = W x^T in tiles of 128 weight rows by N
// tokens: eight warps, a row tile of 16 each, turn packed codes into fp16 and store
// them as the A operand in tensor memory, one warp brings x, one issues the
// products, and four or eight scale and store a finished tile while the next one runs.
//
// The chunks of all tiles, one tile after the other, are divided evenly among
// the CTAs, one an SM, or whole tiles are where that is quicker.  A tile that one
// CTA has whole is stored by it; the parts of the others go to the workspace as fp32
// sums, and a last kernel adds them in order, so that the result has the same bits
// every time.
//
// What bounds it: with 256 tokens a tile the products (4096 tokens through 10240 x
// 8192: 405 to 436 us as the clock goes under the power limit, 1.58 to 1.70 PFLOP/s;
// 1024 tokens 106 to 108 us, the tensor pipe busy 82%); with fewer the weights' bytes, in
// the steady state, and around it the first kernel, the first loads' way and the
// join, some 7 us (64 tokens 23 us, 3.7 TB/s; 129 through 20481 x 5123 37.6 us: the
// two rings in shared memory hold too little of either operand for HBM's latency).
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
__global__ void __launch_bounds__(kWeThreads) w8_expand_kernel(W8Args a, uint8_t *to, int n) {
    // the product may start once everything before this kernel is complete: until
    // its own wait it reads the weights only
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int chunks = a.l.chunks;
    // eight tokens of two chunks a warp
    const long long token = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 1 & 7);
    if (token >= a.tokens) return;
    const unsigned tile = static_cast<unsigned>(token) / n;  // (tokens are below 2^31)
    const int j = threadIdx.x & 1, row = static_cast<int>(token - static_cast<long long>(tile) * n);
    const int8_t *const src = a.x + token * a.x_stride + j * 32;
    uint8_t *const dst = to + static_cast<long long>(tile) * chunks * n * 128;
    for (int c = blockIdx.y * (kWeThreads / 16) + (threadIdx.x >> 4); c < chunks; c += gridDim.y * (kWeThreads / 16)) {
        const int have = a.cols - c * 64 - j * 32;
        const uint4 p = load16_codes(src + c * 64, have), q = load16_codes(src + c * 64 + 16, have - 16);
        const uint32_t u[4] = {p.x, p.y, p.z, p.w}, v[4] = {q.x, q.y, q.z, q.w};
        uint8_t *const block = dst + static_cast<long long>(c) * n * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 o;
            codes_f16(u[i], o.x, o.y);
            codes_f16(v[i], o.z, o.w);
            *reinterpret_cast<uint4 *>(block + swizzled(row, 2 * i + j)) = o;
        }
    }
}

// Up to 192 tokens a tile the weights' bytes bound the kernel, or x's and theirs
// alike: the packed codes come through shared memory, some steps ahead.  With more, x
// fills that, and the products leave time for two steps in the registers of the
// warps that convert them (1024 tokens through 10240 x 8192: through shared memory
// 111 us, registers 108; 129 through 20481 x 5123: 39 and 44).
template <int N>
constexpr bool kWtStaged = N <= 192;
// Warps 0-7 codes, 8 products, 9 x, then those of the results (four where the codes'
// warps need the registers), and a last one for the packed codes' way in.
template <int N>
constexpr int kWtResults = kWtStaged<N> ? 8 : 4;
template <int N>
constexpr int kWtThreads = 32 * (10 + kWtResults<N> + kWtStaged<N>);
constexpr int kWtRows = 128;
constexpr uint32_t kWtColumns = 512;  // of tensor memory: codes, then accumulators
constexpr int kWtMostCtas = 152;  // the workspace has two parts for each

// N: tokens of a tile, at most.
template <int N>
struct WtSmem {
    static constexpr int kBlock = N * 128;
    // chunks of a step; buffers of codes in tensor memory, and of packed ones, a step
    // each; accumulators
    static constexpr int kStep = 4, kA = N <= 64 ? 3 : 2;
    static constexpr int kW = !kWtStaged<N> ? 1 : N > 64 ? 2 : N > 32 ? 3 : 4;
    static constexpr int kD = N > 128 ? 1 : 2;
    static constexpr uint32_t kColD = kA * 32 * kStep;
    static_assert(kColD + kD * N <= kWtColumns, "tensor memory");
    // x: chunks that are handed on together (a wait and a commit take the products'
    // warp some 150 cycles, four chunks' products of 64 tokens run for 512), and
    // buffers of them
    static constexpr int kXc = N > 192 ? 1 : N > 64 ? 2 : 4;
    static constexpr int kX = N > 192 ? 6 : N > 128 ? 3 : N > 64 ? 4 : N > 32 ? 3 : 4;
    uint8_t x[kX * kXc * kBlock];
    uint8_t codes[kW][8][kWtStaged<N> ? kStep * 1024 : 16];  // by warp: its row tile
    uint8_t out[kWtResults<N>][16 * 80];                     // by warp: 16 tokens of 32 rows
    float x_scale[kWtResults<N>][N];                         // by warp
    uint64_t a_full[kA], a_done[kA], x_full[kX], x_done[kX], d_full[kD], d_done[kD], w_full[kW], w_done[kW];
    uint32_t tmem;
    int fail;
};

// The division of the chunks: all = tiles * chunks of them over `ctas`.
struct W8Shares {
    long long all, each;  // each = all / ctas
    int rest;             // all % ctas
    int chunks, row_ctas, ctas, n;  // n: tokens of a tile, a multiple of 16

    __host__ __device__ __forceinline__ long long begin(int cta) const { return each * cta + rest * cta / ctas; }
    // (64-bit divisions take hundreds of cycles at a kernel's start)
    __device__ __forceinline__ long long divide(long long x, int d) const {
        return all <= 0x7fffffff ? static_cast<long long>(static_cast<unsigned>(x) / static_cast<unsigned>(d)) : x / d;
    }
};

// Walks a CTA's chunks, a step of up to STEP chunks of one tile at a time.
template <int STEP>
struct W8Walk {
    long long left;
    int chunk, chunks, row_tile, row_ctas;
    long long token_tile;

    __device__ __forceinline__ W8Walk(const W8Shares &s, int cta) {
        const long long u = s.begin(cta), tile = s.divide(u, s.chunks);
        left = s.begin(cta + 1) - u;
        chunk = static_cast<int>(u - tile * s.chunks);
        chunks = s.chunks;
        row_ctas = s.row_ctas;
        token_tile = s.divide(tile, row_ctas);
        row_tile = static_cast<int>(tile - token_tile * row_ctas);
    }
    __device__ __forceinline__ int step() const {
        return static_cast<int>(min(static_cast<long long>(min(STEP, chunks - chunk)), left));
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
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, block = shares.n * 128;
    int *const fail = &sm.fail;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    W8Walk<S::kStep> at(shares, blockIdx.x);
    if (tid == 0) {
        for (int i = 0; i < S::kA; ++i) {
            mbar_init(&sm.a_full[i], 8);
            mbar_init(&sm.a_done[i], 1);
        }
        for (int i = 0; i < S::kX; ++i) {
            mbar_init(&sm.x_full[i], 1);
            mbar_init(&sm.x_done[i], 1);
        }
        for (int i = 0; i < S::kD; ++i) {
            mbar_init(&sm.d_full[i], 1);
            mbar_init(&sm.d_done[i], kWtResults<N>);
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
            tc_st_fragments(to + b * (32 * S::kStep) + k * 32, v);  // (past the step's last chunk: unused)
        };
        auto hand_on = [&](int b) {
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.a_full[b]);
        };
        bool ok = true;
        if constexpr (kWtStaged<N>) {
            for (unsigned p = 0; at.left > 0; ++p) {
                const unsigned b = p % S::kA, ws = p % S::kW;
                ok = tc_wait_warp(&sm.w_full[ws], (p / S::kW) & 1, fail, timeouts);
                const uint32_t from = smem_addr(sm.codes[ws][2 * quarter + (warp >> 2)]) + lane * 16;
                uint4 w[S::kStep][2];
#pragma unroll
                for (int u = 0; u < S::kStep; ++u) w[u][0] = lds128(from + u * 1024), w[u][1] = lds128(from + u * 1024 + 512);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.w_done[ws]);
                if (ok && p >= S::kA) ok = tc_wait_warp(&sm.a_done[b], (p / S::kA - 1) & 1, fail, timeouts);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int u = 0; u < S::kStep; ++u) convert(w[u][0], w[u][1], b, u);
                hand_on(b);
                at.advance(at.step());
            }
        } else {
            static_assert(S::kA == 2, "a buffer each for two steps");
            W8Walk<S::kStep> ahead = at;
            const int mine = 2 * quarter + (warp >> 2);
            uint4 w[2][S::kStep][2];
            auto fetch = [&](int b) {
                if (ahead.left <= 0) return;
                const int n = ahead.step();
                const long long tile = min(ahead.row_tile * (kWtRows / 16) + mine, a.l.row_tiles - 1);
                const uint4 *const src = reinterpret_cast<const uint4 *>(a.packed) + (tile * a.l.chunks + ahead.chunk) * 64 + lane;
#pragma unroll
                for (int u = 0; u < S::kStep; ++u)
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
                    for (int u = 0; u < S::kStep; ++u) convert(w[b][u][0], w[b][u][1], b, u);
                    hand_on(b);
                    at.advance(at.step());
                    fetch(b);
                }
            }
        }
    } else if (warp == 8) {
        // ---- products
        const bool leader = elect_lane();
        const uint32_t desc = mma_desc(shares.n, false);
        bool ok = true;
        unsigned p = 0, i = 0;
        for (unsigned g = 0; at.left > 0 && ok; ++g) {
            const unsigned d = g % S::kD;
            int n = at.segment();
            if (g >= S::kD) ok = tc_wait_warp(&sm.d_done[d], (g / S::kD - 1) & 1, fail, timeouts);
            bool add = false;
            while (n > 0 && ok) {
                const int s = p % S::kA, chunks = at.step();
                ok = tc_wait_warp(&sm.a_full[s], (p / S::kA) & 1, fail, timeouts);
                for (int u0 = 0; u0 < chunks && ok; u0 += S::kXc, ++i) {
                    const int xs = i % S::kX;
                    ok = tc_wait_warp(&sm.x_full[xs], (i / S::kX) & 1, fail, timeouts);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t x = smem_addr(sm.x) + xs * (S::kXc * S::kBlock), codes = tmem + s * (32 * S::kStep) + u0 * 32;
#pragma unroll
                    for (int k = 0; k < S::kXc; ++k) {
                        if (u0 + k >= chunks) break;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            tc_mma_ts(leader, tmem + S::kColD + d * N, codes + k * 32 + j * 8,
                                      smem_desc(x + k * block + j * 32, 16, 1024), desc, add || k + j > 0);
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
                    const uint32_t bytes = min(S::kXc, chunks - u0) * block;
                    mbar_arrive_expect_tx(&sm.x_full[xs], bytes);
                    bulk_copy_g2s(sm.x + xs * (S::kXc * S::kBlock), x16 + (at.token_tile * at.chunks + at.chunk + u0) * block,
                                  bytes, &sm.x_full[xs]);
                }
                at.advance(chunks);
            }
            // none of the copies is on its way when the CTA leaves
            for (unsigned k = i < S::kX ? 0 : i - S::kX; k < i; ++k) mbar_wait(&sm.x_full[k % S::kX], (k / S::kX) & 1);
        }
        __syncwarp();
    } else if (warp == 10 + kWtResults<N>) {
        // ---- the packed codes' way in: a step of a row tile is one copy
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
    } else {
        // ---- results: a thread per row, 16 tokens at a time
        constexpr int kStride = 4 * kWtResults<N>;  // tokens between a warp's groups
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int mine = warp - 10;
        const uint32_t stage = smem_addr(sm.out[mine]), x_scale = smem_addr(sm.x_scale[mine]);
        const uintptr_t odd = reinterpret_cast<uintptr_t>(a.y) | static_cast<uintptr_t>(a.y_stride * 2);
        const int wide = (odd & 15) == 0 ? 16 : (odd & 7) == 0 ? 8 : 2;  // bytes of a store
        long long held = -1;  // the tokens whose scales are in shared memory
        bool ok = true;
        for (unsigned g = 0; at.left > 0; ++g) {
            const unsigned d = g % S::kD;
            const int n = at.segment();
            const bool whole = n == at.chunks;
            const long long token0 = at.token_tile * shares.n, row0 = static_cast<long long>(at.row_tile) * kWtRows + quarter * 32;
            const int tokens = static_cast<int>(min(static_cast<long long>(shares.n), a.tokens - token0));
            if (whole && held != at.token_tile) {
                held = at.token_tile;
                __syncwarp();
                for (int m = lane; m < N; m += 32) sm.x_scale[mine][m] = m < tokens ? a.x_scales[token0 + m] : 0.0f;
                __syncwarp();
            }
            const float scale = row0 + lane < a.rows ? reinterpret_cast<const float *>(a.packed + a.l.scales_at)[row0 + lane] : 0.0f;
            float *const part = parts + (2ll * blockIdx.x + (at.chunk == 0)) * (kWtRows * N) + quarter * 32 + lane;
            ok = tc_wait_warp(&sm.d_full[d], (g / S::kD) & 1, fail, timeouts);
            if (!ok) break;
            tc_fence_after();
            const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + S::kColD + d * N;
            const int first = (mine >> 2) * 16;
            if (first >= tokens && lane == 0) mbar_arrive(&sm.d_done[d]);
#pragma unroll 1
            for (int m0 = first; m0 < tokens; m0 += kStride) {
                uint32_t v[16];
                tc_ld16(lanes + m0, v);
                tc_wait_ld(v);
                if (m0 + kStride >= tokens) {  // (the accumulator is read)
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.d_done[d]);
                }
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) part[(m0 + e) * kWtRows] = __uint_as_float(v[e]);
                    continue;
                }
                // (the scales first: loads between the stores would wait for them)
                float xs[16];
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const uint4 q = lds128(x_scale + (m0 + e) * 4);
                    xs[e] = __uint_as_float(q.x), xs[e + 1] = __uint_as_float(q.y);
                    xs[e + 2] = __uint_as_float(q.z), xs[e + 3] = __uint_as_float(q.w);
                }
                uint16_t y[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = narrow1<DT>(__uint_as_float(v[e]) * xs[e] * scale);
                if (wide == 2) {
                    uint16_t *const to = a.y + (token0 + m0) * a.y_stride + row0 + lane;
                    if (row0 + lane < a.rows) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (m0 + e < tokens) to[e * a.y_stride] = y[e];
                    }
                    continue;
                }
                // through shared memory, [token][row], to pieces of a token's rows
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(stage + e * 80 + lane * 2), "h"(y[e]) : "memory");
                __syncwarp();
                const int each = wide == 16 ? 8 : 4;  // rows of a piece
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int piece = q * 32 + lane, m = wide == 16 ? piece >> 2 : piece >> 3, k = (wide == 16 ? piece & 3 : piece & 7) * each;
                    if (m >= 16) break;
                    uint16_t *const to = a.y + (token0 + m0 + m) * a.y_stride + row0 + k;
                    const int rows = static_cast<int>(min(a.rows - row0 - k, static_cast<long long>(each)));
                    if (m0 + m >= tokens || rows <= 0) continue;
                    const uint2 lo = lds64(stage + m * 80 + k * 2);
                    if (wide == 16) {
                        const uint2 hi = lds64(stage + m * 80 + k * 2 + 8);
                        if (rows == 8) {
                            *reinterpret_cast<uint4 *>(to) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                        } else {
                            const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
                            for (int r = 0; r < 7; ++r)
                                if (r < rows) to[r] = static_cast<uint16_t>(w[r >> 1] >> (16 * (r & 1)));
                        }
                    } else if (rows == 4) {
                        *reinterpret_cast<uint2 *>(to) = lo;
                    } else {
#pragma unroll
                        for (int r = 0; r < 3; ++r)
                            if (r < rows) to[r] = static_cast<uint16_t>((r < 2 ? lo.x : lo.y) >> (16 * (r & 1)));
                    }
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
// which CTA x's share ends, y a group of tokens of it, kJoinEach for a warp, whose
// lanes are a token's 128 rows.  What is not a part (the scales) was there before
// the product began, and is read before its end.
constexpr int kJoinThreads = 256;
template <int DT, int kJoinEach>
__global__ void __launch_bounds__(kJoinThreads, 4) w8_join_kernel(W8Args a, W8Shares shares, const float *parts, int pitch) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kWarps = kJoinThreads / 32, kJoinTokens = kWarps * kJoinEach;
    const int lane = threadIdx.x & 31, first = blockIdx.x;
    const long long end = shares.begin(first + 1), tile = shares.divide(end - 1, shares.chunks);
    const long long from = tile * shares.chunks, to = from + shares.chunks;
    if (end == to || shares.begin(first) > from) {  // whole, or another block's to add
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    int last = first + 1;
    while (shares.begin(last + 1) < to) ++last;
    const long long token_tile = shares.divide(tile, shares.row_ctas);
    const long long row = (tile - token_tile * shares.row_ctas) * kWtRows + lane * 4;
    const int col = blockIdx.y * kJoinTokens + (threadIdx.x >> 5);  // and every kWarps-th from there
    const long long token = token_tile * shares.n + col;
    const int have = static_cast<int>(min(a.tokens - token, static_cast<long long>(shares.n - col)));  // tokens from here on
    float4 scale = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (row < a.rows) scale = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(a.packed + a.l.scales_at) + row);
    float x_scale[kJoinEach];
#pragma unroll
    for (int k = 0; k < kJoinEach; ++k) x_scale[k] = kWarps * k < have ? a.x_scales[token + kWarps * k] : 0.0f;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (have <= 0) return;
    // CTA c's parts are 2 c and, of the tile that begins in its share, 2 c + 1
    const float4 *const p = reinterpret_cast<const float4 *>(parts) + col * (kWtRows / 4) + lane;
    const long long next = static_cast<long long>(kWtRows / 4) * pitch;
    auto load = [&](float4 (&v)[kJoinEach], long long part) {
#pragma unroll
        for (int k = 0; k < kJoinEach; ++k)
            if (kWarps * k < have) v[k] = __ldcg(p + part * next + k * kWarps * (kWtRows / 4));
    };
    float4 sum[kJoinEach] = {}, v[kJoinEach] = {};
    load(sum, 2ll * first + 1);
#pragma unroll 2
    for (int c = first + 1; c <= last; ++c) {
        load(v, 2ll * c);
#pragma unroll
        for (int k = 0; k < kJoinEach; ++k) sum[k].x += v[k].x, sum[k].y += v[k].y, sum[k].z += v[k].z, sum[k].w += v[k].w;
    }
    const bool vector = (reinterpret_cast<uintptr_t>(a.y) & 7) == 0 && a.y_stride % 4 == 0 && a.rows % 4 == 0;
    uint16_t *to_y = a.y + token * a.y_stride + row;
#pragma unroll
    for (int k = 0; k < kJoinEach; ++k, to_y += kWarps * a.y_stride) {
        if (kWarps * k >= have) break;
        const float s = x_scale[k];
        const uint2 o = make_uint2(narrow2<DT>(sum[k].x * s * scale.x, sum[k].y * s * scale.y),
                                   narrow2<DT>(sum[k].z * s * scale.z, sum[k].w * s * scale.w));
        if (vector) {
            if (row < a.rows) *reinterpret_cast<uint2 *>(to_y) = o;
            continue;
        }
        // a store's lanes on consecutive rows: row 32 j + lane is the (lane % 4)-th of lane 8 j + lane / 4
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = __shfl_sync(~0u, o.x, 8 * j + (lane >> 2)), hi = __shfl_sync(~0u, o.y, 8 * j + (lane >> 2));
            const uint32_t w = lane & 2 ? hi : lo;
            const int at = 32 * j + lane - 4 * lane;  // from this lane's rows
            if (row + at < a.rows) to_y[at] = static_cast<uint16_t>(lane & 1 ? w >> 16 : w);
        }
    }
}

static size_t w8_x16_bytes(long long tokens, int chunks, int n) {
    return static_cast<size_t>((tokens + n - 1) / n * n) * chunks * 128;
}

// The kernel that takes tiles of n tokens.
static int w8_most_tokens(int n) { return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : n <= 192 ? 192 : 256; }

size_t w8_workspace(long long tokens, int cols) {
    // (tiles in equal shares of fewer tokens than 256 hold less than a tile more)
    const int most = tokens <= 32 ? 32 : tokens <= 64 ? 64 : tokens <= 128 ? 128 : 256;
    return w8_x16_bytes(tokens > 256 ? tokens + 256 : tokens, cols / 64 + (cols % 64 != 0), most) + size_t(2) * kWtMostCtas * kWtRows * 4 * most;
}

template <int DT, int N>
static cudaError_t run_w8_tc(const W8Args &a, const W8Shares &shares, uint8_t *workspace, cudaStream_t s) {
    const int n = shares.n;
    auto kern = w8_tc_kernel<DT, N>;
    const int bytes = sizeof(WtSmem<N>) + 1024;
    cudaError_t err = allow_dynamic_smem(reinterpret_cast<const void *>(kern), bytes);
    if (err != cudaSuccess) return err;
    unsigned *timeouts = wait_timeout_counter(&err);
    if (!timeouts) return err;
    float *const parts = reinterpret_cast<float *>(workspace + w8_x16_bytes(a.tokens, a.l.chunks, n));
    err = launch_chained(kern, shares.ctas, kWtThreads<N>, bytes, s, a, shares, static_cast<const uint8_t *>(workspace), parts,
                         timeouts);
    if (err != cudaSuccess) return err;
    bool joined = false;
    for (int c = 1; c < shares.ctas && !joined; ++c) joined = shares.begin(c) % a.l.chunks != 0;
    if (!joined) return cudaSuccess;
    // fewer tokens a warp where there are few (64 tokens: 16 in a block 23.0 us, 32
    // 23.7; 1024 through 1280 x 8192: 32.6 and 30.6)
    auto join = [&](auto kernel, int each) {
        const unsigned groups = static_cast<unsigned>((n + 8 * each - 1) / (8 * each));
        return launch_chained(kernel, dim3(shares.ctas - 1, groups), kJoinThreads, 0, s, a, shares,
                              static_cast<const float *>(parts), N);  // (parts are N tokens apart)
    };
    return n <= 96 ? join(w8_join_kernel<DT, 2>, 2) : join(w8_join_kernel<DT, 4>, 4);
}

template <int DT>
static cudaError_t pick_tokens(const W8Args &a, const W8Shares &p, uint8_t *workspace, cudaStream_t s) {
    switch (w8_most_tokens(p.n)) {
        case 32: return run_w8_tc<DT, 32>(a, p, workspace, s);
        case 64: return run_w8_tc<DT, 64>(a, p, workspace, s);
        case 128: return run_w8_tc<DT, 128>(a, p, workspace, s);
        case 192: return run_w8_tc<DT, 192>(a, p, workspace, s);
        default: return run_w8_tc<DT, 256>(a, p, workspace, s);
    }
}

// The tiles' tokens, equal shares of up to 128, 192 or 256, and the division of their
// chunks: a CTA for each tile where there are no more tiles than SMs, or even shares,
// whose divided tiles' parts are joined; by what each takes, in microseconds.  A chunk is
// bound by its products or its hand-overs, and weights that do not stay in L2 between
// tiles by HBM; a tile's results are stored beside the next one's products where there
// are two accumulators; joining takes a launch, the parts' way to L2 and back, and some
// time for each part of a tile.
static W8Shares w8_shares(const W8Args &a, int sms) {
    W8Shares best = {};
    double least = 0.0;
    for (int most = 128; most <= 256; most += 64) {
        const long long token_tiles = (a.tokens + most - 1) / most;
        const int n = static_cast<int>(((a.tokens + token_tiles - 1) / token_tiles + 15) / 16 * 16);
        W8Shares p = {0, 0, 0, a.l.chunks, (a.l.row_tiles + 7) / 8, 1, n};
        const long long tiles = token_tiles * p.row_ctas;
        p.all = tiles * p.chunks;
        const double chunk = n > 192 ? n * 0.0011 : n > 128 ? 0.3 : a.l.scales_at > (32 << 20) ? 0.22 : 0.19;
        const double results = n * (n > 192 ? 0.013 : 0.007);
        const double tile = n > 128 ? p.chunks * chunk + results : p.chunks * chunk > results ? p.chunks * chunk : results;
        p.ctas = static_cast<int>(tiles < sms ? tiles : sms);
        double cost = static_cast<double>((tiles + p.ctas - 1) / p.ctas) * tile + results;
        for (int c = sms; c >= 8; c = c * 3 / 4) {
            const double each = static_cast<double>(p.all) / c;
            const double split = each / p.chunks * tile + results + 3.0 + (each < p.chunks ? p.chunks / each : 1.0) * 0.3 +
                                 c * n * (4.0 * kWtRows * 4 / 1e7);
            if (each >= 4 && split < cost) cost = split, p.ctas = c;
        }
        if (least == 0.0 || cost < least) least = cost, best = p;
        if (a.tokens <= most) break;
    }
    best.each = best.all / best.ctas;
    best.rest = static_cast<int>(best.all % best.ctas);
    return best;
}

cudaError_t launch_w8_tc(int dtype, const W8Args &a, void *workspace, cudaStream_t s) {
    cudaError_t err = cudaSuccess;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    const W8Shares p = w8_shares(a, sms < kWtMostCtas ? sms : kWtMostCtas);
    uint8_t *const to = static_cast<uint8_t *>(workspace);
    const int sweep = (a.l.chunks + kWeThreads / 16 - 1) / (kWeThreads / 16);
    const dim3 grid(static_cast<unsigned>((a.tokens + 7) / 8), static_cast<unsigned>(sweep < 65535 ? sweep : 65535));
    err = launch_chained(w8_expand_kernel, grid, kWeThreads, 0, s, a, to, p.n);
    if (err != cudaSuccess) return err;
    return dtype ? pick_tokens<1>(a, p, to, s) : pick_tokens<0>(a, p, to, s);
}

}  // namespace qrk
