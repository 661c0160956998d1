// qr_kv_tc.cuh -- attention over the 8-bit paged cache for many query rows, on
// tcgen05.
//
// An item is 256 query rows (a row is a query token and one of the group's
// heads) of one request and key/value head, in two halves of 128; its keys are
// taken 128 at a time.  As in qr_kv_split.cuh the items' key tiles are cut into
// equal shares, one per CTA (here counting only tiles that some row sees), and
// the parts of a divided item are joined by whichever CTA brings the last one.
//
// Thirteen warps of a CTA work.  Four convert: each tile's codes come through
// registers and go to shared memory as fp16 (exact), double buffered; both
// halves use them.  One thread issues the products, S = Q K^T and O += P V,
// with S, P and O in tensor memory.  Four warps per half, a thread per row, do
// the softmax: S is read twice (maximum, then weights, which replace it as
// fp16), 32 values at a time with the next 32 on their way.  While one half's
// weights are computed, the tensor cores work on the other's products.
//
// O stays in tensor memory.  It is rescaled only when a row's maximum has
// grown by more than 2^kSlack, or the power of two under which the values'
// scales are kept by more than 2^kScaleSlack; weights are then below 2^15, and
// fp16 keeps them exact to 2^-12 down to 2^-21 of a weight of 1.  What that
// rounding left is a second P, as in qr_kv_split.cuh (8 prompt chunks of up to
// 1024 queries over up to 8192 keys: 409 us, with one P 364, and outputs 0.001
// of their norm away from a product in 32 bits instead of 0.0001).
//
// What bounds it: latency.  A tile of both halves takes some 4500 cycles, of
// which the products take two thirds and the softmax's and conversion's issue
// about as many; a half's chain of scores, maximum, weights and their store leaves
// gaps that the other half does not fill (8 prompt chunks of up to 1024 queries
// over up to 8192 keys, 40 heads on 8, 128 dimensions: 410 us, 702 TFLOP/s).
#pragma once

#include "qr_kv_split.cuh"
#include "qr_tcgen05.cuh"

namespace qrk {

constexpr int kTcRows = 256, kTcHalf = 128, kTcKeys = 128;
constexpr int kTcThreads = 416;  // warps 0-7 softmax, 8-11 conversion, 12 products
// An item's queries, output, masked tiles and empty pipeline take about as long
// as this many tiles; the shares count them, as tiles before the first one (8
// prompt chunks over up to 8192 keys: 3 436 us, 4 409, 5 414, 8 431; 32 chunks
// of 200 over up to 700 163, 163, 169, 170; 4 of 64 over 20000 120, 119, 121,
// 121; a prompt of 2048 86, 88, 88, 92).
constexpr int kItemSteps = 4;
constexpr int kTcMostCtas = 160;
constexpr float kSlack = 6.0f;
constexpr int kScaleSlack = 2;
constexpr int kTcWeightExp = 7;  // weight 1 of the largest scale is 2^7
// Where a tile's weights are taken together with the values' scales in one
// exponent, the smallest scale is at most so many powers of two below the row's
// power, and that at most so large: a weight of 2^-60 of the row's largest, and
// its part of the sum, are then still normal numbers.
constexpr int kScaleSpan = 64, kMostScaleExp = 64;

// Tensor memory columns: S of both halves (P in its place), O of both halves.
constexpr uint32_t kColS = 0, kColO = 256, kColumns = 512;

// A tile's scales and what follows from them, read a 16-key group ahead of
// its use: beside the products, which read shared memory at its full rate, a
// load of it takes 100 to 170 cycles.
struct alignas(16) TcMeta {
    float4 group[8];  // key scale; log2 of, one over, and the value scale
    int4 tile;        // valid groups; the largest scale_exp among them; whether
                      // every group is valid and no value scale is zero or near
                      // it; the smallest scale_exp if so
};

// Floats of one half's part: accumulators, then (max, sum) pairs.
template <int DP>
constexpr int kTcSlot = kTcHalf * (DP + 2);

// The items of a CTA's share, in order; every warp keeps its own copy, in
// shared memory, which its first lane moves on.
struct TcWalk {
    long long step, last, share, at;
    int r, j, tiles_of_r;
    AttnRequest x;
    // the current item
    long long item_first;
    int head, row0, rows, begin, end, steps, p0;
    int part_first_cta, parts;
    bool more;

    // The keys that some row of row tile `jj` sees, [b, e).
    __device__ __forceinline__ static int range(const KvAttentionArgs &a, const AttnRequest &x, int group, int jj, int *b,
                                                int *e) {
        const int p0 = x.kv - x.nq, rows = min(kTcRows, x.nq * group - jj * kTcRows);
        const int pos_first = p0 + jj * kTcRows / group, pos_last = p0 + (jj * kTcRows + rows - 1) / group;
        *e = a.causal ? max(0, min(x.kv, pos_last + 1)) : x.kv;
        *b = a.window > 0 ? max(0, pos_first - a.window + 1) / 16 * 16 : 0;
        return kItemSteps + (*e > *b ? (*e - *b + kTcKeys - 1) / kTcKeys : 0);
    }
    __device__ __forceinline__ void enter(const KvAttentionArgs &a, const KvView &c, int group, int request) {
        r = request;
        j = 0;
        x = attn_request(a, c, kTcRows, group, r);
        tiles_of_r = x.items / c.heads;
    }
    __device__ __forceinline__ bool next(const KvAttentionArgs &a, const KvView &c, int group, const long long *run_steps) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) more = advance(a, c, group, run_steps);
        __syncwarp();
        return more;
    }
    __device__ __forceinline__ bool advance(const KvAttentionArgs &a, const KvView &c, int group, const long long *run_steps) {
        if (step >= last) return false;
        if (r < 0) {
            int lo = 0, hi = 127;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (run_steps[mid] <= step) lo = mid; else hi = mid - 1;
            }
            at = run_steps[lo];
            enter(a, c, group, lo * ((a.requests + 127) / 128));
        }
        int b, e;
        for (;;) {
            if (j >= tiles_of_r) {
                enter(a, c, group, r + 1);
                continue;
            }
            steps = range(a, x, group, j, &b, &e);
            if (step < at + static_cast<long long>(steps) * c.heads) break;
            at += static_cast<long long>(steps) * c.heads;
            ++j;
        }
        head = static_cast<int>((step - at) / steps);
        item_first = at + static_cast<long long>(head) * steps;
        const int s0 = static_cast<int>(step - item_first), s1 = static_cast<int>(min(item_first + steps, last) - item_first);
        // its first part is the one with its first tile: a share that ends
        // before that leaves the item alone
        const int lead = min(kItemSteps, steps - 1);
        if (s1 <= lead) {
            step = last;
            return false;
        }
        begin = b + max(0, s0 - kItemSteps) * kTcKeys;
        end = min(b + max(0, s1 - kItemSteps) * kTcKeys, e);
        row0 = j * kTcRows;
        rows = min(kTcRows, x.nq * group - row0);
        p0 = x.kv - x.nq;
        part_first_cta = static_cast<int>((item_first + lead) / share);
        parts = static_cast<int>((item_first + steps - 1) / share) - part_first_cta + 1;
        step = item_first + s1;
        return true;
    }
    __device__ __forceinline__ int tiles() const { return end > begin ? (end - begin + kTcKeys - 1) / kTcKeys : 0; }
};

template <int DP>
struct TcSmem {
    static constexpr int kSlabs = DP / 64, kTile = kSlabs * 16384;  // 128 rows of fp16
    uint8_t q[2][kTile];
    uint8_t k[2][kTile];
    uint8_t v[2][kTile];
    TcMeta meta[4];
    long long run_steps[128], warp_sums[4];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];  // by buffer
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];    // by half
    TcWalk walk[13];
    uint32_t tmem;
    unsigned ticket[2];
    int fail;
};

template <bool BF16>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
    if (!BF16) return pack_f16(lo, hi);
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// The 128 threads of one half's softmax.
__device__ __forceinline__ void bar_half(int half) { asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory"); }

template <int DP, bool FULL, bool BF16>
__global__ void __launch_bounds__(kTcThreads, 1)
    kv_attention_tc_kernel(KvAttentionArgs a, KvView c, int group, unsigned *timeouts) {
    chain_entry();
    using S = TcSmem<DP>;
    extern __shared__ uint8_t raw[];
    S &sm = *reinterpret_cast<S *>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
    // weights as two fp16 numbers: kTerms * 8 of S's columns for each 16 keys
    constexpr int kTerms = 2;
    const int dim = FULL ? DP : c.dim;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // sums of the steps over 128 runs of requests
    {
        const int per = (a.requests + 127) / 128;
        long long steps = 0, incl = 0;
        if (tid < 128) {
            const int r0 = min(tid * per, a.requests), r1 = min(r0 + per, a.requests);
            for (int r = r0; r < r1; ++r) {
                const AttnRequest x = attn_request(a, c, kTcRows, group, r);
                int b, e;
                for (int j = 0; j < x.items / c.heads; ++j)
                    steps += static_cast<long long>(TcWalk::range(a, x, group, j, &b, &e)) * c.heads;
            }
            incl = steps;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long o = __shfl_up_sync(~0u, incl, d);
                if (lane >= d) incl += o;
            }
            if (lane == 31) sm.warp_sums[warp] = incl;
        }
        if (tid == 128) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sm.k_full[i], 128);
                mbar_init(&sm.v_full[i], 128);
                mbar_init(&sm.k_empty[i], 1);
                mbar_init(&sm.v_empty[i], 1);
                mbar_init(&sm.q_full[i], 128);
                mbar_init(&sm.s_full[i], 1);
                mbar_init(&sm.p_full[i], 128);
                mbar_init(&sm.o_full[i], 1);
            }
            mbar_init_fence();
            sm.fail = 0;
        }
        if (warp == 12) tc_alloc(&sm.tmem, kColumns);
        __syncthreads();
        if (tid < 128) {
            long long before = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                if (w < warp) before += sm.warp_sums[w];
            sm.run_steps[tid] = before + incl - steps;
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    const uint32_t tmem = sm.tmem;
    TcWalk &walk = sm.walk[warp];
    if (lane == 0) {
        const long long all = sm.warp_sums[0] + sm.warp_sums[1] + sm.warp_sums[2] + sm.warp_sums[3];
        walk.share = (all + gridDim.x - 1) / gridDim.x;
        walk.step = walk.share * blockIdx.x;
        walk.last = min(walk.step + walk.share, all);
        walk.at = 0;
        walk.r = -1;
    }
    int *const fail = &sm.fail;

    if (warp >= 8 && warp < 12) {
        // ---- the codes, through registers, to fp16 tiles in shared memory
        const int ct = tid - 256;
        constexpr int kPer = DP / 16;           // 16-byte pieces of a padded row; also passes
        constexpr int kPassRows = 128 / kPer;
        // a thread's piece and row of a pass: the eight lanes of one phase hold
        // four pieces of an even and of an odd row, whose swizzled places differ
        const int q_l = kPer == 8 ? (lane & 3) | (lane >> 1 & 4) : lane & 3;
        const int row_l = kPer == 8 ? (warp & 3) * 4 + (lane >> 4) * 2 + (lane >> 2 & 1) : (warp & 3) * 8 + (lane >> 2);
        const bool in_row = FULL || q_l * 16 < dim;
        const int in_block = (1 << c.shift) - 1;
        uint32_t it = 0;
        while (walk.next(a, c, group, sm.run_steps)) {
            const int tiles = walk.tiles();
            const int32_t *const table = a.table + static_cast<long long>(walk.r) * a.width;
            const long long khead = walk.head * c.k_head + q_l * 16, vhead = walk.head * c.v_head + q_l * 16;
            int id[kPer], mid = -1;
            float mks = 0.0f, mvs = 0.0f;
            uint4 kr[kPer], vr[kPer];
            auto ids = [&](int i) {
                const int key0 = walk.begin + i * kTcKeys;
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int key = (key0 + row_l + j * kPassRows) & ~15;
                    id[j] = -1;
                    if (key < walk.end) id[j] = table[key >> c.shift];
                    if (id[j] >= c.blocks) id[j] = -1;
                }
                mid = -1;
                if (ct < 8 && key0 + ct * 16 < walk.end) mid = table[(key0 + ct * 16) >> c.shift];
                if (mid >= c.blocks) mid = -1;
            };
            auto load = [&](int i, uint4 (&reg)[kPer], const int8_t *base, long long block, long long head_off) {
                const int key0 = walk.begin + i * kTcKeys;
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    reg[j] = make_uint4(0, 0, 0, 0);
                    if (id[j] >= 0 && in_row)
                        reg[j] = __ldcs(reinterpret_cast<const uint4 *>(
                            base + id[j] * block + head_off + ((key0 + row_l + j * kPassRows) & in_block) * dim));
                }
            };
            auto scales = [&]() {
                mks = mvs = 0.0f;
                if (ct < 8 && mid >= 0) {
                    const long long s = static_cast<long long>(mid) * c.heads + walk.head;
                    mks = c.ks[s];
                    mvs = c.vs[s];
                }
            };
            auto store = [&](const uint4 (&reg)[kPer], uint8_t *tile) {
                const uint32_t base = smem_addr(tile) + (q_l >> 2) * 16384;
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int row = row_l + j * kPassRows;
                    const uint32_t w[4] = {reg[j].x, reg[j].y, reg[j].z, reg[j].w};
                    uint32_t h[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) codes_f16(w[i], h[2 * i], h[2 * i + 1]);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(base + swizzled(row, (q_l & 3) * 2 + i)),
                                     "r"(h[4 * i]), "r"(h[4 * i + 1]), "r"(h[4 * i + 2]), "r"(h[4 * i + 3])
                                     : "memory");
                }
            };
            if (tiles > 0) {
                ids(0);
                load(0, kr, c.k, c.k_block, khead);
                load(0, vr, c.v, c.v_block, vhead);
                scales();
            }
            for (int i = 0; i < tiles; ++i, ++it) {
                const int s = it & 1;
                const uint32_t parity = ((it >> 1) & 1) ^ 1;
                const bool bad = mid < 0;
                const float ks_now = mks, vs_now = mvs;
                if (i + 1 < tiles) ids(i + 1);
                if (it >= 2 && !tc_wait_warp(&sm.k_empty[s], parity, fail, timeouts)) goto out;
                store(kr, sm.k[s]);
                if (warp == 8) {
                    // (entry it % 4: tile it - 3's softmax is done before K of
                    // tile it may be written)
                    TcMeta &meta = sm.meta[it & 3];
                    const uint32_t valid = __ballot_sync(~0u, ct < 8 && !bad);
                    int e = ct < 8 && !bad ? scale_exp(vs_now) : kLeastExp;
                    const uint32_t sized = __ballot_sync(~0u, e > kLeastExp && e < 120);
                    int least = e;
#pragma unroll
                    for (int d = 1; d < 8; d <<= 1) {
                        e = max(e, __shfl_xor_sync(~0u, e, d));
                        least = min(least, __shfl_xor_sync(~0u, least, d));
                    }
                    if (ct < 8) meta.group[ct] = make_float4(ks_now, log2_fast(vs_now), 1.0f / vs_now, vs_now);
                    if (ct == 0) meta.tile = make_int4(static_cast<int>(valid), e, (valid & sized) == 0xffu, least);
                }
                smem_to_tensor_fence();
                mbar_arrive(&sm.k_full[s]);
                if (i + 1 < tiles) {
                    load(i + 1, kr, c.k, c.k_block, khead);
                    scales();
                }
                if (it >= 2 && !tc_wait_warp(&sm.v_empty[s], parity, fail, timeouts)) goto out;
                store(vr, sm.v[s]);
                smem_to_tensor_fence();
                mbar_arrive(&sm.v_full[s]);
                if (i + 1 < tiles) load(i + 1, vr, c.v, c.v_block, vhead);
            }
        }
    } else if (warp == 12) {
        // ---- the products: the warp goes together, one lane issues
        {
            const bool leader = elect_lane();
            constexpr uint32_t kDescS = mma_desc(kTcKeys, false), kDescO = mma_desc(DP, true);
            uint32_t it = 0, count[2] = {0, 0}, items[2] = {0, 0};
            while (walk.next(a, c, group, sm.run_steps)) {
                const int tiles = walk.tiles(), halves = walk.rows > kTcHalf ? 2 : 1;
                if (tiles == 0) continue;
                for (int i = 0; i <= tiles; ++i) {
                    const uint32_t t = it + i, s = t & 1, was = s ^ 1;
                    for (int h = 0; h < halves; ++h) {
                        if (i > 0) {
                            // O += P V of the tile before
                            if (h == 0 && !tc_wait_warp(&sm.v_full[was], ((t - 1) >> 1) & 1, fail, timeouts)) goto out;
                            if (!tc_wait_warp(&sm.p_full[h], count[h] & 1, fail, timeouts)) goto out;
                            ++count[h];
                            tc_fence_after();
                            const uint32_t v = smem_addr(sm.v[was]);
#pragma unroll
                            for (int n = 0; n < kTcKeys / 16; ++n)
#pragma unroll
                                for (int lo = 0; lo < kTerms; ++lo)
                                    tc_mma_ts(leader, tmem + kColO + h * 128, tmem + kColS + h * 128 + (n * kTerms + lo) * 8,
                                              smem_desc(v + n * 2048, 16384, 1024), kDescO, i > 1 || n > 0 || lo > 0);
                            if (h == halves - 1) tc_commit(leader, &sm.v_empty[was]);
                            if (i == tiles) tc_commit(leader, &sm.o_full[h]);
                        }
                        if (i < tiles) {
                            // S = Q K^T of this tile
                            if (h == 0 && !tc_wait_warp(&sm.k_full[s], (t >> 1) & 1, fail, timeouts)) goto out;
                            if (i == 0) {
                                if (!tc_wait_warp(&sm.q_full[h], items[h] & 1, fail, timeouts)) goto out;
                                ++items[h];
                            }
                            tc_fence_after();
                            const uint32_t k = smem_addr(sm.k[s]), q = smem_addr(sm.q[h]);
#pragma unroll
                            for (int n = 0; n < DP / 16; ++n) {
                                const uint32_t at = (n >> 2) * 16384 + (n & 3) * 32;
                                tc_mma_ss(leader, tmem + kColS + h * 128, smem_desc(q + at, 16, 1024), smem_desc(k + at, 16, 1024),
                                          kDescS, n > 0);
                            }
                            tc_commit(leader, &sm.s_full[h]);
                            if (h == halves - 1) tc_commit(leader, &sm.k_empty[s]);
                        }
                    }
                }
                it += tiles;
            }
        }
    } else if (warp < 8) {
        // ---- the softmax, a thread per row.  After a wait that ran out these
        // warps go on (every later wait fails at once), so that none of them is
        // missing at the barriers they share; the results are then void.
        unsigned *const counters = static_cast<unsigned *>(a.workspace);
        float *const partial = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kWorkspaceCounters);
        const int half = warp >> 2, hw = warp & 3, ht = tid & 127;  // half, warp and thread within it
        const uint32_t lanes = tmem + (static_cast<uint32_t>(hw * 32) << 16);
        const uint32_t scol = lanes + kColS + half * 128, ocol = lanes + kColO + half * 128;
        uint32_t it = 0, mine = 0, items = 0;  // tiles of all halves, of this one; its items
        while (walk.next(a, c, group, sm.run_steps)) {
            const int tiles = walk.tiles(), rows = min(kTcHalf, walk.rows - half * kTcHalf), row0 = walk.row0 + half * kTcHalf;
            if (rows <= 0) {
                it += tiles;
                continue;
            }
            // this thread's query: scaled by a power of two to a largest
            // magnitude in [2^12, 2^13), as in qr_kv_split.cuh
            const int row = row0 + ht, token = row / group, head = walk.head * group + (row - token * group), walk_q0 = walk.x.q0;
            // The warp's rows between global memory and the queries' tile, each
            // row by neighbouring lanes in 16-byte pieces: a thread reading its
            // own row would touch 32 lines with every instruction.
            auto rows_move = [&](bool in) {
                constexpr int kPieces = DP / 8, kAtOnce = 32 / kPieces;  // pieces of a row, rows per instruction
                const int i = lane % kPieces;
                const bool on = FULL || i * 8 < dim;
                auto place = [&](int u, const uint16_t *base, long long token_stride, long long head_stride) {
                    const int in_warp = u + lane / kPieces;
                    const long long tok = walk_q0 + __shfl_sync(~0u, token, in_warp), hd = __shfl_sync(~0u, head, in_warp);
                    return base + tok * token_stride + hd * head_stride + i * 8;
                };
                auto tile = [&](int u) {
                    return reinterpret_cast<uint4 *>(sm.q[half] + (i >> 3) * 16384 + swizzled(hw * 32 + u + lane / kPieces, i & 7));
                };
                auto there = [&](int u) { return hw * 32 + u + lane / kPieces < rows && on; };
                if (in) {
                    uint4 w[32 / kAtOnce];  // all on their way at once
#pragma unroll
                    for (int u = 0; u < 32; u += kAtOnce) {
                        const uint16_t *src = place(u, static_cast<const uint16_t *>(a.q), a.q_token, a.q_head);
                        w[u / kAtOnce] = make_uint4(0, 0, 0, 0);
                        if (there(u)) w[u / kAtOnce] = *reinterpret_cast<const uint4 *>(src);
                    }
#pragma unroll
                    for (int u = 0; u < 32; u += kAtOnce) *tile(u) = w[u / kAtOnce];
                } else {
#pragma unroll 4
                    for (int u = 0; u < 32; u += kAtOnce) {
                        const uint16_t *to = place(u, static_cast<uint16_t *>(a.out), a.out_token, a.out_head);
                        if (there(u)) *reinterpret_cast<uint4 *>(const_cast<uint16_t *>(to)) = *tile(u);
                    }
                }
                __syncwarp();
            };
            float row_scale = 0.0f;
            if (tiles > 0) {
                // (loops kept rolled here and below: code that runs once an item
                // comes through the instruction cache each time)
                rows_move(true);
                float amax = 0.0f;
#pragma unroll 2
                for (int i = 0; i < DP / 8; ++i) {
                    float f[8];
                    const uint4 w = *reinterpret_cast<const uint4 *>(sm.q[half] + (i >> 3) * 16384 + swizzled(ht, i & 7));
                    widen8<BF16>(w, f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(f[k]));
                }
                int e = 0;
                if (amax > 0.0f && amax < INFINITY) {
                    frexpf(amax, &e);
                    e -= 13;
                }
                const float down1 = pow2i(-(e / 2)) * (a.scale < 0.0f ? -1.0f : 1.0f), down2 = pow2i(-(e - e / 2));
                // (NaN for an infinite query, as in qr_kv_split.cuh)
                row_scale = amax < INFINITY ? ldexpf(fabsf(a.scale) * 1.4426950408889634f, e) : __uint_as_float(0x7fffffffu);
#pragma unroll 2
                for (int i = 0; i < DP / 8; ++i) {
                    float f[8];
                    uint4 *const at = reinterpret_cast<uint4 *>(sm.q[half] + (i >> 3) * 16384 + swizzled(ht, i & 7));
                    const uint4 w = *at;
                    widen8<BF16>(w, f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = f[k] * down1 * down2;
                    *at = make_uint4(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7]));
                }
                smem_to_tensor_fence();
                mbar_arrive(&sm.q_full[half]);
                __syncwarp();
            }
            const bool active = hw * 32 < rows;  // else no row of the warp is the item's
            const int pos = walk.p0 + token;
            const int row_end = a.causal ? min(walk.x.kv, pos + 1) : walk.x.kv;
            const int row_begin = a.window > 0 ? pos - a.window + 1 : 0;
            // keys that every row of the warp sees
            const int seen_end = __reduce_min_sync(~0u, row_end), seen_begin = __reduce_max_sync(~0u, row_begin);
            const int begin = walk.begin;
            float m = -INFINITY, l = 0.0f;
            int ve = kLeastExp;
            for (int i = 0; i < tiles; ++i, ++it, ++mine) {
                tc_wait(&sm.s_full[half], mine & 1, fail, timeouts);
                __syncwarp();
                tc_fence_after();
                // S is there, and with it the product before is done: O may be
                // rescaled, P written
                if (active) {
                    const TcMeta &meta = sm.meta[it & 3];
                    const int key0 = begin + i * kTcKeys;
                    const int4 tile = meta.tile;
                    float4 now4 = meta.group[0], next4 = meta.group[1];
                    const bool mask = !tile.z || key0 + kTcKeys > seen_end || key0 < seen_begin;
                    float top = -INFINITY;
                    int e;
                    if (!mask) {
                        // scales are not negative: a group's largest score is
                        // its largest product, scaled
                        e = tile.y;
                        uint32_t v[2][32];
                        tc_ld32(scol, v[0]);
                        float ks0 = now4.x, ks1 = next4.x;
#pragma unroll 1
                        for (int cc = 0; cc < 4; cc += 2) {
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int ahead = (cc + u + 1) & 3;
                                tc_wait_ld(v[u]);
                                // (past the last 32 the first ones again, unused)
                                tc_ld32(scol + ahead * 32, v[u ^ 1]);
                                const float f0 = row_scale * ks0, f1 = row_scale * ks1;
                                ks0 = meta.group[ahead * 2].x;
                                ks1 = meta.group[ahead * 2 + 1].x;
#pragma unroll
                                for (int gr = 0; gr < 2; ++gr) {
                                    const uint32_t *w = v[u] + gr * 16;
                                    float x[4];
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        x[k] = max3_nan(max_nan(__uint_as_float(w[4 * k]), __uint_as_float(w[4 * k + 1])),
                                                        __uint_as_float(w[4 * k + 2]), __uint_as_float(w[4 * k + 3]));
                                    const float y = max3_nan(max_nan(x[0], x[1]), x[2], x[3]);
                                    top = max_nan(top, y * (gr ? f1 : f0));
                                }
                            }
                        }
                        tc_wait_ld(v[0]);
                    } else {
                        e = kLeastExp;
#pragma unroll 1
                        for (int g8 = 0; g8 < 8; ++g8) {
                            uint32_t y[16];
                            tc_ld16(scol + g8 * 16, y);
                            tc_wait_ld(y);
                            const int key = key0 + g8 * 16;
                            const float4 scales = meta.group[g8];
                            if ((tile.x >> g8 & 1) && key < row_end && key + 16 > row_begin) {
                                float x = -INFINITY;
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    if (key + k < row_end && key + k >= row_begin) x = max_nan(x, __uint_as_float(y[k]));
                                top = max_nan(top, x * (row_scale * scales.x));
                                e = max(e, scale_exp(scales.w));
                            }
                            __syncwarp();
                        }
                    }
                    const bool grew = !(top <= m + kSlack) || e > ve + kScaleSlack;
                    if (__any_sync(~0u, grew)) {
                        const float m_new = grew ? max_nan(m, top) : m;
                        const int e_new = grew ? max(ve, e) : ve;
                        const float was = m_new == -INFINITY ? 0.0f : m - m_new;
                        const float fo = exp2_fast(was + static_cast<float>(ve - e_new));
                        l *= exp2_fast(was);
                        m = m_new;
                        ve = e_new;
                        if (i > 0) {
#pragma unroll 1
                            for (int cc = 0; cc < DP / 32; ++cc) {
                                uint32_t v[32];
                                tc_ld32(ocol + cc * 32, v);
                                tc_wait_ld(v);
#pragma unroll
                                for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * fo);
                                tc_st32(ocol + cc * 32, v);
                            }
                        }
                    }
                    const float base = m == -INFINITY ? 0.0f : -m;
                    uint32_t x[2][16];
                    tc_ld16(scol, x[0]);
                    // Weight: 2^(s f - m) w with w the values' scale under the
                    // row's power of two, taken in one exponent; a group's sum
                    // is then divided by w.  Not for scores so large that the
                    // fused product's unrounded part would matter, nor for value
                    // scales so far apart that the exponent would leave fp32's range.
                    const bool apart = ve - tile.w > kScaleSpan || ve > kMostScaleExp;
                    // (a row that is NaN does not count: it would change the others' bits)
                    if (!mask && !__any_sync(~0u, fabsf(m) >= 65536.0f || apart)) {
                        const float lift = base + static_cast<float>(kTcWeightExp - ve);
                        float sums = 0.0f;
                        auto exponents = [&](uint32_t (&y)[16], const float4 &scales) {
                            const float f = row_scale * scales.x, add = lift + scales.y;
#pragma unroll
                            for (int k = 0; k < 16; k += 2) {
                                const float2 z = fma2(make_float2(__uint_as_float(y[k]), __uint_as_float(y[k + 1])),
                                                      make_float2(f, f), make_float2(add, add));
                                y[k] = __float_as_uint(z.x);
                                y[k + 1] = __float_as_uint(z.y);
                            }
                        };
                        // a group at a time, the exponentials of the next one
                        // between the conversions and sums of this: one after
                        // the other they would each wait for their own latency
                        tc_wait_ld(x[0]);
                        tc_ld16(scol + 16, x[1]);
                        exponents(x[0], now4);
#pragma unroll
                        for (int k = 0; k < 16; ++k) x[0][k] = __float_as_uint(exp2_fast(__uint_as_float(x[0][k])));
#pragma unroll 1
                        for (int g0 = 0; g0 < 8; g0 += 2) {
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                // (past the last group the first ones again, unused:
                                // P of 16 keys takes no more than their 16 columns, all read before)
                                const int g8 = g0 + u;
                                uint32_t(&now)[16] = x[u], (&next)[16] = x[u ^ 1];
                                tc_wait_ld(next);
                                const float4 ahead4 = meta.group[(g8 + 2) & 7];
                                exponents(next, next4);
                                uint32_t p[kTerms][8];
                                float2 part[2];
#pragma unroll
                                for (int k = 0; k < 8; ++k) {
                                    const float2 y = make_float2(__uint_as_float(now[2 * k]), __uint_as_float(now[2 * k + 1]));
                                    next[2 * k] = __float_as_uint(exp2_fast(__uint_as_float(next[2 * k])));
                                    p[0][k] = pack_f16(y.x, y.y);
                                    p[1][k] = rest_f16(y, p[0][k]);
                                    next[2 * k + 1] = __float_as_uint(exp2_fast(__uint_as_float(next[2 * k + 1])));
                                    part[k & 1] = k < 2 ? y : add2(part[k & 1], y);
                                }
                                part[0] = add2(part[0], part[1]);
                                sums = __fmaf_rn(part[0].x + part[0].y, now4.z, sums);
                                now4 = next4;
                                next4 = ahead4;
                                tc_ld16(scol + ((g8 + 2) & 7) * 16, now);
#pragma unroll
                                for (int lo = 0; lo < kTerms; ++lo) tc_st8(scol + (g8 * kTerms + lo) * 8, p[lo]);
                            }
                        }
                        tc_wait_ld(x[1]);
                        l = __fmaf_rn(sums, pow2i(ve - kTcWeightExp), l);
                    } else {
                        const float up = pow2i(kTcWeightExp - ve);
#pragma unroll 1
                        for (int g8 = 0; g8 < 8; ++g8) {
                            const int key = key0 + g8 * 16;
                            const float4 scales = meta.group[g8];
                            const float f = row_scale * scales.x, vs = scales.w;
                            // (a group beyond the row's power of two is not seen by it)
                            const float w = scale_exp(vs) > ve + kScaleSlack ? 0.0f : vs * up;
                            const bool ok = tile.x >> g8 & 1;
                            uint32_t p[kTerms][8];
                            tc_wait_ld(x[0]);
#pragma unroll
                            for (int k = 0; k < 16; k += 2) {
                                float y[2];
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const float score = __uint_as_float(x[0][k + u]) * f;
                                    const bool sees = ok && key + k + u < row_end && key + k + u >= row_begin;
                                    y[u] = exp2_fast(sees ? score + base : -INFINITY);
                                    l += y[u];
                                }
                                const float2 z = make_float2(y[0] * w, y[1] * w);
                                p[0][k / 2] = pack_f16(z.x, z.y);
                                p[1][k / 2] = rest_f16(z, p[0][k / 2]);
                            }
#pragma unroll
                            for (int lo = 0; lo < kTerms; ++lo) tc_st8(scol + (g8 * kTerms + lo) * 8, p[lo]);
                            if (g8 < 7) tc_ld16(scol + (g8 + 1) * 16, x[0]);
                        }
                    }
                    tc_wait_st();
                }
                tc_fence_before();
                mbar_arrive(&sm.p_full[half]);
            }

            // the item's rows
            auto slot_of = [&](long long cta) { return 2 * cta + (walk.item_first > cta * walk.share ? 1 : 0); };
            auto part_of = [&](long long cta) { return partial + (slot_of(cta) * 2 + half) * kTcSlot<DP>; };
            float *const my_part = part_of(blockIdx.x);
            if (tiles > 0) {
                tc_wait(&sm.o_full[half], items & 1, fail, timeouts);
                ++items;
                __syncwarp();
                tc_fence_after();
            }
            // 32 of a row's values, 32 cc and on: to the tile for the output, or
            // to a part.  A part is [piece of four][row], so that a warp's rows
            // are neighbours in memory.
            const bool in_item = ht < rows;
            auto put = [&](float *part, int cc, const float (&y)[32], float inv) {
                if (part) {
                    if (in_item)
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            __stcg(reinterpret_cast<float4 *>(part + ((cc * 8 + k / 4) * kTcHalf + ht) * 4),
                                   make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]));
                } else {
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        const int i = cc * 4 + k / 8;
                        *reinterpret_cast<uint4 *>(sm.q[half] + (i >> 3) * 16384 + swizzled(ht, i & 7)) =
                            make_uint4(pack_out<BF16>(y[k] * inv, y[k + 1] * inv), pack_out<BF16>(y[k + 2] * inv, y[k + 3] * inv),
                                       pack_out<BF16>(y[k + 4] * inv, y[k + 5] * inv),
                                       pack_out<BF16>(y[k + 6] * inv, y[k + 7] * inv));
                    }
                }
            };
            // the row's maximum and sum, and the warp's rows out of the tile
            auto finish = [&](float *part, float top, float sum) {
                if (part) {
                    if (in_item) __stcg(reinterpret_cast<float2 *>(part + kTcHalf * DP + 2 * ht), make_float2(top, sum));
                    return;
                }
                if (in_item && a.lse)
                    a.lse[(walk_q0 + token) * static_cast<long long>(a.q_heads) + head] =
                        sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
                __syncwarp();
                rows_move(false);
            };
            if (active) {
                const float back = pow2i(ve - kTcWeightExp), inv = l == 0.0f ? 1.0f : 1.0f / l;
                float *const to = walk.parts > 1 ? my_part : nullptr;
#pragma unroll 1
                for (int cc = 0; cc < DP / 32; ++cc) {
                    uint32_t v[32];
                    if (tiles > 0) {
                        tc_ld32(ocol + cc * 32, v);
                        tc_wait_ld(v);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = 0;
                    }
                    float y[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(v[k]) * back;
                    put(to, cc, y, inv);
                }
                finish(to, m, l);
            }
            tc_fence_before();
            if (walk.parts > 1) {
                // as in qr_kv_split.cuh: groups of kGroup parts, then the groups,
                // each half for itself, a thread per row
                static_assert(kTcMostCtas <= kGroup * kGroup, "two levels");
                static_assert(2 * 4 * kTcMostCtas * 4 <= kWorkspaceCounters, "two counters per slot and half");
                const int groups = (walk.parts + kGroup - 1) / kGroup;
                const int my_group = (static_cast<int>(blockIdx.x) - walk.part_first_cta) / kGroup;
                int at_cta = walk.part_first_cta + my_group * kGroup;
                int count = min(kGroup, walk.parts - my_group * kGroup), stride = 1;
                unsigned *counter = counters + slot_of(at_cta) * 2 + half;
                for (int level = 0;; ++level) {
                    bar_half(half);
                    if (ht == 0) {
                        __threadfence();
                        sm.ticket[half] = atomicInc(counter, static_cast<unsigned>(count - 1));
                    }
                    bar_half(half);
                    if (sm.ticket[half] != static_cast<unsigned>(count - 1)) break;
                    __threadfence();
                    const bool last = level == 1 || groups == 1;
                    if (active) {
                        float top = -INFINITY, sum = 0.0f;
#pragma unroll 4
                        for (int k = 0; k < count; ++k) {
                            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(part_of(at_cta + k * stride) + kTcHalf * DP + 2 * ht));
                            const float next = max_nan(top, ml.x);
                            const float zero = next == -INFINITY ? 0.0f : next;
                            sum = __fmaf_rn(ml.y, exp2_fast(ml.x - zero), sum * exp2_fast(top - zero));
                            top = next;
                        }
                        const float zero = top == -INFINITY ? 0.0f : top, inv = sum == 0.0f ? 1.0f : 1.0f / sum;
                        float *const to = last ? nullptr : part_of(at_cta);
#pragma unroll 1
                        for (int cc = 0; cc < DP / 32; ++cc) {
                            float y[32];
#pragma unroll
                            for (int k = 0; k < 32; ++k) y[k] = 0.0f;
#pragma unroll 2
                            for (int k = 0; k < count; ++k) {
                                const float *const src = part_of(at_cta + k * stride);
                                const float f = exp2_fast(__ldcg(src + kTcHalf * DP + 2 * ht) - zero);
                                float4 w[8];
#pragma unroll
                                for (int u = 0; u < 8; ++u)
                                    w[u] = __ldcg(reinterpret_cast<const float4 *>(src + ((cc * 8 + u) * kTcHalf + ht) * 4));
#pragma unroll
                                for (int u = 0; u < 8; ++u) {
                                    y[4 * u] = __fmaf_rn(w[u].x, f, y[4 * u]), y[4 * u + 1] = __fmaf_rn(w[u].y, f, y[4 * u + 1]);
                                    y[4 * u + 2] = __fmaf_rn(w[u].z, f, y[4 * u + 2]), y[4 * u + 3] = __fmaf_rn(w[u].w, f, y[4 * u + 3]);
                                }
                            }
                            put(to, cc, y, inv);
                        }
                        finish(to, top, sum);
                    }
                    if (last) break;
                    counter = counters + 4 * kTcMostCtas + slot_of(walk.part_first_cta) * 2 + half;
                    at_cta = walk.part_first_cta;
                    count = groups;
                    stride = kGroup;
                }
            }
        }
    }
out:
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 12) tc_free(tmem, kColumns);
}

template <int DP, bool FULL, bool BF16>
cudaError_t run_kv_tc(const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s) {
    auto kern = kv_attention_tc_kernel<DP, FULL, BF16>;
    const int bytes = sizeof(TcSmem<DP>) + 1024;
    cudaError_t err = allow_dynamic_smem(reinterpret_cast<const void *>(kern), bytes);
    if (err != cudaSuccess) return err;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    unsigned *timeouts = wait_timeout_counter(&err);
    if (!timeouts) return err;
    return launch_chained(kern, static_cast<unsigned>(sms < kTcMostCtas ? sms : kTcMostCtas), kTcThreads, bytes, s, a, c,
                          group, timeouts);
}

}  // namespace qrk
