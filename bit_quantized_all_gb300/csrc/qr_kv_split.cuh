// qr_kv_split.cuh -- attention over the 8-bit paged cache, split over the keys.
//
// An item is 8 * NT query rows (a row is a query token and one of the group's
// heads) of one request and key/value head; its keys are counted in steps of
// kStep tokens.  All items' steps in a row are cut into equal shares, one per
// CTA, so the load is even whatever the lengths, and every CTA finds its
// share from the same sums over the requests: no host value depends on the
// lengths, and one launch does it all.  An item that lies within one share is
// written straight out; the CTAs of a divided one leave (max, sum,
// accumulators) in the workspace, and the CTA that brings its last part joins
// the parts in order, so the result does not depend on who comes last.
//
// Within a CTA each of four warps takes every fourth tile of 32 keys: copied
// by 16-byte asynchronous copies into the warp's own buffers, converted in
// registers to fp16 (exact for codes) and multiplied on m16n8k16 with the keys
// (then the values' dimensions) as M and the rows as N: a group of up to eight
// heads fills one instruction, and nothing is converted twice.  The order of
// the head's dimensions within a product is free, so a lane's sixteen
// consecutive code bytes of a key are the operands of four instructions, and
// its sixteen bytes of two value rows those of eight.  The weights reach the
// second product's operand order by an 8 x 8 transpose between registers.
// Scores are scaled by the block's scale in fp32.  The values' scale goes into
// the softmax weight before its rounding to fp16, relative to a power of two
// kept per row (the largest among the blocks that the row sees), so that the
// accumulators are the matrix instruction's own.  What that rounding left goes
// through a second product: a weight as one fp16 number is off by up to 2^-12,
// which showed in outputs of both types (0.001 of a bf16 output's norm away
// from a product in 32 bits, with both terms 0.0001; the error of fp16 outputs
// against 64 bits 1.6 times a 32-bit product's, with both the same).  It costs
// nothing where HBM bounds (128 requests of up to 8192 keys 187 and 186 us) and
// 12% where the products do (20 rows over 131075 keys 82 and 92 us).
//
// What bounds it: the codes from HBM when there is enough of them (128 single
// tokens over up to 8192 keys, 8 heads: 188 us, 5.8 TB/s, 0.86 of the copy
// rate); with more than eight rows an item latency, as two or three CTAs an SM
// are all that the accumulators' registers leave, and each warp waits for its
// own chain of copies, conversion, products and softmax (20 rows over 131075
// keys: 93 us, 2.9 TB/s); and below some 20 us the chain of dependent round
// trips: lengths, table, codes, parts, join (16 single tokens over up to 2048
// keys, one head: 12.0 us).
#pragma once

#include <type_traits>

#include "qr_kv_device.cuh"
#include "qr_launch.h"

namespace qrk {

constexpr int kAttnThreads = 128, kAttnWarps = 4;
constexpr int kTile = 32;                      // keys per warp and step of its loop
constexpr int kStep = kTile * kAttnWarps;
constexpr int kWeightExp = 12;                 // weights are at most 2^12: fp16 keeps 26 binades below them exact
constexpr int kMostCtas = 640;
constexpr int kWorkspaceCounters = 16 * kMostCtas;  // bytes: two slots per CTA, two counters per slot
constexpr int kGroup = 16;                     // parts of an item joined at a time
constexpr int kMostParts = kMostCtas / kGroup > kGroup ? kMostCtas / kGroup : kGroup;

// A request as the sums see it: keys [kv - len, kv) are visible to some query.
struct AttnRequest {
    int q0, nq, kv, len, items;
};

__device__ __forceinline__ AttnRequest attn_request(const KvAttentionArgs &a, const KvView &c, int rows, int group,
                                                    int r) {
    AttnRequest x;
    const int tokens = static_cast<int>(a.tokens);
    x.q0 = min(max(a.q_offsets[r], 0), tokens);
    x.nq = max(min(a.q_offsets[r + 1], tokens) - x.q0, 0);
    x.kv = max(0, min(a.kv_lens[r], a.width << c.shift));
    // with a window the first query's first key starts the request's keys
    const long long first = static_cast<long long>(x.kv) - x.nq - a.window + 1;
    x.len = a.window > 0 && first > 0 ? static_cast<int>(max(0LL, x.kv - first / kTile * kTile)) : x.kv;
    x.items = static_cast<int>((static_cast<long long>(x.nq) * group + rows - 1) / rows) * c.heads;
    return x;
}

// Steps of an item; one for an item that sees nothing, whose rows have to be
// written all the same.
__device__ __forceinline__ int attn_steps(int len) { return len > 0 ? (len - 1) / kStep + 1 : 1; }

template <int DP>
__device__ __forceinline__ uint32_t k_offset(int row, int chunk) {
    // the lanes of one 8-lane phase read pieces of two rows: odd rows swap halves
    return DP == 64 ? row * 64 + chunk * 16 : row * DP + ((chunk ^ ((row & 1) << 2)) << 4);
}
template <int DP>
__device__ __forceinline__ uint32_t v_offset(int row, int chunk) {
    // ... and of the values two pieces of four rows 2t
    const int s = ((row >> 1) & 3) << 1;
    return DP == 64 ? (row >> 1) * 128 + ((((row & 1) << 2 | chunk) ^ s) << 4) : row * DP + ((chunk ^ s) << 4);
}

template <int DP, int NT>
struct AttnSmem {
    static constexpr int kRows = 8 * NT;
    static constexpr int kHalf = kTile * DP;       // a tile's keys, or its values
    static constexpr int kRing = kAttnWarps * 2 * kHalf;
    static constexpr int kQ = kRows * DP * 2;      // fp16 fragments
    static constexpr int kOutStride = DP + 4;
    static constexpr int kMerge = kAttnWarps * kRows * (kOutStride + 2) * 4;
    static constexpr int kFirst = kRing > kMerge ? kRing : kMerge;
    static constexpr int kBytes = kFirst + kQ + kRows * 4;
    // CTAs per SM, by registers (accumulators: DP / 4 * NT / 2 a thread)
    static constexpr int kCtas = DP * NT <= 128 ? 4 : DP * NT <= 256 && NT <= 2 ? 3 : 2;
    static constexpr int kSlot = kRows * (DP + 2);  // floats of a part: accumulators, then (max, sum) pairs
};

// One row's 4 values from dimension d on, and with d = 0 its lse.
template <bool BF16>
__device__ __forceinline__ void attn_write(const KvAttentionArgs &a, int dim, long long token, int head, int d, float4 v,
                                           float top, float sum) {
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (d < dim) {
        uint16_t *out = static_cast<uint16_t *>(a.out) + token * a.out_token + head * a.out_head + d;
        uint2 w;
        if (BF16) {
            const __nv_bfloat162 b0 = __floats2bfloat162_rn(v.x * inv, v.y * inv);
            const __nv_bfloat162 b1 = __floats2bfloat162_rn(v.z * inv, v.w * inv);
            w.x = *reinterpret_cast<const uint32_t *>(&b0);
            w.y = *reinterpret_cast<const uint32_t *>(&b1);
        } else {
            w.x = pack_f16(v.x * inv, v.y * inv);
            w.y = pack_f16(v.z * inv, v.w * inv);
        }
        *reinterpret_cast<uint2 *>(out) = w;
    }
    if (a.lse && d == 0)
        a.lse[token * a.q_heads + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

// DP: the head's dimensions padded to 64, 128 or 256; FULL: they are exactly DP;
// BF16: the type of queries and output, otherwise fp16.
template <int DP, int NT, bool FULL, bool BF16>
__global__ void __launch_bounds__(kAttnThreads, AttnSmem<DP, NT>::kCtas)
    kv_attention_split_kernel(KvAttentionArgs a, KvView c, int group) {
    chain_entry();
    using S = AttnSmem<DP, NT>;
    constexpr int kRows = S::kRows, kSteps = DP / 16;
    constexpr int kDimTiles = DP / 16;                     // output tiles of 16 dimensions
    constexpr int kDims = DP == 64 ? 8 : 16;               // a lane's dimensions in a piece of a value row
    constexpr bool kQRegs = NT * DP <= 128;
    const int dim = FULL ? DP : c.dim;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long warp_sums[kAttnWarps];
    __shared__ long long run_steps[kAttnThreads];
    __shared__ AttnRequest run_request[kAttnThreads];  // each run's first request
    __shared__ unsigned s_ticket;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;

    // sums of steps over each thread's run of requests
    const int per = (a.requests + kAttnThreads - 1) / kAttnThreads;
    long long steps_all;
    {
        const int r0 = min(tid * per, a.requests), r1 = min(r0 + per, a.requests);
        long long steps = 0;
        for (int r = r0; r < r1; ++r) {
            const AttnRequest x = attn_request(a, c, kRows, group, r);
            if (r == r0) run_request[tid] = x;
            steps += static_cast<long long>(x.items) * attn_steps(x.len);
        }
        long long incl = steps;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(~0u, incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        long long before = 0;
        steps_all = 0;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            if (w < warp) before += warp_sums[w];
            steps_all += warp_sums[w];
        }
        run_steps[tid] = before + incl - steps;
        __syncthreads();
    }
    const long long share = (steps_all + gridDim.x - 1) / gridDim.x;
    const long long my_first = share * blockIdx.x, my_last = min(my_first + share, steps_all);

    unsigned *const counters = static_cast<unsigned *>(a.workspace);
    float *const partial = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kWorkspaceCounters);
    uint32_t *const q_frag = reinterpret_cast<uint32_t *>(smem + S::kFirst);
    float *const row_scale = reinterpret_cast<float *>(smem + S::kFirst + S::kQ);
    const uint32_t kaddr = smem_addr(smem + warp * (2 * S::kHalf)), vaddr = kaddr + S::kHalf;

    long long at = 0;  // first step of request r
    int r = -1;
    AttnRequest x;
    x.items = 0;
    int n_steps = 1;
    for (long long step = my_first; step < my_last;) {
        // the request of this step: by bisection over the runs, then along them
        if (r < 0) {
            int lo = 0, hi = kAttnThreads - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (run_steps[mid] <= step) lo = mid; else hi = mid - 1;
            }
            at = run_steps[lo];
            r = lo * per;
            x = run_request[lo];
            n_steps = attn_steps(x.len);
        }
        while (step >= at + static_cast<long long>(x.items) * n_steps) {
            at += static_cast<long long>(x.items) * n_steps;
            x = attn_request(a, c, kRows, group, ++r);
            n_steps = attn_steps(x.len);
        }
        const int item = static_cast<int>((step - at) / n_steps);
        const long long item_first = at + static_cast<long long>(item) * n_steps;
        const int s0 = static_cast<int>(step - item_first);
        const int s1 = static_cast<int>(min(item_first + n_steps, my_last) - item_first);
        // the CTAs that share the item: parts first_cta .. last_cta
        const long long first_cta = item_first / share, last_cta = (item_first + n_steps - 1) / share;
        const int parts = static_cast<int>(last_cta - first_cta) + 1;
        step = item_first + s1;

        const int h = item % c.heads, row0 = item / c.heads * kRows;
        const int rows_here = min(kRows, x.nq * group - row0);
        // positions of the item's first and last query
        const int p0 = x.kv - x.nq;
        const int pos_first = p0 + row0 / group, pos_last = p0 + (row0 + rows_here - 1) / group;
        int begin = x.kv - x.len + s0 * kStep;
        int end = static_cast<int>(min(static_cast<long long>(x.kv - x.len) + static_cast<long long>(s1) * kStep,
                                       static_cast<long long>(x.kv)));
        if (a.causal) end = min(end, pos_last + 1);
        if (a.window > 0 && pos_first - a.window + 1 > begin)
            begin += (pos_first - a.window + 1 - begin) / kTile * kTile;

        const int tiles = end > begin ? (end - begin + kTile - 1) / kTile : 0;
        const int mine = tiles > warp ? (tiles - warp + kAttnWarps - 1) / kAttnWarps : 0;
        // A lane holds one 16-key group's block and scales at a time: lane
        // 2 i + k the k-th group of the warp's tile 16 * batch + i.
        int id = -1;
        float ks = 0.0f, vs = 0.0f;
        auto look_up = [&](int first_tile) {
            const int i = first_tile + (lane >> 1);
            const int key = begin + (i * kAttnWarps + warp) * kTile + (lane & 1) * 16;
            id = -1;
            ks = vs = 0.0f;
            if (i < mine && key < end) {
                id = a.table[static_cast<long long>(r) * a.width + (key >> c.shift)];
                if (id < 0 || id >= c.blocks) {
                    id = -1;
                } else {
                    const long long s = static_cast<long long>(id) * c.heads + h;
                    ks = c.ks[s];
                    vs = c.vs[s];
                }
            }
        };
        const int in_block = (1 << c.shift) - 1;
        // Copies the keys (or the values) of the warp's i-th tile.
        auto issue = [&](int i, auto values) {
            constexpr bool kValues = decltype(values)::value;
            constexpr int kPer = DP / 16;  // 16-byte pieces of a padded row
            const int row_l = lane / kPer, q_l = lane % kPer;
            if (i < mine) {
                const int key = begin + (i * kAttnWarps + warp) * kTile;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int b = __shfl_sync(~0u, id, 2 * (i & 15) + k);
                    if (b >= 0 && (FULL || q_l * 16 < dim)) {
                        const int8_t *src = (kValues ? c.v + (b * c.v_block + h * c.v_head)
                                                     : c.k + (b * c.k_block + h * c.k_head)) +
                                            (((key + 16 * k) & in_block) + row_l) * dim + q_l * 16;
#pragma unroll
                        for (int j = 0; j < 16 * kPer / 32; ++j) {
                            const int row = j * (32 / kPer);
                            copy16_async(kValues ? vaddr + v_offset<DP>(16 * k + row + row_l, q_l)
                                                 : kaddr + k_offset<DP>(16 * k + row + row_l, q_l),
                                         src + row * dim);
                        }
                    }
                }
            }
            copy_commit();
        };
        constexpr std::false_type kKeysTag{};
        constexpr std::true_type kValuesTag{};

        // one buffer each for keys and values: a tile's keys are copied while
        // the one before is weighted and summed, its values while the next
        // tile's scores are taken; the first tile's while the queries are laid out
        __syncthreads();
        look_up(0);
        issue(0, kKeysTag);
        issue(0, kValuesTag);

        // the queries as fp16 fragments, each row scaled by a power of two to
        // a largest magnitude in [2^12, 2^13): exact for fp16 and bf16 inputs
        // down to 2^-26 of it, and the inverse goes into the score's factor.
        // A lane holds four dimensions (and four more, 128 on) of each of the
        // warp's rows; all rows are loaded before the first is waited for.
        constexpr int kQRows = kRows / kAttnWarps, kQFours = DP <= 128 ? 1 : DP / 128;
        uint2 raw[kQRows][kQFours];
#pragma unroll
        for (int n = 0; n < kQRows; ++n) {
            const int rr = warp + n * kAttnWarps, row = row0 + rr;
            const uint16_t *q = static_cast<const uint16_t *>(a.q) + (x.q0 + row / group) * a.q_token +
                                (static_cast<long long>(h) * group + row % group) * a.q_head;
#pragma unroll
            for (int i = 0; i < kQFours; ++i) {
                const int d = lane * 4 + i * 128;
                raw[n][i] = rr < rows_here && d < dim ? *reinterpret_cast<const uint2 *>(q + d) : make_uint2(0, 0);
            }
        }
#pragma unroll
        for (int n = 0; n < kQRows; ++n) {
            const int rr = warp + n * kAttnWarps;
            float f[kQFours][4], amax = 0.0f;
#pragma unroll
            for (int i = 0; i < kQFours; ++i)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t word = w < 2 ? raw[n][i].x : raw[n][i].y;
                    f[i][w] = widen1<BF16>(static_cast<uint16_t>(word >> (w & 1) * 16));
                    amax = fmaxf(amax, fabsf(f[i][w]));
                }
#pragma unroll
            for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
            // (a largest magnitude below 2^-126 is scaled as 2^-126 is)
            const int e = amax > 0.0f && amax < INFINITY ? max(static_cast<int>(__float_as_uint(amax) >> 23), 1) - 139 : 0;
            // 2^-e in two factors, as e may pass the range of one; a negative
            // scale's sign goes into the query, so that the factor is not negative
            const float down1 = pow2i(-(e / 2)) * (a.scale < 0.0f ? -1.0f : 1.0f), down2 = pow2i(-(e - e / 2));
            // (of an infinite query all scores could be -inf, as if it saw
            // nothing: its factor is NaN; one that is NaN has NaN products)
            if (lane == 0)
                row_scale[rr] = amax < INFINITY ? fabsf(a.scale) * 1.4426950408889634f * pow2i(e / 2) * pow2i(e - e / 2)
                                                : __uint_as_float(0x7fffffffu);
#pragma unroll
            for (int i = 0; i < kQFours; ++i) {
                // dimension d = 64 c + 16 t + 4 j + w is element w of lane
                // (row % 8, t) in step 4 c + j
                const int d = lane * 4 + i * 128;
                const int ks = (d >> 6) * 4 + ((d >> 2) & 3), ft = (d >> 4) & 3;
                uint2 y;
                y.x = pack_f16(f[i][0] * down1 * down2, f[i][1] * down1 * down2);
                y.y = pack_f16(f[i][2] * down1 * down2, f[i][3] * down1 * down2);
                if (d < DP) reinterpret_cast<uint2 *>(q_frag)[((rr >> 3) * kSteps + ks) * 32 + (rr & 7) * 4 + ft] = y;
            }
        }
        __syncthreads();
        uint32_t qf[kQRegs ? NT * kSteps : 1][2];
        if constexpr (kQRegs) {
#pragma unroll
            for (int i = 0; i < NT * kSteps; ++i)
                *reinterpret_cast<uint2 *>(qf[i]) = reinterpret_cast<const uint2 *>(q_frag)[i * 32 + lane];
        }
        // keys that every row sees: [seen_begin, seen_end); rows past the
        // item's are zero queries, whose sums are finite and not written
        const int seen_end = a.causal ? min(x.kv, pos_first + 1) : x.kv;
        const int seen_begin = a.window > 0 ? pos_last - a.window + 1 : 0;

        float o[NT][kDimTiles][4], m[NT][2], l[NT][2];
        int ve[NT][2];  // the row's power of two of the values' scales
#pragma unroll
        for (int q = 0; q < NT; ++q) {
#pragma unroll
            for (int j = 0; j < kDimTiles; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[q][j][k] = 0.0f;
            m[q][0] = m[q][1] = -INFINITY;
            l[q][0] = l[q][1] = 0.0f;
            ve[q][0] = ve[q][1] = kLeastExp;
        }

        for (int i = 0; i < mine; ++i) {
            float ks_cur[2], vs_cur[2];
            bool valid[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ks_cur[k] = __shfl_sync(~0u, ks, 2 * (i & 15) + k);
                vs_cur[k] = __shfl_sync(~0u, vs, 2 * (i & 15) + k);
                valid[k] = __shfl_sync(~0u, id, 2 * (i & 15) + k) >= 0;
            }
            const int key0 = begin + (i * kAttnWarps + warp) * kTile;
            copy_wait<1>();
            __syncwarp();

            // scores of 32 keys, as [key][row]
            float s[NT][2][4];
#pragma unroll
            for (int cc = 0; cc < DP / 64; ++cc) {
                uint32_t qv[kQRegs ? 1 : NT][4][2];
                if constexpr (!kQRegs) {
#pragma unroll
                    for (int q = 0; q < NT; ++q)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint2 *>(qv[q][j]) =
                                reinterpret_cast<const uint2 *>(q_frag)[(q * kSteps + cc * 4 + j) * 32 + lane];
                }
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) {
                    const uint4 lo = lds128(kaddr + k_offset<DP>(kt * 16 + g, cc * 4 + t));
                    const uint4 hi = lds128(kaddr + k_offset<DP>(kt * 16 + 8 + g, cc * 4 + t));
                    const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t ka[4];
                        codes_f16(lw[j], ka[0], ka[2]);
                        codes_f16(hw[j], ka[1], ka[3]);
#pragma unroll
                        for (int q = 0; q < NT; ++q) {
                            const uint32_t(&f)[2] = kQRegs ? qf[q * kSteps + cc * 4 + j] : qv[kQRegs ? 0 : q][j];
                            if (cc == 0 && j == 0)
                                mma_f16(s[q][kt], ka, f[0], f[1], 0.0f, 0.0f, 0.0f, 0.0f);
                            else
                                mma_f16_acc(s[q][kt], ka, f[0], f[1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (((i + 1) & 15) == 0) look_up(i + 1);
            issue(i + 1, kKeysTag);

            // running maximum and sum in powers of two; a tile that some row
            // does not see whole is masked first
            const bool mask = !valid[0] || !valid[1] || key0 + kTile > seen_end || key0 < seen_begin;
            const int vexp[2] = {scale_exp(vs_cur[0]), scale_exp(vs_cur[1])};
            uint32_t p[NT][2][2];     // B fragments of the two 16-key groups
            uint32_t lo_p[NT][2][2];  // what their rounding left
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                // (a score is rounded before the maximum is taken from it: of
                // scores of 2^30 a fused product would leave a remainder of 64)
                const float2 row = *reinterpret_cast<const float2 *>(row_scale + q * 8 + 2 * t);
                int e[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt) {
                        const float f = (k ? row.y : row.x) * ks_cur[kt];
                        s[q][kt][k] *= f;
                        s[q][kt][2 + k] *= f;
                    }
                    e[k] = max(vexp[0], vexp[1]);
                }
                if (mask) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int pos = p0 + (row0 + q * 8 + 2 * t + k) / group;
                        const int row_end = a.causal ? min(x.kv, pos + 1) : x.kv;
                        const int row_begin = a.window > 0 ? pos - a.window + 1 : 0;
                        e[k] = kLeastExp;
#pragma unroll
                        for (int kt = 0; kt < 2; ++kt) {
                            const int key = key0 + 16 * kt;
                            if (valid[kt] && key < row_end && key + 16 > row_begin) e[k] = max(e[k], vexp[kt]);
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int at_key = key + 8 * u + g;
                                if (!valid[kt] || at_key >= row_end || at_key < row_begin) s[q][kt][2 * u + k] = -INFINITY;
                            }
                        }
                    }
                }
                float mx[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    mx[k] = max_nan(max_nan(s[q][0][k], s[q][0][2 + k]), max_nan(s[q][1][k], s[q][1][2 + k]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx[k] = max_nan(mx[k], __shfl_xor_sync(~0u, mx[k], d));
                }
                const bool grew = !(mx[0] <= m[q][0]) || !(mx[1] <= m[q][1]) || e[0] > ve[q][0] || e[1] > ve[q][1];
                if (__any_sync(~0u, grew)) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float top = max_nan(m[q][k], mx[k]);
                        const float was = top == -INFINITY ? 0.0f : m[q][k] - top;
                        const int e_new = max(e[k], ve[q][k]);
                        l[q][k] *= exp2_fast(was);
                        const float fo = exp2_fast(was + static_cast<float>(ve[q][k] - e_new));
                        m[q][k] = top;
                        ve[q][k] = e_new;
#pragma unroll
                        for (int j = 0; j < kDimTiles; ++j) {
                            o[q][j][k] *= fo;
                            o[q][j][2 + k] *= fo;
                        }
                    }
                }
                float w[2][2], base[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    base[k] = m[q][k] == -INFINITY ? 0.0f : m[q][k];
                    const float up = pow2i(kWeightExp - ve[q][k]);
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt)
                        // (a group whose scale is above the row's power is not seen by it)
                        w[k][kt] = mask && vexp[kt] > ve[q][k] ? 0.0f : vs_cur[kt] * up;
                }
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) {
                    float y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        y[k] = exp2_fast(s[q][kt][k] - base[k & 1]);
                        l[q][k & 1] += y[k];
                        y[k] *= w[k & 1][kt];
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t hi = pack_f16(y[2 * u], y[2 * u + 1]);
                        p[q][kt][u] = transpose8(hi);
                        lo_p[q][kt][u] = transpose8(rest_f16(make_float2(y[2 * u], y[2 * u + 1]), hi));
                    }
                }
            }

            // values, as [dimension][row]
            copy_wait<1>();
            __syncwarp();
            constexpr int kPieces = DP == 64 ? 1 : DP / 128;
#pragma unroll
            for (int pc = 0; pc < kPieces; ++pc)
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) {
                    uint32_t vw[4][kDims / 4];  // rows 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                    for (int rr = 0; rr < 4; ++rr) {
                        const int row = 16 * kt + 2 * t + (rr & 1) + 8 * (rr >> 1);
                        if constexpr (DP == 64) {
                            const uint2 v2 = lds64(vaddr + v_offset<DP>(row, g >> 1) + (g & 1) * 8);
                            vw[rr][0] = v2.x, vw[rr][1] = v2.y;
                        } else {
                            const uint4 v4 = lds128(vaddr + v_offset<DP>(row, pc * 8 + g));
                            vw[rr][0] = v4.x, vw[rr][1] = v4.y, vw[rr][2] = v4.z, vw[rr][3] = v4.w;
                        }
                    }
#pragma unroll
                    for (int wd = 0; wd < kDims / 4; ++wd) {
                        uint32_t lo[4], hi[4];
                        codes_f16_pairs(vw[0][wd], vw[1][wd], lo);
                        codes_f16_pairs(vw[2][wd], vw[3][wd], hi);
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            // dimensions 2u and 2u + 1 of the word: the tile's rows g and g + 8
                            const uint32_t va[4] = {lo[2 * u], lo[2 * u + 1], hi[2 * u], hi[2 * u + 1]};
#pragma unroll
                            for (int q = 0; q < NT; ++q)
                                mma_f16_acc(o[q][pc * 8 + wd * 2 + u], va, p[q][kt][0], p[q][kt][1]);
#pragma unroll
                            for (int q = 0; q < NT; ++q)
                                mma_f16_acc(o[q][pc * 8 + wd * 2 + u], va, lo_p[q][kt][0], lo_p[q][kt][1]);
                        }
                    }
                }
            __syncwarp();
            issue(i + 1, kValuesTag);
        }
        copy_wait<0>();

        // join the four warps
        float *const merge_o = reinterpret_cast<float *>(smem);
        float *const merge_m = merge_o + kAttnWarps * kRows * S::kOutStride;
        float *const merge_l = merge_m + kAttnWarps * kRows;
        float *const merge_sum = merge_o + kRows * (kMostParts + 2);  // (when parts are joined)
        __syncthreads();
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float sum = l[q][k];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
                const int rr = warp * kRows + q * 8 + 2 * t + k;
                if (g == 0) {
                    merge_m[rr] = m[q][k];
                    merge_l[rr] = sum;
                }
                float *dst = merge_o + rr * S::kOutStride;
                const float back = pow2i(ve[q][k] - kWeightExp);
#pragma unroll
                for (int j = 0; j < kDimTiles; j += 2) {
                    // output tile j holds dimensions 2 (j % 8) and the next of
                    // the lane's piece
                    const int d = DP == 64 ? g * 8 + 2 * j : (j / 8) * 128 + g * 16 + 2 * (j % 8);
                    *reinterpret_cast<float4 *>(dst + d) = make_float4(o[q][j][k] * back, o[q][j][2 + k] * back,
                                                                       o[q][j + 1][k] * back, o[q][j + 1][2 + k] * back);
                }
            }
        __syncthreads();

        constexpr int kQuads = DP / 4;
        // a CTA holds parts of at most two divided items: the one that begins
        // its share, or began before it, and the one that it leaves unfinished
        auto slot_of = [&](long long cta) { return 2 * cta + (item_first > cta * share ? 1 : 0); };
        float *const my_slot = partial + slot_of(blockIdx.x) * S::kSlot;
        for (int i = tid; i < rows_here * kQuads; i += kAttnThreads) {
            const int rr = i / kQuads, d = i % kQuads * 4;
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) top = max_nan(top, merge_m[k * kRows + rr]);
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (top != -INFINITY) {
#pragma unroll
                for (int k = 0; k < kAttnWarps; ++k) {
                    const float f = exp2_fast(merge_m[k * kRows + rr] - top);
                    const float4 y = *reinterpret_cast<const float4 *>(merge_o + (k * kRows + rr) * S::kOutStride + d);
                    sum = __fmaf_rn(merge_l[k * kRows + rr], f, sum);
                    v.x = __fmaf_rn(y.x, f, v.x), v.y = __fmaf_rn(y.y, f, v.y);
                    v.z = __fmaf_rn(y.z, f, v.z), v.w = __fmaf_rn(y.w, f, v.w);
                }
            }
            if (parts == 1) {
                const int row = row0 + rr;
                attn_write<BF16>(a, dim, x.q0 + row / group, h * group + row % group, d, v, top, sum);
            } else {
                __stcg(reinterpret_cast<float4 *>(my_slot + rr * DP + d), v);
                if (d == 0) __stcg(reinterpret_cast<float2 *>(my_slot + kRows * DP + 2 * rr), make_float2(top, sum));
            }
        }
        if (parts > 1) {
            // In groups of kGroup parts, then the groups: whichever CTA brings the
            // last one joins them.  A counter wraps to 0 with its last arrival,
            // ready for the next call.
            const int groups = (parts + kGroup - 1) / kGroup;
            const int my_group = static_cast<int>(blockIdx.x - first_cta) / kGroup;
            long long at_cta = first_cta + my_group * kGroup;
            int count = min(kGroup, parts - my_group * kGroup), stride = 1;
            unsigned *counter = counters + slot_of(at_cta);
            for (int level = 0;; ++level) {
                __syncthreads();
                if (tid == 0) {
                    __threadfence();
                    s_ticket = atomicInc(counter, static_cast<unsigned>(count - 1));
                }
                __syncthreads();
                if (s_ticket != static_cast<unsigned>(count - 1)) break;
                __threadfence();
                // every row's maximum, sum and the parts' weights
                float *const weight = reinterpret_cast<float *>(smem);  // [row][part]
                float2 *const total = reinterpret_cast<float2 *>(weight + kRows * kMostParts);
                for (int i = tid; i < rows_here * count; i += kAttnThreads) {
                    const int rr = i / count, k = i % count;
                    const float *src = partial + slot_of(at_cta + k * stride) * S::kSlot + kRows * DP + 2 * rr;
                    const float2 ml = __ldcg(reinterpret_cast<const float2 *>(src));
                    weight[rr * kMostParts + k] = ml.x;
                    merge_sum[rr * kMostParts + k] = ml.y;
                }
                __syncthreads();
                if (tid < rows_here) {
                    float top = -INFINITY, sum = 0.0f;
                    for (int k = 0; k < count; ++k) top = max_nan(top, weight[tid * kMostParts + k]);
                    for (int k = 0; k < count; ++k) {
                        const float f = top == -INFINITY ? 0.0f : exp2_fast(weight[tid * kMostParts + k] - top);
                        sum = __fmaf_rn(merge_sum[tid * kMostParts + k], f, sum);
                        weight[tid * kMostParts + k] = f;
                    }
                    total[tid] = make_float2(top, sum);
                }
                __syncthreads();
                const bool last = level == 1 || groups == 1;
                float *const to = partial + slot_of(at_cta) * S::kSlot;
                // two pieces a thread at a time, eight parts of each on their way
                for (int i0 = tid; i0 < rows_here * kQuads; i0 += 2 * kAttnThreads) {
                    const int piece[2] = {i0, min(i0 + kAttnThreads, rows_here * kQuads - 1)};
                    float4 v[2];
                    v[0] = v[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
                    for (int k = 0; k < count; ++k) {
                        const float *const part = partial + slot_of(at_cta + k * stride) * S::kSlot;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float4 y = __ldcg(reinterpret_cast<const float4 *>(part + piece[u] * 4));
                            const float f = weight[piece[u] / kQuads * kMostParts + k];
                            v[u].x = __fmaf_rn(y.x, f, v[u].x), v[u].y = __fmaf_rn(y.y, f, v[u].y);
                            v[u].z = __fmaf_rn(y.z, f, v[u].z), v[u].w = __fmaf_rn(y.w, f, v[u].w);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int rr = piece[u] / kQuads, d = piece[u] % kQuads * 4, row = row0 + rr;
                        if (i0 + u * kAttnThreads >= rows_here * kQuads) break;
                        const float2 ts = total[rr];
                        if (last) {
                            attn_write<BF16>(a, dim, x.q0 + row / group, h * group + row % group, d, v[u], ts.x, ts.y);
                        } else {
                            __stcg(reinterpret_cast<float4 *>(to + rr * DP + d), v[u]);
                            if (d == 0) __stcg(reinterpret_cast<float2 *>(to + kRows * DP + 2 * rr), ts);
                        }
                    }
                }
                if (last) break;
                counter = counters + 2 * kMostCtas + slot_of(first_cta);
                at_cta = first_cta;
                count = groups;
                stride = kGroup;
            }
        }
    }
}

template <int DP, int NT, bool FULL, bool BF16>
cudaError_t run_kv_split(const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s) {
    using S = AttnSmem<DP, NT>;
    auto kern = kv_attention_split_kernel<DP, NT, FULL, BF16>;
    cudaError_t err = allow_dynamic_smem(reinterpret_cast<const void *>(kern), S::kBytes);
    if (err != cudaSuccess) return err;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    // no more CTAs than there can be steps
    const long long by_tokens = a.tokens * group / (8 * NT) + a.requests;
    const long long by_requests = ((static_cast<long long>(a.max_q) * group + 8 * NT - 1) / (8 * NT)) * a.requests;
    const long long items = (by_tokens < by_requests ? by_tokens : by_requests) * c.heads;
    const long long most = items * (((static_cast<long long>(a.width) << c.shift) + kStep - 1) / kStep);
    long long grid = static_cast<long long>(sms) * S::kCtas;
    grid = grid > kMostCtas ? kMostCtas : grid;
    return launch_chained(kern, static_cast<unsigned>(most < grid ? most : grid), kAttnThreads, S::kBytes, s, a, c,
                          group);
}

template <int DP, int NT, bool BF16>
cudaError_t run_kv_split(const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s) {
    return c.dim == DP ? run_kv_split<DP, NT, true, BF16>(a, c, group, s) : run_kv_split<DP, NT, false, BF16>(a, c, group, s);
}

// As few column tiles as hold the rows: 20 rows over 131075 keys take 91 us as
// three and 116 as four.  Above 128 dimensions the accumulators leave room for
// two, and more rows are more items.
template <bool BF16>
cudaError_t pick_kv_split(const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s) {
    const long long rows = static_cast<long long>(a.max_q) * group;
    if (c.dim <= 64)
        return rows <= 8    ? run_kv_split<64, 1, BF16>(a, c, group, s)
               : rows <= 16 ? run_kv_split<64, 2, BF16>(a, c, group, s)
               : rows <= 24 ? run_kv_split<64, 3, BF16>(a, c, group, s)
                            : run_kv_split<64, 4, BF16>(a, c, group, s);
    if (c.dim <= 128)
        return rows <= 8    ? run_kv_split<128, 1, BF16>(a, c, group, s)
               : rows <= 16 ? run_kv_split<128, 2, BF16>(a, c, group, s)
               : rows <= 24 ? run_kv_split<128, 3, BF16>(a, c, group, s)
                            : run_kv_split<128, 4, BF16>(a, c, group, s);
    return rows <= 8 ? run_kv_split<256, 1, BF16>(a, c, group, s) : run_kv_split<256, 2, BF16>(a, c, group, s);
}

}  // namespace qrk
