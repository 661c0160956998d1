// qr_kv_split.cuh -- attention over the 8-bit paged cache, split over the keys.
//
// An item is 16 * MT query rows (a row is a query token and one of the group's
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
// by 16-byte asynchronous copies into the warp's own ring, converted in
// registers to fp16 (exact for codes) and multiplied on m16n8k16.  The order
// of the head's dimensions within a product is free, so a lane's sixteen
// consecutive code bytes of a key are the operands of four instructions, and
// its sixteen bytes of two value rows those of sixteen.  Scores are scaled by
// the block's scale in fp32.  The values' scale goes into the softmax weight
// before its rounding to fp16, relative to a power of two kept per row (the
// largest among the blocks that the row sees), so that the accumulators are
// the matrix instruction's own.
#pragma once

#include "qr_kv_device.cuh"
#include "qr_launch.h"

namespace qrk {

constexpr int kAttnThreads = 128, kAttnWarps = 4;
constexpr int kTile = 32;                      // keys per warp and step of its loop
constexpr int kStages = 2;
constexpr int kStep = kTile * kAttnWarps;
constexpr int kWeightExp = 12;                 // weights are at most 2^12: fp16 keeps 26 binades below them exact
constexpr int kWorkspaceCounters = 4096;       // bytes: one counter per slot, two slots per CTA
constexpr int kMostCtas = kWorkspaceCounters / 8;

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

__device__ __forceinline__ float widen1(bool bf16, uint16_t u) {
    return bf16 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u));
}

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

template <int DP, int MT>
struct AttnSmem {
    static constexpr int kStage = 2 * kTile * DP;  // keys, values
    static constexpr int kRing = kAttnWarps * kStages * kStage;
    static constexpr int kQ = 16 * MT * DP * 2;    // fp16 fragments
    static constexpr int kOutStride = DP + 4;
    static constexpr int kMerge = kAttnWarps * 16 * MT * (kOutStride + 2) * 4;
    static constexpr int kFirst = kRing > kMerge ? kRing : kMerge;
    static constexpr int kBytes = kFirst + kQ + 16 * MT * 4;
    static constexpr int kCtas = DP <= 128 && MT == 1 ? 3 : 2;  // per SM, by registers and shared memory
    static constexpr int kSlot = 16 * MT * (DP + 2);          // floats of a part: accumulators, then (max, sum) pairs
};

// One row's 4 values from dimension d on, and with d = 0 its lse.
__device__ __forceinline__ void attn_write(const KvAttentionArgs &a, bool bf16, int dim, long long token, int head,
                                           int d, float4 v, float top, float sum) {
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (d < dim) {
        uint16_t *out = static_cast<uint16_t *>(a.out) + token * a.out_token + head * a.out_head + d;
        uint2 w;
        if (bf16) {
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

// DP: the head's dimensions padded to 64, 128 or 256; FULL: they are exactly DP.
template <int DP, int MT, bool FULL>
__global__ void __launch_bounds__(kAttnThreads, AttnSmem<DP, MT>::kCtas)
    kv_attention_split_kernel(KvAttentionArgs a, KvView c, bool bf16, int group) {
    chain_entry();
    using S = AttnSmem<DP, MT>;
    constexpr int kRows = 16 * MT, kSteps = DP / 16, kOut = DP / 8;
    constexpr bool kQRegs = MT * DP <= 128;
    const int dim = FULL ? DP : c.dim;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long warp_sums[kAttnWarps];
    __shared__ long long run_steps[kAttnThreads];
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
    const uint32_t ring_addr = smem_addr(smem + warp * (kStages * S::kStage));

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
            x = attn_request(a, c, kRows, group, r);
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

        // the queries as fp16 fragments, each row scaled by a power of two to
        // a largest magnitude in [2^12, 2^13): exact for fp16 and bf16 inputs
        // down to 2^-26 of it, and the inverse goes into the score's factor
        __syncthreads();
        for (int rr = warp; rr < kRows; rr += kAttnWarps) {
            const int row = row0 + rr;
            const uint16_t *q = static_cast<const uint16_t *>(a.q) + (x.q0 + row / group) * a.q_token +
                                (static_cast<long long>(h) * group + row % group) * a.q_head;
            float f[DP / 32], amax = 0.0f;
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                const int d = lane + 32 * i;
                f[i] = rr < rows_here && d < dim ? widen1(bf16, q[d]) : 0.0f;
                amax = fmaxf(amax, fabsf(f[i]));
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
            int e = 0;
            if (amax > 0.0f && amax < INFINITY) {
                frexpf(amax, &e);
                e -= 13;
            }
            // 2^-e in two factors, as e may pass the range of one; a negative
            // scale's sign goes into the query, so that the factor is not negative
            const float down1 = pow2i(-(e / 2)) * (a.scale < 0.0f ? -1.0f : 1.0f), down2 = pow2i(-(e - e / 2));
            if (lane == 0) row_scale[rr] = ldexpf(fabsf(a.scale) * 1.4426950408889634f, e);
            __half *frag = reinterpret_cast<__half *>(q_frag);
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                // dimension d = 64 c + 16 t + 4 j + w is element w of lane
                // (row, t) in step 4 c + j: fragment register (row >= 8) + 2 (w / 2)
                const int d = lane + 32 * i;
                const int ks = (d >> 6) * 4 + ((d >> 2) & 3), ft = (d >> 4) & 3, w = d & 3;
                const int tile = rr >> 4, fr = rr & 15;
                frag[(((tile * kSteps + ks) * 32 + (fr & 7) * 4 + ft) * 4 + (fr >> 3) + 2 * (w >> 1)) * 2 + (w & 1)] =
                    __float2half_rn(f[i] * down1 * down2);
            }
        }
        __syncthreads();
        uint32_t qf[kQRegs ? MT * kSteps : 1][4];
        if constexpr (kQRegs) {
#pragma unroll
            for (int i = 0; i < MT * kSteps; ++i)
                *reinterpret_cast<uint4 *>(qf[i]) = reinterpret_cast<const uint4 *>(q_frag)[i * 32 + lane];
        }
        // keys that every row sees: [seen_begin, seen_end); rows past the
        // item's are zero queries, whose sums are finite and not written
        const int seen_end = a.causal ? min(x.kv, pos_first + 1) : x.kv;
        const int seen_begin = a.window > 0 ? pos_last - a.window + 1 : 0;

        float o[MT][kOut][4], m[MT][2], l[MT][2];
        int ve[MT][2];  // the row's power of two of the values' scales
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int j = 0; j < kOut; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][j][k] = 0.0f;
            m[i][0] = m[i][1] = -INFINITY;
            l[i][0] = l[i][1] = 0.0f;
            ve[i][0] = ve[i][1] = kLeastExp;
        }

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
        auto issue = [&](int i) {
            const uint32_t dst = ring_addr + (i % kStages) * S::kStage;
            const int key = begin + (i * kAttnWarps + warp) * kTile;
            constexpr int kPer = DP / 16;  // 16-byte pieces of a padded row
            const int row_l = lane / kPer, q_l = lane % kPer;  // this lane's piece, for DP <= 512
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int b = __shfl_sync(~0u, id, 2 * (i & 15) + k);
                if (b >= 0 && (FULL || q_l * 16 < dim)) {
                    const long long off = ((key + 16 * k) & in_block) * dim + row_l * dim + q_l * 16;
                    const int8_t *kp = c.k + (b * c.k_block + h * c.k_head + off);
                    const int8_t *vp = c.v + (b * c.v_block + h * c.v_head + off);
#pragma unroll
                    for (int j = 0; j < 16 * kPer / 32; ++j) {
                        const int row = j * (32 / kPer);
                        copy16_async(dst + k_offset<DP>(16 * k + row + row_l, q_l), kp + row * dim);
                        copy16_async(dst + kTile * DP + v_offset<DP>(16 * k + row + row_l, q_l), vp + row * dim);
                    }
                }
            }
            copy_commit();
        };

        look_up(0);
        if (mine > 0) issue(0);
        for (int i = 0; i < mine; ++i) {
            float ks_cur[2], vs_cur[2];
            bool valid[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ks_cur[k] = __shfl_sync(~0u, ks, 2 * (i & 15) + k);
                vs_cur[k] = __shfl_sync(~0u, vs, 2 * (i & 15) + k);
                valid[k] = __shfl_sync(~0u, id, 2 * (i & 15) + k) >= 0;
            }
            if (i + 1 < mine) {
                if (((i + 1) & 15) == 0) look_up(i + 1);
                issue(i + 1);
                copy_wait<1>();
            } else {
                copy_wait<0>();
            }
            __syncwarp();
            const uint32_t kaddr = ring_addr + (i % kStages) * S::kStage, vaddr = kaddr + kTile * DP;
            const int key0 = begin + (i * kAttnWarps + warp) * kTile;

            // scores of 32 keys
            float s[MT][4][4];
#pragma unroll
            for (int cc = 0; cc < DP / 64; ++cc) {
                uint32_t qv[kQRegs ? 1 : MT][4][4];
                if constexpr (!kQRegs) {
#pragma unroll
                    for (int q = 0; q < MT; ++q)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint4 *>(qv[q][j]) =
                                reinterpret_cast<const uint4 *>(q_frag)[(q * kSteps + cc * 4 + j) * 32 + lane];
                }
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const uint4 kv4 = lds128(kaddr + k_offset<DP>(nt * 8 + g, cc * 4 + t));
                    const uint32_t kw[4] = {kv4.x, kv4.y, kv4.z, kv4.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t b0, b1;
                        codes_f16(kw[j], b0, b1);
#pragma unroll
                        for (int q = 0; q < MT; ++q) {
                            const uint32_t(&f)[4] = kQRegs ? qf[q * kSteps + cc * 4 + j] : qv[kQRegs ? 0 : q][j];
                            if (cc == 0 && j == 0)
                                mma_f16(s[q][nt], f, b0, b1, 0.0f, 0.0f, 0.0f, 0.0f);
                            else
                                mma_f16_acc(s[q][nt], f, b0, b1);
                        }
                    }
                }
            }

            // running maximum and sum in powers of two; a tile that some row
            // does not see whole is scaled and masked first
            const bool mask = !valid[0] || !valid[1] || key0 + kTile > seen_end || key0 < seen_begin;
            const int e0 = scale_exp(vs_cur[0]), e1 = scale_exp(vs_cur[1]);
            uint32_t p[MT][2][4];  // A fragments of the two 16-key groups
#pragma unroll
            for (int q = 0; q < MT; ++q) {
                float f[2][2];
                int e[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float row = row_scale[q * 16 + g + 8 * k];
                    f[k][0] = row * ks_cur[0];
                    f[k][1] = row * ks_cur[1];
                    e[k] = max(e0, e1);
                }
                if (mask) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int rr = q * 16 + g + 8 * k, pos = p0 + (row0 + rr) / group;
                        const int row_end = a.causal ? min(x.kv, pos + 1) : x.kv;
                        const int row_begin = a.window > 0 ? pos - a.window + 1 : 0;
                        e[k] = kLeastExp;
#pragma unroll
                        for (int gr = 0; gr < 2; ++gr) {
                            const int key = key0 + 16 * gr;
                            if (valid[gr] && key < row_end && key + 16 > row_begin) e[k] = max(e[k], gr ? e1 : e0);
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int col = key + 8 * (u >> 1) + 2 * t + (u & 1);
                                float &v = s[q][2 * gr + (u >> 1)][2 * k + (u & 1)];
                                v = valid[gr] && col < row_end && col >= row_begin ? v * f[k][gr] : -INFINITY;
                            }
                        }
                        f[k][0] = f[k][1] = 1.0f;
                    }
                }
                float w0[2], w1[2], base[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float a0 = max_nan(max_nan(s[q][0][2 * k], s[q][0][2 * k + 1]),
                                             max_nan(s[q][1][2 * k], s[q][1][2 * k + 1]));
                    const float a1 = max_nan(max_nan(s[q][2][2 * k], s[q][2][2 * k + 1]),
                                             max_nan(s[q][3][2 * k], s[q][3][2 * k + 1]));
                    float mx = max_nan(a0 * f[k][0], a1 * f[k][1]);
                    mx = max_nan(mx, __shfl_xor_sync(~0u, mx, 1));
                    mx = max_nan(mx, __shfl_xor_sync(~0u, mx, 2));
                    base[k] = mx;
                }
                const bool grew = !(base[0] <= m[q][0]) || !(base[1] <= m[q][1]) || e[0] > ve[q][0] || e[1] > ve[q][1];
                if (__any_sync(~0u, grew)) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float top = max_nan(m[q][k], base[k]);
                        const float was = top == -INFINITY ? 0.0f : m[q][k] - top;
                        const int e_new = max(e[k], ve[q][k]);
                        l[q][k] *= exp2_fast(was);
                        const float fo = exp2_fast(was + static_cast<float>(ve[q][k] - e_new));
                        m[q][k] = top;
                        ve[q][k] = e_new;
#pragma unroll
                        for (int j = 0; j < kOut; ++j) {
                            o[q][j][2 * k] *= fo;
                            o[q][j][2 * k + 1] *= fo;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    base[k] = m[q][k] == -INFINITY ? 0.0f : -m[q][k];
                    const float up = pow2i(kWeightExp - ve[q][k]);
                    w0[k] = vs_cur[0] * up;
                    w1[k] = vs_cur[1] * up;
                    if (mask && e0 > ve[q][k]) w0[k] = 0.0f;  // a group that the row does not see
                    if (mask && e1 > ve[q][k]) w1[k] = 0.0f;
                }
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    float y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        y[k] = exp2_fast(__fmaf_rn(s[q][nt][k], f[k >> 1][nt >> 1], base[k >> 1]));
                        l[q][k >> 1] += y[k];
                        y[k] *= nt < 2 ? w0[k >> 1] : w1[k >> 1];
                    }
                    p[q][nt >> 1][2 * (nt & 1)] = pack_f16(y[0], y[1]);
                    p[q][nt >> 1][2 * (nt & 1) + 1] = pack_f16(y[2], y[3]);
                }
            }

            constexpr int kPieces = DP == 64 ? 1 : DP / 128;  // 16- or 8-byte pieces of a value row per lane
            constexpr int kWords = DP == 64 ? 2 : 4;
#pragma unroll
            for (int pc = 0; pc < kPieces; ++pc)
#pragma unroll
                for (int gr = 0; gr < 2; ++gr) {
                    uint32_t vw[4][4];  // rows 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                    for (int rr = 0; rr < 4; ++rr) {
                        const int row = 16 * gr + 2 * t + (rr & 1) + 8 * (rr >> 1);
                        if constexpr (DP == 64) {
                            const uint2 v2 = lds64(vaddr + v_offset<DP>(row, g >> 1) + (g & 1) * 8);
                            vw[rr][0] = v2.x, vw[rr][1] = v2.y;
                        } else {
                            const uint4 v4 = lds128(vaddr + v_offset<DP>(row, pc * 8 + g));
                            vw[rr][0] = v4.x, vw[rr][1] = v4.y, vw[rr][2] = v4.z, vw[rr][3] = v4.w;
                        }
                    }
#pragma unroll
                    for (int wd = 0; wd < kWords; ++wd) {
                        uint32_t b0[4], b1[4];
                        codes_f16_pairs(vw[0][wd], vw[1][wd], b0);
                        codes_f16_pairs(vw[2][wd], vw[3][wd], b1);
#pragma unroll
                        for (int q = 0; q < MT; ++q)
#pragma unroll
                            for (int d = 0; d < 4; ++d) mma_f16_acc(o[q][pc * 16 + wd * 4 + d], p[q][gr], b0[d], b1[d]);
                    }
                }
            __syncwarp();
        }

        // join the four warps
        float *const merge_o = reinterpret_cast<float *>(smem);
        float *const merge_m = merge_o + kAttnWarps * kRows * S::kOutStride;
        float *const merge_l = merge_m + kAttnWarps * kRows;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < MT; ++q)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float sum = l[q][k];
                sum += __shfl_xor_sync(~0u, sum, 1);
                sum += __shfl_xor_sync(~0u, sum, 2);
                const int rr = warp * kRows + q * 16 + g + 8 * k;
                if (t == 0) {
                    merge_m[rr] = m[q][k];
                    merge_l[rr] = sum;
                }
                float *dst = merge_o + rr * S::kOutStride;
                const float back = pow2i(min(ve[q][k] - kWeightExp, 127));
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    // column 2t + half of output tile j is dimension j % kDims
                    // of piece 2t + half
                    constexpr int kDims = DP == 64 ? 8 : 16;
#pragma unroll
                    for (int j = 0; j < kOut; j += 4) {
                        const int d = (j / kDims) * 128 + (2 * t + half) * kDims + j % kDims, u = 2 * k + half;
                        *reinterpret_cast<float4 *>(dst + d) =
                            make_float4(o[q][j][u] * back, o[q][j + 1][u] * back, o[q][j + 2][u] * back, o[q][j + 3][u] * back);
                    }
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
                attn_write(a, bf16, dim, x.q0 + row / group, h * group + row % group, d, v, top, sum);
            } else {
                __stcg(reinterpret_cast<float4 *>(my_slot + rr * DP + d), v);
                if (d == 0) __stcg(reinterpret_cast<float2 *>(my_slot + kRows * DP + 2 * rr), make_float2(top, sum));
            }
        }
        if (parts > 1) {
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                // wraps to 0 with the item's last part: ready for the next call
                s_ticket = atomicInc(counters + slot_of(first_cta), static_cast<unsigned>(parts - 1));
            }
            __syncthreads();
            if (s_ticket == static_cast<unsigned>(parts - 1)) {
                __threadfence();
                for (int i = tid; i < rows_here * kQuads; i += kAttnThreads) {
                    const int rr = i / kQuads, d = i % kQuads * 4, row = row0 + rr;
                    float top = -INFINITY, sum = 0.0f;
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
                    for (int k = 0; k < parts; ++k) {
                        const float *src = partial + slot_of(first_cta + k) * S::kSlot;
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(src + kRows * DP + 2 * rr));
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(src + rr * DP + d));
                        const float next = max_nan(top, ml.x);
                        const float base = next == -INFINITY ? 0.0f : next;
                        const float f0 = exp2_fast(top - base), f1 = exp2_fast(ml.x - base);
                        top = next;
                        sum = __fmaf_rn(ml.y, f1, sum * f0);
                        v.x = __fmaf_rn(y.x, f1, v.x * f0), v.y = __fmaf_rn(y.y, f1, v.y * f0);
                        v.z = __fmaf_rn(y.z, f1, v.z * f0), v.w = __fmaf_rn(y.w, f1, v.w * f0);
                    }
                    attn_write(a, bf16, dim, x.q0 + row / group, h * group + row % group, d, v, top, sum);
                }
            }
        }
    }
}

template <int DP, int MT, bool FULL>
cudaError_t run_kv_split(int dtype, const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s) {
    using S = AttnSmem<DP, MT>;
    auto kern = kv_attention_split_kernel<DP, MT, FULL>;
    cudaError_t err = allow_dynamic_smem(reinterpret_cast<const void *>(kern), S::kBytes);
    if (err != cudaSuccess) return err;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    // no more CTAs than there can be steps
    const long long items = (a.tokens * group / (16 * MT) + a.requests) * c.heads;
    const long long most = items * (((static_cast<long long>(a.width) << c.shift) + kStep - 1) / kStep);
    long long grid = static_cast<long long>(sms) * S::kCtas;
    grid = grid > kMostCtas ? kMostCtas : grid;
    return launch_chained(kern, static_cast<unsigned>(most < grid ? most : grid), kAttnThreads, S::kBytes, s, a, c,
                          dtype != 0, group);
}

}  // namespace qrk
