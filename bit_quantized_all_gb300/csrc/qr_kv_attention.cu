// qr_kv_attention.cu -- attention over the 8-bit paged cache
// (qr_kv_attention).
//
// Split over the keys.  An item is 16 * MT query rows (a row is a query token
// and one of the group's heads) of one request and key/value head; its keys
// are cut into chunks of C tokens, and a CTA takes one (item, chunk) at a
// time.  C comes from the lengths on the device, so that all items together
// make about kTargetUnits chunks whatever the batch: every CTA takes the same
// sums over the requests, no host value depends on the lengths and no launch
// but this one is needed.  An item of one chunk is written straight out; the
// others leave (max, sum, accumulators) in the workspace, and the CTA that
// brings an item's last chunk joins them in chunk order, so the result does
// not depend on who comes last.
//
// Within a CTA each of four warps takes every fourth tile of 32 keys: copied
// by 16-byte asynchronous copies into the warp's own ring, converted in
// registers to fp16 (exact for codes) and multiplied on m16n8k16.  The order
// of the head's dimensions within a product is free, so a lane's sixteen
// consecutive code bytes of a key are the operands of four instructions, and
// its sixteen bytes of two value rows those of sixteen.  Scores are scaled by
// the block's scale in fp32; the product with the values is accumulated for
// one block scale at a time and then added scaled, so no code is ever
// rounded.
//
// What bounds it: the bytes of the cache.  A tile of 32 keys (8 KB at 128
// dimensions) costs a warp about 700 instructions at MT = 1, half of what the
// SM can issue while HBM delivers the tile.
#include "qr_kv_device.cuh"
#include "qr_launch.h"

namespace qrk {

constexpr int kAttnThreads = 128, kAttnWarps = 4;
constexpr int kTile = 32;           // keys per warp and step
constexpr int kStages = 2;
constexpr int kTargetUnits = 608;   // chunks aimed at: two per resident CTA
constexpr int kMinChunk = kTile * kAttnWarps;
constexpr int kMostSlots = 2 * kTargetUnits;  // an item of several chunks has len > C, so at most twice the target

constexpr int kWorkspaceCounters = 8192;      // bytes: one counter per slot

struct AttnShape {
    int rows;       // rows per item: 16 * MT
    int group;      // query heads per key/value head
};

// A request as the sums see it.
struct AttnRequest {
    int q0, nq, kv, len, items;  // keys visible to it are [kv - len, kv) or fewer
};

__device__ __forceinline__ AttnRequest attn_request(const KvAttentionArgs &a, const KvView &c, int rows, int group, int r) {
    AttnRequest x;
    const int tokens = static_cast<int>(a.tokens);
    x.q0 = min(max(a.q_offsets[r], 0), tokens);
    x.nq = max(min(a.q_offsets[r + 1], tokens) - x.q0, 0);
    const int most = a.width << c.shift;
    x.kv = max(0, min(a.kv_lens[r], most));
    // with a window the first query's first key starts the request's keys
    const long long first = static_cast<long long>(x.kv) - x.nq - a.window + 1;
    x.len = a.window > 0 && first > 0 ? static_cast<int>(max(0LL, x.kv - first / kTile * kTile)) : x.kv;
    x.items = static_cast<int>((static_cast<long long>(x.nq) * group + rows - 1) / rows) * c.heads;
    return x;
}

// Chunks of an item over `len` keys; one for an item that sees nothing, whose
// rows have to be written all the same.
__device__ __forceinline__ int attn_chunks(int len, long long chunk) {
    return len > 0 ? static_cast<int>((len - 1) / chunk) + 1 : 1;
}

// Exclusive sum of `v` over the CTA's threads and the total.
__device__ __forceinline__ long long block_scan(long long v, long long *total, long long *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(~0u, incl, d);
        if (lane >= d) incl += o;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *total = all;
    return before + incl - v;
}

__device__ __forceinline__ float widen1(bool bf16, uint16_t u) {
    return bf16 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u));
}

template <int DP>
__device__ __forceinline__ uint32_t k_offset(int row, int chunk) {
    // lanes of one 8-lane phase read two rows' halves: odd rows swap theirs
    return DP == 64 ? row * 64 + chunk * 16 : row * DP + ((chunk ^ ((row & 1) << 2)) << 4);
}
template <int DP>
__device__ __forceinline__ uint32_t v_offset(int row, int chunk) {
    // ... and of the values two 16-byte pieces of four rows 2t
    const int s = ((row >> 1) & 3) << 1;
    return DP == 64 ? (row >> 1) * 128 + ((((row & 1) << 2 | chunk) ^ s) << 4) : row * DP + ((chunk ^ s) << 4);
}

// One item's rows over one range of keys, by one warp.
template <int DP, int MT>
struct AttnWarp {
    static constexpr int kSteps = DP / 16;   // products per score tile
    static constexpr int kOut = DP / 8;      // output tiles of 8 dimensions
    float o[MT][kOut][4];
    float m[MT][2], l[MT][2];
};

template <int DP, int MT>
struct AttnSmem {
    static constexpr int kStage = 2 * kTile * DP;                    // keys, values
    static constexpr int kRing = kAttnWarps * kStages * kStage;
    static constexpr int kQ = 16 * MT * DP * 2;                      // fp16 fragments
    static constexpr int kOutStride = DP + 4;
    static constexpr int kMerge = kAttnWarps * 16 * MT * (kOutStride + 2) * 4;
    static constexpr int kBytes = (kRing > kMerge ? kRing : kMerge) + kQ + 16 * MT * 4;
};

template <int DP, int MT>
__global__ void __launch_bounds__(kAttnThreads, DP * MT <= 128 ? 3 : 2)
    kv_attention_split_kernel(KvAttentionArgs a, KvView c, bool bf16, int group) {
    chain_entry();
    using S = AttnSmem<DP, MT>;
    constexpr int kRows = 16 * MT, kSteps = DP / 16, kOut = DP / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long warp_sums[kAttnWarps];
    __shared__ long long run_units[kAttnThreads], run_slots[kAttnThreads];
    __shared__ unsigned s_ticket;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;

    // the chunk length and every thread's run of requests
    const int per = (a.requests + kAttnThreads - 1) / kAttnThreads;
    const int r0 = min(tid * per, a.requests), r1 = min(r0 + per, a.requests);
    long long total = 0, units_all, slots_all;
    for (int r = r0; r < r1; ++r) {
        const AttnRequest x = attn_request(a, c, kRows, group, r);
        total += static_cast<long long>(x.items) * x.len;
    }
    block_scan(total, &total, warp_sums);
    const long long want = (total + kTargetUnits - 1) / kTargetUnits;
    const long long chunk = max(static_cast<long long>(kMinChunk), (want + kMinChunk - 1) / kMinChunk * kMinChunk);
    long long units = 0, slots = 0;
    for (int r = r0; r < r1; ++r) {
        const AttnRequest x = attn_request(a, c, kRows, group, r);
        const long long n = attn_chunks(x.len, chunk);
        units += x.items * n;
        slots += n > 1 ? x.items * n : 0;
    }
    const long long units_before = block_scan(units, &units_all, warp_sums);
    const long long slots_before = block_scan(slots, &slots_all, warp_sums);
    run_units[tid] = units_before;
    run_slots[tid] = slots_before;
    __syncthreads();

    unsigned *const counters = static_cast<unsigned *>(a.workspace);
    float *const partial = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kWorkspaceCounters);
    constexpr int kSlot = kRows * (DP + 2);  // floats: rows x DP accumulators, then max and sum per row

    uint8_t *const ring = smem + warp * (kStages * S::kStage);
    uint32_t *const q_frag = reinterpret_cast<uint32_t *>(smem + (S::kRing > S::kMerge ? S::kRing : S::kMerge));
    float *const row_scale = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(q_frag) + S::kQ);
    const uint32_t ring_addr = smem_addr(ring);

    for (long long unit = blockIdx.x; unit < units_all; unit += gridDim.x) {
        // the unit's request: its run by bisection, then along the run
        int lo = 0, hi = kAttnThreads - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (run_units[mid] <= unit) lo = mid; else hi = mid - 1;
        }
        long long at = run_units[lo], slot = run_slots[lo];
        int r = lo * per, n;
        AttnRequest x;
        for (;; ++r) {
            x = attn_request(a, c, kRows, group, r);
            n = attn_chunks(x.len, chunk);
            const long long here = static_cast<long long>(x.items) * n;
            if (unit < at + here) break;
            at += here;
            slot += n > 1 ? here : 0;
        }
        const int in = static_cast<int>(unit - at);
        const int part = in % n, item = in / n;
        const int h = item % c.heads, row0 = item / c.heads * kRows;
        slot += static_cast<long long>(item) * n;
        const int rows_here = min(kRows, x.nq * group - row0);
        // positions of the item's first and last query
        const long long p0 = static_cast<long long>(x.kv) - x.nq;
        const long long pos_first = p0 + row0 / group, pos_last = p0 + (row0 + rows_here - 1) / group;
        long long begin = x.kv - x.len + static_cast<long long>(part) * chunk;
        long long end = min(begin + chunk, static_cast<long long>(x.kv));
        if (a.causal) end = min(end, pos_last + 1);
        if (a.window > 0) begin = max(begin, (pos_first - a.window + 1) / kTile * kTile);

        // the queries as fp16 fragments, each row scaled by a power of two to
        // a largest magnitude in [2^12, 2^13): exact for fp16 and bf16 inputs
        // down to 2^-26 of it, and the inverse goes into the score's factor
        __syncthreads();
        for (int rr = warp; rr < kRows; rr += kAttnWarps) {
            const bool in_row = rr < rows_here;
            const int row = row0 + rr;
            const uint16_t *q = static_cast<const uint16_t *>(a.q) + (x.q0 + row / group) * a.q_token +
                                (static_cast<long long>(h) * group + row % group) * a.q_head;
            float f[DP / 32], amax = 0.0f;
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                const int d = lane + 32 * i;
                f[i] = in_row && d < c.dim ? widen1(bf16, q[d]) : 0.0f;
                amax = fmaxf(amax, fabsf(f[i]));
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
            // 2^e with amax * 2^-e in [2^12, 2^13); two factors, as e may pass
            // the range of one
            int e = 0;
            if (amax > 0.0f && amax < INFINITY) {
                frexpf(amax, &e);
                e -= 13;
            }
            const float down1 = exp2f(static_cast<float>(-(e / 2))), down2 = exp2f(static_cast<float>(-(e - e / 2)));
            if (lane == 0)
                row_scale[rr] = ldexpf(a.scale * 1.4426950408889634f, e);
            __half *frag = reinterpret_cast<__half *>(q_frag);
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                const int d = lane + 32 * i;
                // dimension d = 64 c + 16 t + 4 j + w is element w of lane
                // (row, t) in step 4 c + j: fragment register (row >= 8) + 2 (w / 2)
                const int step = (d >> 6) * 4 + ((d >> 2) & 3), ft = (d >> 4) & 3, w = d & 3;
                const int tile = rr >> 4, fr = rr & 15;
                frag[(((tile * kSteps + step) * 32 + (fr & 7) * 4 + ft) * 4 + (fr >> 3) + 2 * (w >> 1)) * 2 + (w & 1)] =
                    __float2half_rn(f[i] * down1 * down2);
            }
        }
        __syncthreads();
        uint32_t qf[MT * DP <= 128 ? MT * kSteps : 1][4];
        if constexpr (MT * DP <= 128) {
#pragma unroll
            for (int i = 0; i < MT * kSteps; ++i)
                *reinterpret_cast<uint4 *>(qf[i]) = reinterpret_cast<const uint4 *>(q_frag)[i * 32 + lane];
        }
        float factor[MT][2];
        int row_end[MT][2], row_begin[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int rr = i * 16 + g + 8 * k;
                factor[i][k] = row_scale[rr];
                const long long pos = p0 + (row0 + rr) / group;
                long long e = x.kv, b = 0;
                if (a.causal) e = min(e, pos + 1);
                if (a.window > 0) b = max(b, pos - a.window + 1);
                row_end[i][k] = rr < rows_here ? static_cast<int>(max(e, 0LL)) : 0;
                row_begin[i][k] = static_cast<int>(min(b, static_cast<long long>(x.kv)));
            }
        // keys that every row sees: [seen_begin, seen_end)
        const long long seen_end = a.causal ? min(static_cast<long long>(x.kv), pos_first + 1) : x.kv;
        const long long seen_begin = a.window > 0 ? pos_last - a.window + 1 : 0;
        const bool partial_rows = rows_here < kRows;

        AttnWarp<DP, MT> w;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int j = 0; j < kOut; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) w.o[i][j][k] = 0.0f;
            w.m[i][0] = w.m[i][1] = -INFINITY;
            w.l[i][0] = w.l[i][1] = 0.0f;
        }

        const int tiles = end > begin ? static_cast<int>((end - begin + kTile - 1) / kTile) : 0;
        const int mine = tiles > warp ? (tiles - warp + kAttnWarps - 1) / kAttnWarps : 0;
        // A lane holds one 16-key group's block and scales at a time: lane
        // 2 i + k the k-th group of the warp's tile 16 * batch + i.
        int id = -1;
        float ks = 0.0f, vs = 0.0f;
        auto look_up = [&](int batch) {
            const int i = batch * 16 + (lane >> 1);
            const long long key = begin + (static_cast<long long>(i) * kAttnWarps + warp) * kTile + (lane & 1) * 16;
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
            const int slot_i = i % kStages;
            const uint32_t dst = ring_addr + slot_i * S::kStage;
            const long long key = begin + (static_cast<long long>(i) * kAttnWarps + warp) * kTile;
            const int vec = c.dim >> 4;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int b = __shfl_sync(~0u, id, 2 * (i & 15) + k);
                if (b >= 0) {
                    const long long off = ((key + 16 * k) & in_block) * c.dim;
                    const int8_t *kp = c.k + b * c.k_block + h * c.k_head + off;
                    const int8_t *vp = c.v + b * c.v_block + h * c.v_head + off;
                    constexpr int kPer = DP / 16;  // 16-byte pieces of a padded row
#pragma unroll
                    for (int j = 0; j < 16 * kPer / 32; ++j) {
                        const int p = j * 32 + lane, row = p / kPer, q = p % kPer;
                        if (q < vec) {
                            copy16_async(dst + k_offset<DP>(16 * k + row, q), kp + row * c.dim + q * 16);
                            copy16_async(dst + kTile * DP + v_offset<DP>(16 * k + row, q), vp + row * c.dim + q * 16);
                        }
                    }
                }
            }
            copy_commit();
        };

        float ks_cur[2], vs_cur[2];
        bool bad_cur;
        look_up(0);
        if (mine > 0) issue(0);
        for (int i = 0; i < mine; ++i) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ks_cur[k] = __shfl_sync(~0u, ks, 2 * (i & 15) + k);
                vs_cur[k] = __shfl_sync(~0u, vs, 2 * (i & 15) + k);
            }
            bad_cur = __shfl_sync(~0u, id, 2 * (i & 15)) < 0 || __shfl_sync(~0u, id, 2 * (i & 15) + 1) < 0;
            const int valid = (__shfl_sync(~0u, id, 2 * (i & 15)) >= 0 ? 1 : 0) |
                              (__shfl_sync(~0u, id, 2 * (i & 15) + 1) >= 0 ? 2 : 0);
            if (i + 1 < mine) {
                if (((i + 1) & 15) == 0) look_up((i + 1) >> 4);
                issue(i + 1);
                copy_wait<1>();
            } else {
                copy_wait<0>();
            }
            __syncwarp();
            const uint32_t kaddr = ring_addr + (i % kStages) * S::kStage, vaddr = kaddr + kTile * DP;
            const long long key0 = begin + (static_cast<long long>(i) * kAttnWarps + warp) * kTile;

            // scores of 32 keys
            float s[MT][4][4];
#pragma unroll
            for (int q = 0; q < MT; ++q)
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[q][nt][k] = 0.0f;
#pragma unroll
            for (int cc = 0; cc < DP / 64; ++cc) {
                uint4 qv[MT][4];
                if constexpr (MT * DP > 128) {
#pragma unroll
                    for (int q = 0; q < MT; ++q)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            qv[q][j] = reinterpret_cast<const uint4 *>(q_frag)[(q * kSteps + cc * 4 + j) * 32 + lane];
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
                            if constexpr (MT * DP <= 128) {
                                const uint32_t *f = qf[q * kSteps + cc * 4 + j];
                                mma_f16(s[q][nt], f[0], f[1], f[2], f[3], b0, b1);
                            } else {
                                mma_f16(s[q][nt], qv[q][j].x, qv[q][j].y, qv[q][j].z, qv[q][j].w, b0, b1);
                            }
                        }
                    }
                }
            }

            // scale, mask, running maximum and sum (in powers of two)
            const bool mask = partial_rows || bad_cur || key0 + kTile > seen_end || key0 < seen_begin;
            uint32_t p[MT][4][2];
#pragma unroll
            for (int q = 0; q < MT; ++q) {
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float v = s[q][nt][k] * (factor[q][k >> 1] * ks_cur[nt >> 1]);
                        if (mask) {
                            const long long key = key0 + nt * 8 + 2 * t + (k & 1);
                            if (key >= row_end[q][k >> 1] || key < row_begin[q][k >> 1] || !(valid & (1 << (nt >> 1))))
                                v = -INFINITY;
                        }
                        s[q][nt][k] = v;
                        mx[k >> 1] = max_nan(mx[k >> 1], v);
                    }
                float base[2];
                bool grew = false;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    mx[k] = max_nan(mx[k], __shfl_xor_sync(~0u, mx[k], 1));
                    mx[k] = max_nan(mx[k], __shfl_xor_sync(~0u, mx[k], 2));
                    grew |= !(mx[k] <= w.m[q][k]);
                }
                if (__any_sync(~0u, grew)) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float top = max_nan(w.m[q][k], mx[k]);
                        const float f = top == -INFINITY ? 1.0f : exp2_fast(w.m[q][k] - top);
                        w.m[q][k] = top;
                        w.l[q][k] *= f;
#pragma unroll
                        for (int j = 0; j < kOut; ++j) {
                            w.o[q][j][2 * k] *= f;
                            w.o[q][j][2 * k + 1] *= f;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) base[k] = w.m[q][k] == -INFINITY ? 0.0f : w.m[q][k];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    float e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        e[k] = exp2_fast(s[q][nt][k] - base[k >> 1]);
                        w.l[q][k >> 1] += e[k];
                    }
                    p[q][nt][0] = pack_f16(e[0], e[1]);
                    p[q][nt][1] = pack_f16(e[2], e[3]);
                }
            }

            // values: one block scale at a time
            const bool one = vs_cur[0] == vs_cur[1];
            constexpr int kPieces = DP == 64 ? 1 : DP / 128;  // 16- or 8-byte pieces of a value row per lane
            constexpr int kDims = DP == 64 ? 8 : 16;
#pragma unroll
            for (int pc = 0; pc < kPieces; ++pc) {
                uint32_t vw[2][4][4];  // group, row 2t / 2t+1 / 2t+8 / 2t+9, words
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int rr = 0; rr < 4; ++rr) {
                        const int row = 16 * k + 2 * t + (rr & 1) + 8 * (rr >> 1);
                        if constexpr (DP == 64) {
                            const uint2 v2 = lds64(vaddr + v_offset<DP>(row, g >> 1) + (g & 1) * 8);
                            vw[k][rr][0] = v2.x;
                            vw[k][rr][1] = v2.y;
                        } else {
                            const uint4 v4 = lds128(vaddr + v_offset<DP>(row, pc * 8 + g));
                            vw[k][rr][0] = v4.x, vw[k][rr][1] = v4.y, vw[k][rr][2] = v4.z, vw[k][rr][3] = v4.w;
                        }
                    }
#pragma unroll
                for (int wd = 0; wd < kDims / 4; ++wd) {
                    uint32_t b0[2][4], b1[2][4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        codes_f16_pairs(vw[k][0][wd], vw[k][1][wd], b0[k]);
                        codes_f16_pairs(vw[k][2][wd], vw[k][3][wd], b1[k]);
                    }
#pragma unroll
                    for (int q = 0; q < MT; ++q)
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            float *o = w.o[q][pc * 16 + wd * 4 + d];
                            float tmp[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma_f16(tmp, p[q][0][0], p[q][0][1], p[q][1][0], p[q][1][1], b0[0][d], b1[0][d]);
                            if (!one) {
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    o[k] = __fmaf_rn(tmp[k], vs_cur[0], o[k]);
                                    tmp[k] = 0.0f;
                                }
                            }
                            mma_f16(tmp, p[q][2][0], p[q][2][1], p[q][3][0], p[q][3][1], b0[1][d], b1[1][d]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) o[k] = __fmaf_rn(tmp[k], vs_cur[1], o[k]);
                        }
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
                float l = w.l[q][k];
                l += __shfl_xor_sync(~0u, l, 1);
                l += __shfl_xor_sync(~0u, l, 2);
                const int rr = warp * kRows + q * 16 + g + 8 * k;
                if (t == 0) {
                    merge_m[rr] = w.m[q][k];
                    merge_l[rr] = l;
                }
                float *dst = merge_o + rr * S::kOutStride;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    // column 2t + half of output tile j is dimension j % kDims
                    // of piece 2t + half
                    constexpr int kDims = DP == 64 ? 8 : 16;
#pragma unroll
                    for (int j = 0; j < kOut; j += 4) {
                        const int d = (j / kDims) * 128 + (2 * t + half) * kDims + j % kDims;
                        *reinterpret_cast<float4 *>(dst + d) =
                            make_float4(w.o[q][j][2 * k + half], w.o[q][j + 1][2 * k + half],
                                        w.o[q][j + 2][2 * k + half], w.o[q][j + 3][2 * k + half]);
                    }
                }
            }
        __syncthreads();

        auto write_out = [&](int rr, int d, float4 v, float top, float sum) {
            // a row's 4 values from dimension d on, and its lse
            const int row = row0 + rr;
            const long long token = x.q0 + row / group;
            const int head = h * group + row % group;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            if (d < c.dim) {
                uint16_t *out = static_cast<uint16_t *>(a.out) + token * a.out_token + head * a.out_head + d;
                uint32_t lo, hi;
                if (bf16) {
                    const __nv_bfloat162 b0 = __floats2bfloat162_rn(v.x * inv, v.y * inv);
                    const __nv_bfloat162 b1 = __floats2bfloat162_rn(v.z * inv, v.w * inv);
                    lo = *reinterpret_cast<const uint32_t *>(&b0);
                    hi = *reinterpret_cast<const uint32_t *>(&b1);
                } else {
                    lo = pack_f16(v.x * inv, v.y * inv);
                    hi = pack_f16(v.z * inv, v.w * inv);
                }
                *reinterpret_cast<uint2 *>(out) = make_uint2(lo, hi);
            }
            if (a.lse && d == 0)
                a.lse[token * a.q_heads + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
        };

        constexpr int kQuads = DP / 4;
        float *const my_slot = partial + slot * kSlot;
        for (int i = tid; i < rows_here * kQuads; i += kAttnThreads) {
            const int rr = i / kQuads, d = i % kQuads * 4;
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) top = max_nan(top, merge_m[k * kRows + rr]);
            float sum = 0.0f;
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
            if (n == 1) {
                write_out(rr, d, v, top, sum);
            } else {
                float *dst = my_slot + static_cast<long long>(part) * kSlot;
                __stcg(reinterpret_cast<float4 *>(dst + rr * DP + d), v);
                if (d == 0) __stcg(reinterpret_cast<float2 *>(dst + kRows * DP + 2 * rr), make_float2(top, sum));
            }
        }
        if (n > 1) {
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                // wraps to 0 with the item's last chunk: ready for the next call
                s_ticket = atomicInc(counters + slot, static_cast<unsigned>(n - 1));
            }
            __syncthreads();
            if (s_ticket == static_cast<unsigned>(n - 1)) {
                __threadfence();
                for (int i = tid; i < rows_here * kQuads; i += kAttnThreads) {
                    const int rr = i / kQuads, d = i % kQuads * 4;
                    float top = -INFINITY, sum = 0.0f;
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                    for (int k = 0; k < n; ++k) {
                        const float *src = my_slot + static_cast<long long>(k) * kSlot;
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(src + kRows * DP + 2 * rr));
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(src + rr * DP + d));
                        if (ml.x == -INFINITY) continue;
                        const float next = max_nan(top, ml.x);
                        const float f0 = exp2_fast(top - next), f1 = exp2_fast(ml.x - next);
                        top = next;
                        sum = __fmaf_rn(ml.y, f1, sum * f0);
                        v.x = __fmaf_rn(y.x, f1, v.x * f0), v.y = __fmaf_rn(y.y, f1, v.y * f0);
                        v.z = __fmaf_rn(y.z, f1, v.z * f0), v.w = __fmaf_rn(y.w, f1, v.w * f0);
                    }
                    write_out(rr, d, v, top, sum);
                }
            }
        }
    }
}

size_t kv_attention_workspace(int, long long, int, int, int head_dim) {
    const size_t dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    return kWorkspaceCounters + size_t(kMostSlots) * (dp <= 128 ? 32 : 16) * (dp + 2) * 4;
}

template <int DP, int MT>
static cudaError_t run_split(int dtype, const KvAttentionArgs &a, const KvView &c, int group, cudaStream_t s) {
    using S = AttnSmem<DP, MT>;
    auto kern = kv_attention_split_kernel<DP, MT>;
    cudaError_t err = allow_dynamic_smem(reinterpret_cast<const void *>(kern), S::kBytes);
    if (err != cudaSuccess) return err;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    // no more CTAs than there can be chunks
    const long long items = (a.tokens * group / (16 * MT) + a.requests) * c.heads;
    const long long most = items * (((static_cast<long long>(a.width) << c.shift) + kMinChunk - 1) / kMinChunk);
    const long long resident = static_cast<long long>(sms) * (DP * MT <= 128 ? 3 : 2);
    return launch_chained(kern, static_cast<unsigned>(most < resident ? most : resident), kAttnThreads, S::kBytes, s, a,
                          c, dtype != 0, group);
}

cudaError_t launch_kv_attention(int dtype, const KvAttentionArgs &a, const qr_kv_cache_t &cache, cudaStream_t s) {
    const KvView c = kv_view(cache);
    const int group = a.q_heads / c.heads;
    const bool one = static_cast<long long>(a.max_q) * group <= 16;
    if (c.dim <= 64) return one ? run_split<64, 1>(dtype, a, c, group, s) : run_split<64, 2>(dtype, a, c, group, s);
    if (c.dim <= 128) return one ? run_split<128, 1>(dtype, a, c, group, s) : run_split<128, 2>(dtype, a, c, group, s);
    return run_split<256, 1>(dtype, a, c, group, s);
}

}  // namespace qrk
