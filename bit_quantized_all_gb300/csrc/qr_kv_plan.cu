// qr_kv_plan.cu -- block tables and slots of a serving step from the
// requests' lengths (qr_kv_plan).
//
// One launch.  A CTA owns a range of the new tokens.  It goes over the
// requests kChunk at a time, eight per thread, takes the exclusive sums of
// their new tokens and newly needed blocks, keeps them in shared memory, and
// writes the slots of its tokens among them, finding each token's request by
// bisection.  A token that begins a block which the request did not hold also
// enters that block in the request's table row, so no CTA waits for another's
// result: a slot's block is either an entry that was there before the call or
// one of free_blocks, never one written here.  Every CTA takes the same sums:
// reading the lengths again costs less than a second launch or a flag.
#include <climits>

#include "qr_device.cuh"
#include "qr_launch.h"
#include "qr_serving.h"

namespace qrk {

constexpr int kPlanThreads = 256;
constexpr int kEach = 8;                         // requests per thread and chunk
constexpr int kChunk = kPlanThreads * kEach;

// The two sums a request adds: its new tokens and the blocks it takes.
struct PlanSum {
    long long tokens, blocks;
};

__device__ __forceinline__ long long blocks_of(long long tokens, int shift) {
    return (tokens + (1LL << shift) - 1) >> shift;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(KvPlanArgs a, int shift, long long range) {
    chain_entry();
    __shared__ PlanSum warp_sums[kPlanThreads / 32];
    __shared__ long long s_token[kChunk], s_block[kChunk];
    __shared__ int s_cached[kChunk];
    __shared__ unsigned long long s_beyond;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the last CTA also sees to tokens past max_tokens, which have blocks but no slots
    const long long lo = range * blockIdx.x, hi = blockIdx.x + 1 == gridDim.x ? LLONG_MAX : lo + range;
    if (tid == 0) s_beyond = 0;
    PlanSum all = {0, 0};
    for (int c0 = 0; c0 < a.requests; c0 += kChunk) {
        const int r0 = c0 + tid * kEach;
        int cached[kEach], fresh[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            cached[k] = r0 + k < a.requests ? max(__ldg(a.cached + r0 + k), 0) : 0;
            fresh[k] = r0 + k < a.requests ? max(__ldg(a.fresh + r0 + k), 0) : 0;
        }
        PlanSum mine = {0, 0};
        unsigned long long beyond = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const long long need = blocks_of(static_cast<long long>(cached[k]) + fresh[k], shift);
            mine.tokens += fresh[k];
            mine.blocks += need - blocks_of(cached[k], shift);
            beyond += need > a.width ? need - a.width : 0;
        }
        PlanSum incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long t = __shfl_up_sync(~0u, incl.tokens, d), b = __shfl_up_sync(~0u, incl.blocks, d);
            if (lane >= d) {
                incl.tokens += t;
                incl.blocks += b;
            }
        }
        __syncthreads();
        if (lane == 31) warp_sums[warp] = incl;
        if (blockIdx.x == 0 && beyond) atomicAdd(&s_beyond, beyond);
        __syncthreads();
        PlanSum at = all;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < warp) {
                at.tokens += warp_sums[w].tokens;
                at.blocks += warp_sums[w].blocks;
            }
            all.tokens += warp_sums[w].tokens;
            all.blocks += warp_sums[w].blocks;
        }
        at.tokens += incl.tokens - mine.tokens;
        at.blocks += incl.blocks - mine.blocks;
        const long long chunk_lo = all.tokens - (warp_sums[0].tokens + warp_sums[1].tokens + warp_sums[2].tokens +
                                                 warp_sums[3].tokens + warp_sums[4].tokens + warp_sums[5].tokens +
                                                 warp_sums[6].tokens + warp_sums[7].tokens);
        // this CTA's share of the per-request outputs, and the chunk's sums
        const bool writes = (c0 / kEach + tid) % gridDim.x == blockIdx.x;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = tid * kEach + k;
            s_token[i] = at.tokens;
            s_block[i] = at.blocks;
            s_cached[i] = cached[k];
            if (writes && r0 + k < a.requests) {
                a.q_offsets[r0 + k] = static_cast<int>(min(at.tokens, a.max_tokens));
                a.kv_lens[r0 + k] =
                    static_cast<int>(min(static_cast<long long>(cached[k]) + fresh[k], static_cast<long long>(INT_MAX)));
            }
            at.tokens += fresh[k];
            at.blocks += blocks_of(static_cast<long long>(cached[k]) + fresh[k], shift) - blocks_of(cached[k], shift);
        }
        __syncthreads();
        const long long from = max(lo, chunk_lo), to = min(hi, all.tokens);
        for (long long t = from + tid; t < to; t += kPlanThreads) {
            // the last request whose first token is not after t (those past the
            // last request, and those without new tokens, are passed over)
            int i = 0;
#pragma unroll
            for (int step = kChunk / 2; step; step >>= 1)
                if (s_token[i + step] <= t) i += step;
            const int r = c0 + i;
            const long long c = s_cached[i];
            const long long pos = c + (t - s_token[i]), b = pos >> shift, have = blocks_of(c, shift);
            const long long in_block = pos & ((1LL << shift) - 1);
            int id = -1;
            if (b < have) {
                if (b < a.width) id = a.table[static_cast<long long>(r) * a.width + b];
            } else {
                const long long f = s_block[i] + (b - have);
                if (f < a.num_free) id = __ldg(a.free_blocks + f);
                if (b >= a.width)
                    id = -1;
                else if (in_block == 0)
                    a.table[static_cast<long long>(r) * a.width + b] = id;
            }
            if (t < a.max_tokens) a.slots[t] = id >= 0 ? (static_cast<long long>(id) << shift) + in_block : -1;
        }
    }
    for (long long t = max(lo, all.tokens) + tid; t < min(hi, a.max_tokens); t += kPlanThreads) a.slots[t] = -1;
    if (blockIdx.x == 0 && tid == 0) {
        const long long most = INT_MAX;
        a.q_offsets[a.requests] = static_cast<int>(min(all.tokens, a.max_tokens));
        a.counts[0] = static_cast<int>(min(all.blocks, static_cast<long long>(a.num_free)));
        a.counts[1] = static_cast<int>(min(all.tokens, most));
        a.counts[2] = static_cast<int>(min(max(all.blocks - a.num_free, 0LL), most));
        a.counts[3] = static_cast<int>(min(s_beyond, static_cast<unsigned long long>(most)));
    }
}

cudaError_t launch_kv_plan(const KvPlanArgs &a, cudaStream_t s) {
    int shift = 0;
    while ((1 << shift) < a.block_size) ++shift;
    cudaError_t err = cudaSuccess;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    long long grid = (a.max_tokens + kPlanThreads - 1) / kPlanThreads;
    grid = grid < 1 ? 1 : grid > 2 * sms ? 2 * sms : grid;
    const long long range = (a.max_tokens + grid - 1) / grid;
    return launch_chained(kv_plan_kernel, static_cast<unsigned>(grid), kPlanThreads, 0, s, a, shift, range);
}

}  // namespace qrk
