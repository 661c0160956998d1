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
//
// What bounds it: the launch and the dependent round trips (16 requests 3.5 us;
// 2048 requests with a million new tokens 11 us, 0.8 TB/s).
#include <climits>

#include "qr_device.cuh"
#include "qr_kv_plan_range.h"
#include "qr_launch.h"
#include "qr_serving.h"

namespace qrk {

constexpr int kEach = 8;                         // requests per thread and chunk
constexpr int kChunk = kPlanThreads * kEach;
constexpr long long kMostTokens = kPlanMostTokens;
constexpr int kWide = kPlanWide;
static_assert(kMostTokens == INT_MAX, "token numbers are kept as int");

// The two sums a request adds: its new tokens and the blocks it takes.
struct PlanSum {
    long long tokens, blocks;
};

// Blocks of a length below 2^32.
__device__ __forceinline__ uint32_t blocks_of(uint32_t tokens, int shift) {
    return tokens ? ((tokens - 1) >> shift) + 1 : 0;
}

__global__ void __launch_bounds__(kPlanThreads, 3) kv_plan_kernel(KvPlanArgs a, int shift, long long range) {
    chain_entry();
    __shared__ PlanSum warp_sums[kPlanThreads / 32];
    // request 8 j + k of a chunk at [k][j]: the threads' stores meet no bank
    // twice, and the search goes over the j first
    __shared__ int s_token[kEach][kPlanThreads], s_block[kEach][kPlanThreads], s_cached[kEach][kPlanThreads];
    __shared__ unsigned long long s_beyond;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the last CTA also sees to tokens past max_tokens, which have blocks but no slots
    const long long lo = range * blockIdx.x, hi = blockIdx.x + 1 == gridDim.x ? kMostTokens : lo + range;
    if (tid == 0) s_beyond = 0;
    PlanSum all = {0, 0};
    for (int c0 = 0; c0 < a.requests; c0 += kChunk) {
        const int r0 = c0 + tid * kEach;
        int cached[kEach], fresh[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            cached[k] = r0 + k < a.requests ? max(a.cached[r0 + k], 0) : 0;
            fresh[k] = r0 + k < a.requests ? max(a.fresh[r0 + k], 0) : 0;
        }
        PlanSum mine = {0, 0};
        unsigned long long beyond = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const uint32_t c = cached[k], need = blocks_of(c + fresh[k], shift);
            mine.tokens += fresh[k];
            mine.blocks += need - blocks_of(c, shift);
            beyond += need > static_cast<uint32_t>(a.width) ? need - a.width : 0;
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
        const long long chunk_lo = all.tokens;
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
        // this CTA's share of the per-request outputs, and the chunk's sums
        const bool writes = (c0 / kEach + tid) % gridDim.x == blockIdx.x;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            s_token[k][tid] = static_cast<int>(min(at.tokens, kMostTokens));
            s_block[k][tid] = static_cast<int>(min(at.blocks, kMostTokens));
            s_cached[k][tid] = cached[k];
            if (writes && r0 + k < a.requests) {
                a.q_offsets[r0 + k] = static_cast<int>(min(at.tokens, a.max_tokens));
                a.kv_lens[r0 + k] =
                    static_cast<int>(min(static_cast<uint32_t>(cached[k]) + fresh[k], static_cast<uint32_t>(INT_MAX)));
            }
            at.tokens += fresh[k];
            at.blocks += blocks_of(static_cast<uint32_t>(cached[k]) + fresh[k], shift) - blocks_of(cached[k], shift);
        }
        __syncthreads();
        // in 64 bits: a chunk may begin past the last token that an int holds
        const PlanTokens range_here = plan_tokens(lo, hi, chunk_lo, all.tokens);
        const long long to = range_here.to;
        for (long long t0 = plan_first(range_here, tid); t0 < to; t0 += kWide * kPlanThreads) {
            // kWide tokens in a row: the first one's request is the last whose
            // first token is not after it (those past the last request, and
            // those without new tokens, are passed over), the others' follow
            int j = 0, k = 0;
#pragma unroll
            for (int step = kPlanThreads / 2; step; step >>= 1)
                if (s_token[0][j + step] <= t0) j += step;
#pragma unroll
            for (int step = kEach / 2; step; step >>= 1)
                if (s_token[k + step][j] <= t0) k += step;
            int i = j * kEach + k, id[kWide];
            uint32_t pos[kWide];
            int request[kWide];
#pragma unroll
            for (int u = 0; u < kWide; ++u) {
                if (u && t0 + u < to)
                    while (i + 1 < kChunk && s_token[(i + 1) % kEach][(i + 1) / kEach] <= t0 + u) ++i;
                k = i % kEach, j = i / kEach;
                request[u] = c0 + i;
                const uint32_t c = s_cached[k][j], have = blocks_of(c, shift);
                pos[u] = c + (static_cast<uint32_t>(t0) + u - static_cast<uint32_t>(s_token[k][j]));
                const uint32_t b = pos[u] >> shift, f = s_block[k][j] + (b - have);
                const bool held = b < have;
                id[u] = -1;
                if (t0 + u < to && (held ? b < static_cast<uint32_t>(a.width) : f < static_cast<uint32_t>(a.num_free)))
                    id[u] = held ? a.table[static_cast<long long>(request[u]) * a.width + b] : a.free_blocks[f];
            }
#pragma unroll
            for (int u = 0; u < kWide; ++u) {
                const long long t = t0 + u;
                const uint32_t b = pos[u] >> shift, in_block = pos[u] & ((1u << shift) - 1);
                if (t >= to) break;
                if (b >= static_cast<uint32_t>(a.width))
                    id[u] = -1;
                else if (in_block == 0)
                    a.table[static_cast<long long>(request[u]) * a.width + b] = id[u];
                if (t < a.max_tokens)
                    a.slots[t] = id[u] >= 0 ? (static_cast<long long>(id[u]) << shift) + in_block : -1;
            }
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
    grid = grid < 1 ? 1 : grid > 3 * sms ? 3 * sms : grid;
    const long long range = (a.max_tokens + grid - 1) / grid;
    return launch_chained(kv_plan_kernel, static_cast<unsigned>(grid), kPlanThreads, 0, s, a, shift, range);
}

}  // namespace qrk
