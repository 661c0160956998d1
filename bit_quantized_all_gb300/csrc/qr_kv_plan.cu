// qr_kv_plan.cu -- block tables and slots of a serving step from the
// requests' lengths (qr_kv_plan).
//
// One launch.  Every CTA takes the same two exclusive sums over the requests
// (new tokens and newly needed blocks), each thread over its own run of
// requests, and keeps the requests that meet its slice of kSlice tokens; then
// its threads write the slice's slots, finding each token's request by
// bisection in shared memory.  A token that begins a block which the request
// did not hold also enters that block in the request's table row, so no CTA
// waits for another's result: a slot's block is either an entry that was
// there before the call or one of free_blocks, never one written here.
#include <climits>

#include "qr_device.cuh"
#include "qr_launch.h"
#include "qr_serving.h"

namespace qrk {

constexpr int kPlanThreads = 256;
constexpr int kSlice = 1024;  // tokens per CTA and step

__device__ __forceinline__ long long div_up_pow2(long long x, int shift) { return (x + (1LL << shift) - 1) >> shift; }

// The two sums a request adds: its new tokens and the blocks it takes.
struct PlanSum {
    long long tokens, blocks;
};

__device__ __forceinline__ PlanSum plan_request(const KvPlanArgs &a, int r, int shift, long long *cached) {
    const long long c = max(a.cached[r], 0), n = max(a.fresh[r], 0);
    *cached = c;
    return {n, div_up_pow2(c + n, shift) - div_up_pow2(c, shift)};
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(KvPlanArgs a, int shift) {
    chain_entry();
    __shared__ PlanSum warp_sums[kPlanThreads / 32];
    __shared__ int s_request[kSlice];
    __shared__ long long s_token[kSlice], s_block[kSlice];
    __shared__ int s_count;
    __shared__ long long s_beyond;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.requests + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(tid * per, a.requests), r1 = min(r0 + per, a.requests);

    // exclusive sums over the threads' runs
    PlanSum mine = {0, 0};
    long long beyond = 0, cached;
    for (int r = r0; r < r1; ++r) {
        const PlanSum x = plan_request(a, r, shift, &cached);
        mine.tokens += x.tokens;
        mine.blocks += x.blocks;
        beyond += max(0LL, div_up_pow2(cached + x.tokens, shift) - a.width);
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
    if (lane == 31) warp_sums[warp] = incl;
    if (tid == 0) s_beyond = 0;
    __syncthreads();
    PlanSum before = {0, 0}, all = {0, 0};
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w == warp) before = all;
        all.tokens += warp_sums[w].tokens;
        all.blocks += warp_sums[w].blocks;
    }
    before.tokens += incl.tokens - mine.tokens;
    before.blocks += incl.blocks - mine.blocks;

    // the per-request outputs, a share of the requests per CTA
    {
        PlanSum at = before;
        for (int r = r0; r < r1; ++r) {
            const PlanSum x = plan_request(a, r, shift, &cached);
            if (r % static_cast<int>(gridDim.x) == static_cast<int>(blockIdx.x)) {
                a.q_offsets[r] = static_cast<int>(min(at.tokens, a.max_tokens));
                a.kv_lens[r] = static_cast<int>(min(cached + x.tokens, static_cast<long long>(INT_MAX)));
            }
            at.tokens += x.tokens;
            at.blocks += x.blocks;
        }
    }
    if (blockIdx.x == 0) {
        if (beyond) atomicAdd(reinterpret_cast<unsigned long long *>(&s_beyond), static_cast<unsigned long long>(beyond));
        __syncthreads();
        if (tid == 0) {
            const long long most = INT_MAX;
            a.q_offsets[a.requests] = static_cast<int>(min(all.tokens, a.max_tokens));
            a.counts[0] = static_cast<int>(min(all.blocks, static_cast<long long>(a.num_free)));
            a.counts[1] = static_cast<int>(min(all.tokens, most));
            a.counts[2] = static_cast<int>(min(max(all.blocks - a.num_free, 0LL), most));
            a.counts[3] = static_cast<int>(min(s_beyond, most));
        }
    }

    const long long last = max(all.tokens, a.max_tokens);
    for (long long base = static_cast<long long>(blockIdx.x) * kSlice; base < last;
         base += static_cast<long long>(gridDim.x) * kSlice) {
        // the requests that meet [base, base + kSlice), in order: at most one
        // per token, as those without new tokens are left out
        __syncthreads();
        if (tid == 0) s_count = 0;
        __syncthreads();
        const long long end = base + kSlice;
        if (before.tokens < end && before.tokens + mine.tokens > base) {
            PlanSum at = before;
            for (int r = r0; r < r1 && at.tokens < end; ++r) {
                const PlanSum x = plan_request(a, r, shift, &cached);
                if (x.tokens > 0 && at.tokens + x.tokens > base) {
                    const int i = atomicAdd(&s_count, 1);
                    s_request[i] = r;
                    s_token[i] = at.tokens;
                    s_block[i] = at.blocks;
                }
                at.tokens += x.tokens;
                at.blocks += x.blocks;
            }
        }
        __syncthreads();
        const int count = s_count;
        // the atomics leave the list unordered across threads: rank each entry
        // by its first token, all entries in registers before any is moved
        constexpr int kEach = kSlice / kPlanThreads;
        int rank[kEach], req[kEach];
        long long tok[kEach], blk[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = tid + j * kPlanThreads;
            if (i < count) {
                req[j] = s_request[i];
                tok[j] = s_token[i];
                blk[j] = s_block[i];
                int k = 0;
                for (int m = 0; m < count; ++m) k += s_token[m] < tok[j];
                rank[j] = k;
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            if (tid + j * kPlanThreads < count) {
                s_request[rank[j]] = req[j];
                s_token[rank[j]] = tok[j];
                s_block[rank[j]] = blk[j];
            }
        __syncthreads();
        for (int j = 0; j < kEach; ++j) {
            const long long t = base + tid + j * kPlanThreads;
            if (t >= last) continue;
            long long slot = -1;
            if (t < all.tokens) {
                int lo = 0, hi = count - 1;  // the last entry whose first token is <= t
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (s_token[mid] <= t) lo = mid; else hi = mid - 1;
                }
                const int r = s_request[lo];
                const long long c = max(a.cached[r], 0);
                const long long pos = c + (t - s_token[lo]), b = pos >> shift, have = div_up_pow2(c, shift);
                int id = -1;
                if (b < have) {
                    if (b < a.width) id = a.table[static_cast<long long>(r) * a.width + b];
                } else {
                    const long long f = s_block[lo] + (b - have);
                    if (f < a.num_free) id = a.free_blocks[f];
                    if ((pos & ((1LL << shift) - 1)) == 0 && b < a.width)
                        a.table[static_cast<long long>(r) * a.width + b] = id;
                    if (b >= a.width) id = -1;
                }
                if (id >= 0) slot = (static_cast<long long>(id) << shift) + (pos & ((1LL << shift) - 1));
            }
            if (t < a.max_tokens) a.slots[t] = slot;
        }
    }
}

cudaError_t launch_kv_plan(const KvPlanArgs &a, cudaStream_t s) {
    int shift = 0;
    while ((1 << shift) < a.block_size) ++shift;
    cudaError_t err = cudaSuccess;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    long long grid = (a.max_tokens + kSlice - 1) / kSlice;
    grid = grid < 1 ? 1 : grid > 4 * sms ? 4 * sms : grid;
    return launch_chained(kv_plan_kernel, static_cast<unsigned>(grid), kPlanThreads, 0, s, a, shift);
}

}  // namespace qrk
