// qr_kv_plan_range.h -- which new tokens a CTA of qr_kv_plan's kernel goes
// over within a chunk of requests.  Plain C++, so that the bounds are tested
// without a GPU.
#pragma once

#ifdef __CUDACC__
#define QR_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define QR_HOST_DEVICE inline
#endif

namespace qrk {

constexpr long long kPlanMostTokens = 2147483647;  // tokens past it are counted, and get neither block nor slot
constexpr int kPlanThreads = 256;
constexpr int kPlanWide = 4;                       // tokens per thread and step

// Tokens [from, to), empty if from >= to; all of them below kPlanMostTokens.
struct PlanTokens {
    long long from, to;
};

// The CTA owns tokens [lo, hi); the chunk's requests bring the tokens
// [chunk_lo, chunk_hi), which may lie past 2^31.
QR_HOST_DEVICE PlanTokens plan_tokens(long long lo, long long hi, long long chunk_lo, long long chunk_hi) {
    PlanTokens t;
    t.from = lo > chunk_lo ? lo : chunk_lo;
    t.to = hi < chunk_hi ? hi : chunk_hi;
    if (t.to > kPlanMostTokens) t.to = kPlanMostTokens;
    return t;
}

// A thread's first token; it goes on by kPlanWide * kPlanThreads.
QR_HOST_DEVICE long long plan_first(PlanTokens t, int thread) {
    return t.from + static_cast<long long>(kPlanWide) * thread;
}

}  // namespace qrk
