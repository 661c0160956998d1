// qr_rope.cu -- rotary positions of queries and keys (qr_rope).
//
// A position times a frequency, both integers, in turns times 2^64, wraps at
// whole turns by itself, whatever the position; as a signed number it is the angle
// in half turns times 2^63, which becomes fp32 to the last bit but one.
//
// A CTA takes a few tokens.  Its threads first work out each token's sines and
// cosines, once for all heads, in shared memory; then a thread takes a unit of 2 VP
// values, VP rotated pairs in two loads of VP values (or as many that are only
// copied), of one head at a time.
//
// What bounds it: HBM (32768 tokens of 48 heads of 128, slices of a projection, 143 us,
// 5.6 TB/s of reads and writes, 0.83 of the copy rate); for few tokens the launch,
// position, sine and store one after the other (16 tokens 1.8 us).
#include "qr_device.cuh"
#include "qr_launch.h"
#include "qr_serving.h"

namespace qrk {

constexpr int kRopeThreads = 128;
constexpr int kRopePairs = 2048;  // of a CTA's tokens, at most
constexpr int kRopeTokens = 32;

struct RopeShape {
    int tokens;              // of a CTA
    int rot_units, units;    // of a head: those that are rotated, all
    int heads;
    uint32_t inv_units, inv_heads;  // see quotient()
};

// x / d: the high word of x times inv = ceil(2^32 / d), exact where x d < 2^32; inv
// is 0 where d is 1 or such x occur.
__device__ __forceinline__ int quotient(int x, int d, uint32_t inv) {
    return inv ? static_cast<int>(__umulhi(static_cast<uint32_t>(x), inv)) : x / d;
}

// The last request that begins at or before token t, by all lanes: of 32 places
// at a time.  (Requests without tokens begin where the next one does.)
__device__ __forceinline__ int request_of(const int32_t *q_offsets, int requests, long long t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = requests;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const bool at = lane * step < n && q_offsets[lo + lane * step] <= t;
        const unsigned m = __ballot_sync(~0u, at) | 1u;
        const int k = 31 - __clz(m);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// A signed number of 64 bits times 2^-63 (one conversion of all of it: 16 tokens 1.93
// us for 1.8).  The low word is signed too, so that a small negative number is not the
// difference of large ones; a high word that the carry takes past its largest value
// becomes -1, the same angle as 1.
__device__ __forceinline__ float half_turns(unsigned long long turn) {
    const int low = static_cast<int>(turn), high = static_cast<int>((turn + 0x80000000ull) >> 32);
    return __fmaf_rn(static_cast<float>(low), 0x1p-63f, static_cast<float>(high) * 0x1p-31f);
}

template <int VP>
struct RopeVec;  // VP 16-bit values in one access
template <> struct RopeVec<8> { using T = uint4; };
template <> struct RopeVec<4> { using T = uint2; };
template <> struct RopeVec<2> { using T = uint32_t; };
template <> struct RopeVec<1> { using T = uint16_t; };

template <int VP>
union RopePiece {
    typename RopeVec<VP>::T v;
    uint16_t h[VP];
};

template <int DT, bool INTERLEAVED, int VP>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a, RopeShape s) {
    chain_entry();
    using V = typename RopeVec<VP>::T;
    __shared__ __align__(16) float2 s_turn[kRopePairs];
    __shared__ int s_pos[kRopeTokens], s_skip[kRopeTokens];
    const int tid = threadIdx.x, pairs = a.rot / 2;
    const long long token0 = static_cast<long long>(blockIdx.x) * s.tokens;
    const int tokens = static_cast<int>(min(static_cast<long long>(s.tokens), a.tokens - token0));
    if (!a.positions) {
        for (int i = tid >> 5; i < tokens; i += kRopeThreads / 32) {
            const int r = request_of(a.q_offsets, a.requests, token0 + i);
            if ((tid & 31) == 0) {
                const long long end = a.q_offsets[r + 1];
                s_skip[i] = token0 + i >= end || token0 + i < a.q_offsets[r];
                s_pos[i] = static_cast<int>(a.kv_lens[r] - (end - (token0 + i)));
            }
        }
        __syncthreads();
    }

    const int tasks = tokens * s.heads * s.units;
    // units under way (four: 32768 x 48 heads 141 us for 143, 16 tokens 2.1 for 1.8,
    // 4097 of 10 heads 10.4 for 9.7; a round of them ahead: 154 us)
    constexpr int kEach = 2;
    struct Unit {
        const uint16_t *in;
        uint16_t *out;
        int turn;  // its first pair's place, -1 where it is copied
        bool on;
    };
    const int apart = INTERLEAVED ? VP : pairs;
    auto unit = [&](int i) {
        Unit u;
        const int q = quotient(i, s.units, s.inv_units), j = i - q * s.units, t = quotient(q, s.heads, s.inv_heads);
        int head = q - t * s.heads;
        const int which = head >= a.heads[0];
        if (which) head -= a.heads[0];
        const bool turned = j < s.rot_units;
        const int at = turned ? (INTERLEAVED ? 2 * j * VP : j * VP) : a.rot + (j - s.rot_units) * 2 * VP;
        u.on = i < tasks && (a.positions || !s_skip[t]);
        u.in = (which ? a.in[1] : a.in[0]) + (token0 + t) * (which ? a.in_token[1] : a.in_token[0]) +
               head * (which ? a.in_head[1] : a.in_head[0]) + at;
        u.out = (which ? a.out[1] : a.out[0]) + (token0 + t) * (which ? a.out_token[1] : a.out_token[0]) +
                head * (which ? a.out_head[1] : a.out_head[0]) + at;
        u.turn = turned ? t * pairs + j * VP : -1;
        return u;
    };
    Unit u[kEach];
    RopePiece<VP> x[kEach], y[kEach];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            u[k] = unit(i0 + k * kRopeThreads);
            if (u[k].on) {
                x[k].v = *reinterpret_cast<const V *>(u[k].in);
                y[k].v = *reinterpret_cast<const V *>(u[k].in + (u[k].turn < 0 ? VP : apart));
            }
        }
    };
    load(tid);
    for (int i = tid; i < tokens * pairs; i += kRopeThreads) {
        const int t = i / pairs, j = i - t * pairs;
        const long long p = a.positions ? a.positions[token0 + t] : s_pos[t];
        const unsigned long long turn = static_cast<unsigned long long>(p) * a.turns[j];
        float sn, cs;
        sincospif(half_turns(turn), &sn, &cs);
        s_turn[i] = make_float2(cs * a.factor, sn * a.factor);
    }
    __syncthreads();
    for (int i0 = tid; i0 < tasks; i0 += kEach * kRopeThreads) {
        if (i0 != tid) load(i0);
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (!u[k].on) continue;
            if (u[k].turn >= 0) {
                float2 cs[VP];
                if constexpr (VP >= 2) {
#pragma unroll
                    for (int e = 0; e < VP; e += 2) {
                        const float4 two = *reinterpret_cast<const float4 *>(s_turn + u[k].turn + e);
                        cs[e] = make_float2(two.x, two.y);
                        cs[e + 1] = make_float2(two.z, two.w);
                    }
                } else {
                    cs[0] = s_turn[u[k].turn];
                }
#pragma unroll
                for (int e = 0; e < VP; ++e) {
                    // pair e: values e of both pieces, or 2e and 2e + 1 of the two as one
                    uint16_t &ha = INTERLEAVED ? (2 * e < VP ? x[k].h[2 * e] : y[k].h[2 * e - VP]) : x[k].h[e];
                    uint16_t &hb = INTERLEAVED ? (2 * e + 1 < VP ? x[k].h[2 * e + 1] : y[k].h[2 * e + 1 - VP]) : y[k].h[e];
                    const float fa = widen1<DT>(ha), fb = widen1<DT>(hb);
                    ha = narrow1<DT>(__fmaf_rn(fa, cs[e].x, -__fmul_rn(fb, cs[e].y)));
                    hb = narrow1<DT>(__fmaf_rn(fb, cs[e].x, __fmul_rn(fa, cs[e].y)));
                }
            }
            *reinterpret_cast<V *>(u[k].out) = x[k].v;
            *reinterpret_cast<V *>(u[k].out + (u[k].turn < 0 ? VP : apart)) = y[k].v;
        }
    }
}

template <int DT, bool INTERLEAVED, int VP>
static cudaError_t run_rope(const RopeArgs &a, bool copies, cudaStream_t s) {
    cudaError_t err = cudaSuccess;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    RopeShape p;
    p.rot_units = a.rot / 2 / VP;
    p.units = p.rot_units + (copies ? (a.head_dim - a.rot) / (2 * VP) : 0);
    p.heads = a.heads[0] + a.heads[1];
    const int each = p.heads * p.units;
    p.tokens = 1;
    while (2 * p.tokens <= kRopeTokens && p.tokens * each < 8 * kRopeThreads && 2 * p.tokens * (a.rot / 2) <= kRopePairs &&
           a.tokens / (2 * p.tokens) >= 8ll * sms)
        p.tokens *= 2;
    // (threads past the last task divide too, up to a round further)
    const unsigned long long most = static_cast<unsigned long long>(p.tokens) * each + 8 * kRopeThreads;
    auto inverse = [&](int d) { return d == 1 || most * d >> 32 ? 0u : static_cast<uint32_t>(((1ull << 32) + d - 1) / d); };
    p.inv_units = inverse(p.units);
    p.inv_heads = inverse(p.heads);
    const long long grid = (a.tokens + p.tokens - 1) / p.tokens;
    return launch_chained(rope_kernel<DT, INTERLEAVED, VP>, static_cast<unsigned>(grid), kRopeThreads, 0, s, a, p);
}

template <int DT, bool INTERLEAVED>
static cudaError_t pick_rope(const RopeArgs &a, cudaStream_t s) {
    // a head's values past the rotated ones need no copying where nothing moves
    bool copies = false;
    int vp = 8;
    auto fits = [&](int n) {
        if (a.rot / 2 % n || (copies && (a.head_dim - a.rot) % (2 * n))) return false;
        for (int i = 0; i < (a.heads[1] ? 2 : 1); ++i) {
            const uintptr_t mask = 2 * n - 1;
            if ((reinterpret_cast<uintptr_t>(a.in[i]) & mask) || (reinterpret_cast<uintptr_t>(a.out[i]) & mask) ||
                a.in_token[i] % n || a.in_head[i] % n || a.out_token[i] % n || a.out_head[i] % n)
                return false;
        }
        return true;
    };
    for (int i = 0; i < 2; ++i) copies = copies || (a.in[i] != a.out[i] && a.rot < a.head_dim);
    while (vp > 1 && !fits(vp)) vp /= 2;
    return vp == 8   ? run_rope<DT, INTERLEAVED, 8>(a, copies, s)
           : vp == 4 ? run_rope<DT, INTERLEAVED, 4>(a, copies, s)
           : vp == 2 ? run_rope<DT, INTERLEAVED, 2>(a, copies, s)
                     : run_rope<DT, INTERLEAVED, 1>(a, copies, s);
}

cudaError_t launch_rope(int dtype, bool interleaved, const RopeArgs &a, cudaStream_t s) {
    if (dtype) return interleaved ? pick_rope<1, true>(a, s) : pick_rope<1, false>(a, s);
    return interleaved ? pick_rope<0, true>(a, s) : pick_rope<0, false>(a, s);
}

}  // namespace qrk
