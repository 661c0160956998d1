// qr_kv_append.cu -- writes keys and values into the 8-bit paged cache
// (qr_kv_append).
#include "qr_device.cuh"
#include "qr_launch.h"
#include "qr_serving.h"

namespace qrk {

constexpr int kAppendThreads = 256;

struct KvAppendArgs {
    const uint16_t *x[2];            // keys, values
    long long x_token[2], x_head[2];
    int8_t *codes[2];
    float *scales[2];
    long long block_stride[2], head_stride[2];
    const int64_t *slots;
    long long tokens, num_slots;
    int heads, dim, shift;           // block_size = 1 << shift
    uint32_t inv;
};

// 1 / s, or 0 where that is not a number of fp32: s is 0, or at most 2^-128, which
// only bf16 magnitudes up to 2^-121 make it (codes of 0 are off by no more).
__device__ __forceinline__ float inverse_scale(float s) {
    const float r = __frcp_rn(s);
    return r < INFINITY ? r : 0.0f;
}

// Four codes as the bytes of a word.  |x| is at most 128 s and r 1 / s rounded,
// or 0, so |x r| is at most 128 (1 + 2^-23) and only the upper end can be left;
// adding 1.5 * 2^23 rounds half to even and leaves the integer in the low bits.
__device__ __forceinline__ uint32_t quantize4(const float *x, float r) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(__fadd_rn(fminf(__fmul_rn(x[i], r), 127.0f), 12582912.0f));
    return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
}

// A run is the call's tokens of one block, for one head of the keys or the
// values.  A CTA covers `window` tokens: it marks, in one pass over their
// slots, where runs begin and how far they go, and its warps take the runs, a
// warp each, or TEAM warps where a run is longer than a warp's registers.
// kPieces 16-byte pieces a lane stay in registers from the search for the
// largest magnitude to the quantization, so a run of 2048 * TEAM values is
// read once (a longer one twice).
//
// What bounds it: the bytes of a prompt (32 x 1024 tokens of 8 heads x 128:
// 37 us, 5.4 TB/s of reads and writes, 0.81 of the copy rate); for single
// tokens the launch and three dependent round trips, slot, block, codes (16
// tokens 2.9 us, 256 tokens of 8 heads 4.2 us).
constexpr int kPieces = 8;
constexpr int kMarks = 2 * kAppendThreads;  // the window, and a block's length past it

template <int DT>
struct AppendRun {
    const uint16_t *src;
    int8_t *dst;       // the codes of the run's first token
    long long stride;
    int pieces, vpr;
    uint32_t inv;      // ceil(2^32 / vpr): p / vpr is the high word of p * inv for these small p

    __device__ __forceinline__ uint4 load(int p) const {
        const int row = __umulhi(p, inv);
        return *reinterpret_cast<const uint4 *>(src + row * stride + (p - row * vpr) * 8);
    }
    // Pieces p0 + k * step of this lane; their largest magnitude.
    __device__ __forceinline__ float read(uint4 (&held)[kPieces], int p0, int step) const {
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
            if (p0 + k * step < pieces) held[k] = load(p0 + k * step);
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
            if (p0 + k * step < pieces) {
                float f[8];
                widen8<DT>(held[k], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
            }
        return amax;
    }
    __device__ __forceinline__ void write(const uint4 (&held)[kPieces], int p0, int step, float r) const {
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
            if (p0 + k * step < pieces) {
                float f[8];
                widen8<DT>(held[k], f);
                // the page's rows follow one another, so piece p is its 8 bytes p
                reinterpret_cast<uint2 *>(dst)[p0 + k * step] = make_uint2(quantize4(f, r), quantize4(f + 4, r));
            }
    }
};

template <int DT, int TEAM>
__global__ void __launch_bounds__(kAppendThreads, 4) kv_append_kernel(KvAppendArgs a, int window) {
    chain_entry();
    constexpr int kWarps = kAppendThreads / 32, kTeams = kWarps / TEAM;
    __shared__ unsigned s_goes_on[kMarks / 32 + 1];            // tokens that continue a run
    __shared__ int s_list[kAppendThreads];                     // runs: a warp's from the front, a team's from the back
    __shared__ int s_short, s_long;
    __shared__ float s_max[2][kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = blockIdx.y, half = blockIdx.z;
    const long long xt = a.x_token[half];
    const int bs = 1 << a.shift, vpr = a.dim >> 3;
    const long long base = static_cast<long long>(blockIdx.x) * window;

    bool begins = false;
    int first_o = 0;
    if (tid == 0) s_short = s_long = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = tid + j * kAppendThreads;
        const long long t = base + i;
        bool on = false;
        if (i < window + bs && t < a.tokens) {
            const long long slot = a.slots[t];
            const int o = static_cast<int>(slot & (bs - 1));
            on = o > 0 && t > 0 && a.slots[t - 1] == slot - 1;
            if (j == 0) {
                begins = i < window && slot >= 0 && slot < a.num_slots && !on;
                first_o = o;
            }
        }
        const unsigned m = __ballot_sync(~0u, on);
        if (lane == 0) s_goes_on[i >> 5] = m;
    }
    __syncthreads();
    const int most_warp = kPieces * 32 / vpr;  // tokens that a warp's registers hold
    if (begins) {
        // the run goes on until a token that does not continue it
        int i = tid + 1;
        const int stop = tid + bs - first_o;
        for (;;) {
            const unsigned rest = ~s_goes_on[i >> 5] >> (i & 31);
            if (rest) {
                i += __ffs(rest) - 1;
                break;
            }
            i = (i | 31) + 1;
            if (i >= stop) break;
        }
        const int n = min(i, stop) - tid;
        const int entry = tid | (n - 1) << 16;
        if (TEAM == 1 || n <= most_warp)
            s_list[atomicAdd(&s_short, 1)] = entry;
        else
            s_list[kAppendThreads - 1 - atomicAdd(&s_long, 1)] = entry;
    }
    __syncthreads();

    // One run by `lanes` threads, of which this is the `me`-th; the old scale
    // is read before join() and the new one written after it.
    auto take = [&](int entry, int me, int lanes, auto join) {
        const long long t0 = base + (entry & 0xffff);
        const int n = (entry >> 16) + 1;
        const long long slot = a.slots[t0], b = slot >> a.shift;
        const int o = static_cast<int>(slot & (bs - 1));
        float *const sp = a.scales[half] + b * a.heads + head;
        int8_t *const page = a.codes[half] + (b * a.block_stride[half] + head * a.head_stride[half]);
        const AppendRun<DT> run = {a.x[half] + head * a.x_head[half] + t0 * xt, page + o * a.dim, xt, n * vpr, vpr, a.inv};
        const float old = o > 0 ? *sp : 0.0f;
        const int batch = kPieces * lanes;
        uint4 held[kPieces];
        float amax = 0.0f;
        for (int p0 = 0; p0 < run.pieces; p0 += batch) amax = fmaxf(amax, run.read(held, p0 + me, lanes));
#pragma unroll
        for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
        amax = join(amax);
        const float s = fmaxf(old, __fmul_rn(amax, 0.0078125f));
        const float r = inverse_scale(s);
        if (me == 0) *sp = s;
        if (o > 0 && s > old) {
            for (int i = me; i < o * a.dim / 16; i += lanes) {
                const uint4 c = reinterpret_cast<uint4 *>(page)[i];
                uint32_t u[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float f[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        f[j] = __fmul_rn(static_cast<float>(static_cast<int8_t>(u[k] >> (8 * j))), old);
                    u[k] = quantize4(f, r);
                }
                reinterpret_cast<uint4 *>(page)[i] = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
        if (run.pieces <= batch) {
            run.write(held, me, lanes, r);
        } else {
            for (int p0 = 0; p0 < run.pieces; p0 += batch) {
                run.read(held, p0 + me, lanes);
                run.write(held, p0 + me, lanes, r);
            }
        }
    };
    for (int i = warp; i < s_short; i += kWarps)
        take(s_list[i], lane, 32, [](float amax) {
            __syncwarp();
            return amax;
        });
    if constexpr (TEAM > 1) {
        // every team goes round as often, as the warps of one meet at the barrier
        const int team = warp / TEAM, runs = s_long;
        for (int i0 = 0, turn = 0; i0 < runs; i0 += kTeams, turn ^= 1) {
            auto join = [&](float amax) {
                if (lane == 0) s_max[turn][warp] = amax;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < TEAM; ++w) amax = fmaxf(amax, s_max[turn][team * TEAM + w]);
                return amax;
            };
            if (i0 + team < runs)
                take(s_list[kAppendThreads - 1 - (i0 + team)], tid % (32 * TEAM), 32 * TEAM, join);
            else
                join(0.0f);
        }
    }
}

cudaError_t launch_kv_append(int dtype, long long tokens, const void *k, const void *v, long long k_token,
                             long long k_head, long long v_token, long long v_head, const int64_t *slots,
                             const qr_kv_cache_t &cache, cudaStream_t s) {
    KvAppendArgs a;
    a.x[0] = static_cast<const uint16_t *>(k);
    a.x[1] = static_cast<const uint16_t *>(v);
    a.x_token[0] = k_token, a.x_token[1] = v_token;
    a.x_head[0] = k_head, a.x_head[1] = v_head;
    a.codes[0] = static_cast<int8_t *>(cache.k_codes), a.codes[1] = static_cast<int8_t *>(cache.v_codes);
    a.scales[0] = cache.k_scales, a.scales[1] = cache.v_scales;
    a.block_stride[0] = cache.k_block_stride, a.block_stride[1] = cache.v_block_stride;
    a.head_stride[0] = cache.k_head_stride, a.head_stride[1] = cache.v_head_stride;
    a.slots = slots;
    a.tokens = tokens;
    a.num_slots = static_cast<long long>(cache.blocks) * cache.block_size;
    a.heads = cache.heads;
    a.dim = cache.head_dim;
    a.inv = static_cast<uint32_t>(((1ull << 32) + a.dim / 8 - 1) / (a.dim / 8));
    for (a.shift = 0; (1 << a.shift) < cache.block_size;) ++a.shift;
    // teams for runs of a whole block (8 x 1024 tokens into blocks of 128 of 256
    // dimensions 25 us, a warp each 59; 32 x 1024 into blocks of 32 of 128 37 and
    // 43); a window of eight tokens, more when the call would otherwise make over
    // eight CTAs a SM, most of them, in a prompt, with no run that begins in them
    // (the latter prompt with eight 142 us; 256 single tokens 4.2 us, with 256 38)
    cudaError_t err = cudaSuccess;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    const int run = cache.block_size * cache.head_dim;
    const int team = run <= 2048 ? 1 : run <= 4096 ? 2 : run <= 8192 ? 4 : 8;
    int window = kAppendThreads / 32;
    while (window < kAppendThreads && tokens * cache.heads * 2 > static_cast<long long>(8) * sms * window) window *= 2;
    const dim3 grid(static_cast<unsigned>((tokens + window - 1) / window), cache.heads, 2);
    auto kern = dtype ? (team == 1   ? kv_append_kernel<1, 1>
                         : team == 2 ? kv_append_kernel<1, 2>
                         : team == 4 ? kv_append_kernel<1, 4>
                                     : kv_append_kernel<1, 8>)
                      : (team == 1   ? kv_append_kernel<0, 1>
                         : team == 2 ? kv_append_kernel<0, 2>
                         : team == 4 ? kv_append_kernel<0, 4>
                                     : kv_append_kernel<0, 8>);
    return launch_chained(kern, grid, kAppendThreads, 0, s, a, window);
}

}  // namespace qrk
