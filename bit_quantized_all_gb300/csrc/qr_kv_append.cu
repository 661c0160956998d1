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
};

__device__ __forceinline__ int quantize8(float x, float r) {
    return __float2int_rn(fminf(fmaxf(__fmul_rn(x, r), -128.0f), 127.0f));
}

// A warp takes one run: the call's tokens of one block, one head, keys or
// values.  Its first pass finds the largest magnitude, its second quantizes.
template <int DT>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(KvAppendArgs a, int window) {
    chain_entry();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = blockIdx.y, half = blockIdx.z;
    const uint16_t *x = a.x[half] + head * a.x_head[half];
    const long long xt = a.x_token[half];
    const int bs = 1 << a.shift, vpr = a.dim >> 3;
    const long long first = static_cast<long long>(blockIdx.x) * window;
    for (int w = warp; w < window; w += kAppendThreads / 32) {
        const long long t0 = first + w;
        if (t0 >= a.tokens) break;
        const long long slot = a.slots[t0];
        if (slot < 0 || slot >= a.num_slots) continue;
        const int o = static_cast<int>(slot & (bs - 1));
        if (t0 > 0 && o > 0 && a.slots[t0 - 1] == slot - 1) continue;  // inside another run
        // the run: consecutive slots up to the block's end
        int n = 1;
        const int most = static_cast<int>(min(static_cast<long long>(bs - o), a.tokens - t0));
        for (bool on = true; on && n < most;) {
            const int i = n + lane;
            const bool same = i < most && a.slots[t0 + i] == slot + i;
            const unsigned m = __ballot_sync(~0u, same);
            const int c = m == ~0u ? 32 : __ffs(~m) - 1;
            n += c;
            on = c == 32;
        }
        const long long b = slot >> a.shift;
        float amax = 0.0f;
        for (int i = lane; i < n * vpr; i += 32) {
            float f[8];
            widen8<DT>(*reinterpret_cast<const uint4 *>(x + (t0 + i / vpr) * xt + (i % vpr) * 8), f);
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(f[k]));
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
        float *sp = a.scales[half] + b * a.heads + head;
        const float old = o > 0 ? *sp : 0.0f;
        const float s = fmaxf(old, __fmul_rn(amax, 0.0078125f));
        const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
        __syncwarp();
        if (lane == 0) *sp = s;
        int8_t *page = a.codes[half] + b * a.block_stride[half] + head * a.head_stride[half];
        if (o > 0 && s > old) {
            for (int i = lane; i < o * a.dim / 16; i += 32) {
                uint4 c = reinterpret_cast<uint4 *>(page)[i];
                uint32_t *u = &c.x;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t v = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float q = static_cast<float>(static_cast<int8_t>(u[k] >> (8 * j)));
                        v |= static_cast<uint32_t>(quantize8(__fmul_rn(q, old), r) & 255) << (8 * j);
                    }
                    u[k] = v;
                }
                reinterpret_cast<uint4 *>(page)[i] = c;
            }
        }
        for (int i = lane; i < n * vpr; i += 32) {
            const int row = i / vpr, col = i % vpr;
            float f[8];
            widen8<DT>(*reinterpret_cast<const uint4 *>(x + (t0 + row) * xt + col * 8), f);
            uint32_t v[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k / 4] |= static_cast<uint32_t>(quantize8(f[k], r) & 255) << (8 * (k % 4));
            *reinterpret_cast<uint2 *>(page + (o + row) * a.dim + col * 8) = make_uint2(v[0], v[1]);
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
    for (a.shift = 0; (1 << a.shift) < cache.block_size;) ++a.shift;
    const int window = 8;
    const dim3 grid(static_cast<unsigned>((tokens + window - 1) / window), cache.heads, 2);
    return launch_chained(dtype ? kv_append_kernel<1> : kv_append_kernel<0>, grid, kAppendThreads, 0, s, a, window);
}

}  // namespace qrk
