// qr_norm.cuh -- rows in 8 bits and the root-mean-square norm with the
// residual's addition (qr_q8_quantize, qr_rms_norm, qr_rms_norm_q8);
// instantiated per type in qr_norm_f16.cu and qr_norm_bf16.cu.
//
// One pass: a row stays in registers between its sum of squares and largest
// magnitude and its output.  The 8-bit codes of (h rs w) do not depend on rs, a
// factor of the whole row, so that they come from h w, and rs goes into the
// scale; both reductions share one barrier.
#pragma once

#include "qr_device.cuh"
#include "qr_kv_device.cuh"
#include "qr_launch.h"
#include "qr_serving.h"
#include "qr_w4.cuh"

namespace qrk {

// Eight 16-bit values, any alignment, those before `have`.
template <bool ALIGNED>
__device__ __forceinline__ uint4 load8(const uint16_t *p, int have) {
    if constexpr (ALIGNED) return have > 0 ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
    else return load8_any(p, have);
}

// ... and back, by the widest stores that the address allows.
template <bool ALIGNED>
__device__ __forceinline__ void store8(uint16_t *p, const uint4 o, int have) {
    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15;
    if (ALIGNED || (have >= 8 && off == 0)) {
        if (have > 0) *reinterpret_cast<uint4 *>(p) = o;
    } else if (have >= 8 && (off & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t *>(p)[i] = w[i];
    } else if (have >= 8) {
        p[0] = static_cast<uint16_t>(w[0]);
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t *>(p + 1 + 2 * i) = __funnelshift_r(w[i], w[i + 1], 16);
        p[7] = static_cast<uint16_t>(w[3] >> 16);
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < have) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
}

// W: weight none (0), in x's type (1), fp32 (2).
template <int DT, int W, bool ALIGNED>
struct NormWeight {
    uint4 raw[W == 2 ? 2 : 1];

    __device__ __forceinline__ void load(const void *weight, int i, int have) {
        if constexpr (W == 1) raw[0] = load8<ALIGNED>(static_cast<const uint16_t *>(weight) + i, have);
        if constexpr (W == 2) {
            const float *const p = static_cast<const float *>(weight) + i;
            if (ALIGNED) {
                if (have > 0) raw[0] = reinterpret_cast<const uint4 *>(p)[0], raw[1] = reinterpret_cast<const uint4 *>(p)[1];
            } else {
                uint32_t v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = e < have ? __float_as_uint(p[e]) : 0u;
                raw[0] = make_uint4(v[0], v[1], v[2], v[3]);
                raw[1] = make_uint4(v[4], v[5], v[6], v[7]);
            }
        }
    }
    __device__ __forceinline__ void get(float (&w)[8]) const {
        if constexpr (W == 1) widen8<DT>(raw[0], w);
        if constexpr (W == 2) {
            const uint32_t v[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __uint_as_float(v[e]);
        }
    }
};

// The bytes of four codes of v * f (|v f| is at most 127 (1 + 2^-23), or NaN,
// which gives what it gives): adding 1.5 * 2^23 rounds half to even and leaves
// the integer in the low bits.
__device__ __forceinline__ uint32_t row_codes(const float *v, float f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(__fadd_rn(__fmul_rn(v[i], f), 12582912.0f));
    return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
}

// 127 / most, 0 where that is not finite.
__device__ __forceinline__ float row_factor(float most) {
    const float f = __fdiv_rn(127.0f, most);
    return f < INFINITY ? f : 0.0f;
}

__device__ __forceinline__ float norm_factor(float sum, const NormArgs &a) {
    return __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(a.cols)), a.eps));
}

// A row's sum and largest magnitude over its threads: a warp (WARP), or the CTA.
template <bool WARP, bool SUM, bool MAX>
__device__ __forceinline__ void row_reduce(float &sum, float &most, float2 *s, int turn) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        if (SUM) sum += __shfl_xor_sync(~0u, sum, d);
        if (MAX) most = max_nan(most, __shfl_xor_sync(~0u, most, d));
    }
    if constexpr (!WARP) {
        // (two buffers in turn: nobody is two barriers ahead)
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) s[turn * 32 + (threadIdx.x >> 5)] = make_float2(sum, most);
        __syncthreads();
        const float2 p = lane < warps ? s[turn * 32 + lane] : make_float2(0.0f, 0.0f);
        sum = p.x, most = p.y;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            if (SUM) sum += __shfl_xor_sync(~0u, sum, d);
            if (MAX) most = max_nan(most, __shfl_xor_sync(~0u, most, d));
        }
    }
}

// A row a CTA, or a warp (WARP); P pieces of eight values a thread, THREADS at
// most.  HOLD: the weights stay in registers from row to row, and the next row is
// on its way while this one is reduced.
template <int DT, int W, bool EIGHT, bool ALIGNED, bool WARP, int P, int THREADS, bool HOLD>
__global__ void __launch_bounds__(THREADS) norm_kernel(NormArgs a) {
    chain_entry();
    __shared__ float2 s_part[64];
    const int threads = WARP ? 32 : blockDim.x, me = WARP ? threadIdx.x & 31 : threadIdx.x;
    const long long stride = WARP ? gridDim.x * (blockDim.x / 32ll) : gridDim.x;
    long long t = WARP ? blockIdx.x * (blockDim.x / 32ll) + (threadIdx.x >> 5) : blockIdx.x;
    const auto *const x = static_cast<const uint16_t *>(a.x), *const res = static_cast<const uint16_t *>(a.residual);
    const bool has_res = W && res != nullptr;

    NormWeight<DT, W, ALIGNED> weight[HOLD ? P : 1];
    uint4 rx[P], rr[P];
    auto load = [&](long long row) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int i = (me + p * threads) * 8;
            rx[p] = load8<ALIGNED>(x + row * a.x_row + i, a.cols - i);
            if (has_res) rr[p] = load8<ALIGNED>(res + row * a.residual_row + i, a.cols - i);
        }
    };
    auto weights = [&](int p, float (&w)[8]) {
        if (!HOLD) weight[0].load(a.weight, (me + p * threads) * 8, a.cols - (me + p * threads) * 8);
        weight[HOLD ? p : 0].get(w);
    };
    if (HOLD) {
        if (t < a.tokens) load(t);
#pragma unroll
        for (int p = 0; p < P; ++p)
            weight[HOLD ? p : 0].load(a.weight, (me + p * threads) * 8, a.cols - (me + p * threads) * 8);
    }
    for (int turn = 0; t < a.tokens; t += stride, turn ^= 1) {
        float h[P][8];  // in 8 bits: h times the weight
        float sum = 0.0f, most = 0.0f;
        if (!HOLD) load(t);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int i = (me + p * threads) * 8;
            widen8<DT>(rx[p], h[p]);
            if (has_res) {
                float r[8];
                widen8<DT>(rr[p], r);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[p][e] = __fadd_rn(h[p][e], r[e]);
                if (a.residual_out) {
                    uint4 o;
                    o.x = narrow2<DT>(h[p][0], h[p][1]), o.y = narrow2<DT>(h[p][2], h[p][3]);
                    o.z = narrow2<DT>(h[p][4], h[p][5]), o.w = narrow2<DT>(h[p][6], h[p][7]);
                    store8<ALIGNED>(static_cast<uint16_t *>(a.residual_out) + t * a.residual_out_row + i, o, a.cols - i);
                }
            }
            if (i >= a.cols) continue;
            float w[8];
            if (W && EIGHT) weights(p, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (W) sum = __fmaf_rn(h[p][e], h[p][e], sum);
                if (W && EIGHT) h[p][e] = __fmul_rn(h[p][e], w[e]);
                if (EIGHT) most = max_nan(most, fabsf(h[p][e]));
            }
        }
        if (HOLD && t + stride < a.tokens) load(t + stride);
        row_reduce<WARP, W != 0, EIGHT>(sum, most, s_part, turn);
        const float rs = W ? norm_factor(sum, a) : 1.0f;
        if constexpr (EIGHT) {
            const float f = row_factor(most);
            if (me == 0) a.scales[t] = __fmul_rn(__fdiv_rn(most, 127.0f), rs);
            uint8_t *const to = static_cast<uint8_t *>(a.y) + t * a.y_row;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int i = (me + p * threads) * 8;
                if (i >= a.cols) break;
                const uint2 o = make_uint2(row_codes(h[p], f), row_codes(h[p] + 4, f));
                if (ALIGNED || i + 8 <= a.cols) {
                    *reinterpret_cast<uint2 *>(to + i) = o;
                } else {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (i + e < a.cols) to[i + e] = static_cast<uint8_t>((e < 4 ? o.x : o.y) >> (8 * (e & 3)));
                }
            }
        } else {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int i = (me + p * threads) * 8;
                if (i >= a.cols) break;
                float w[8];
                weights(p, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[p][e] = h[p][e] * rs * w[e];
                uint4 o;
                o.x = narrow2<DT>(h[p][0], h[p][1]), o.y = narrow2<DT>(h[p][2], h[p][3]);
                o.z = narrow2<DT>(h[p][4], h[p][5]), o.w = narrow2<DT>(h[p][6], h[p][7]);
                store8<ALIGNED>(static_cast<uint16_t *>(a.y) + t * a.y_row + i, o, a.cols - i);
            }
        }
    }
}

// Rows longer than a CTA's registers: read twice, a value a thread at a time.
constexpr int kNormLongThreads = 1024;
template <int DT, int W, bool EIGHT>
__global__ void __launch_bounds__(kNormLongThreads) norm_long_kernel(NormArgs a) {
    chain_entry();
    __shared__ float2 s_part[64];
    const auto *const x = static_cast<const uint16_t *>(a.x), *const res = static_cast<const uint16_t *>(a.residual);
    int turn = 0;
    for (long long t = blockIdx.x; t < a.tokens; t += gridDim.x, turn ^= 1) {
        auto h_at = [&](int i) {
            float h = widen1<DT>(x[t * a.x_row + i]);
            if (W && res) h = __fadd_rn(h, widen1<DT>(res[t * a.residual_row + i]));
            return h;
        };
        auto w_at = [&](int i) {
            if (W == 2) return static_cast<const float *>(a.weight)[i];
            return W == 1 ? widen1<DT>(static_cast<const uint16_t *>(a.weight)[i]) : 1.0f;
        };
        float sum = 0.0f, most = 0.0f;
        for (int i = threadIdx.x; i < a.cols; i += kNormLongThreads) {
            const float h = h_at(i);
            if (W) sum = __fmaf_rn(h, h, sum);
            if (EIGHT) most = max_nan(most, fabsf(W ? __fmul_rn(h, w_at(i)) : h));
        }
        row_reduce<false, W != 0, EIGHT>(sum, most, s_part, turn);
        const float rs = W ? norm_factor(sum, a) : 1.0f, f = row_factor(most);
        if (EIGHT && threadIdx.x == 0) a.scales[t] = __fmul_rn(__fdiv_rn(most, 127.0f), rs);
        for (int i = threadIdx.x; i < a.cols; i += kNormLongThreads) {
            const float h = h_at(i);
            if (W && a.residual_out) static_cast<uint16_t *>(a.residual_out)[t * a.residual_out_row + i] = narrow1<DT>(h);
            if constexpr (EIGHT) {
                const float v[4] = {W ? __fmul_rn(h, w_at(i)) : h, 0.0f, 0.0f, 0.0f};
                static_cast<uint8_t *>(a.y)[t * a.y_row + i] = static_cast<uint8_t>(row_codes(v, f));
            } else {
                static_cast<uint16_t *>(a.y)[t * a.y_row + i] = narrow1<DT>(h * rs * w_at(i));
            }
        }
    }
}

template <int DT, int W, bool EIGHT, bool ALIGNED>
static cudaError_t run_norm(const NormArgs &a, cudaStream_t s) {
    cudaError_t err = cudaSuccess;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    auto launch = [&](auto kern, int threads, int rows) {
        const int grid = grid_for(reinterpret_cast<const void *>(kern), threads, (a.tokens + rows - 1) / rows, 0, 1, &err);
        return grid <= 0 ? err : launch_chained(kern, grid, threads, 0, s, a);
    };
    if (a.cols > 32768) return launch(norm_long_kernel<DT, W, EIGHT>, kNormLongThreads, 1);
    const int pieces = (a.cols + 7) / 8;
    if (a.cols <= 1024 && a.tokens > 8 * sms)
        return launch(norm_kernel<DT, W, EIGHT, ALIGNED, true, 4, 256, ALIGNED>, 256, 8);
    if (pieces <= 1024 && a.tokens <= 2 * sms)
        return launch(norm_kernel<DT, W, EIGHT, ALIGNED, false, 1, 1024, false>, (pieces + 31) / 32 * 32, 1);
    if (pieces <= 2048)
        return launch(norm_kernel<DT, W, EIGHT, ALIGNED, false, 4, 512, ALIGNED>, (pieces + 127) / 128 * 32, 1);
    return launch(norm_kernel<DT, W, EIGHT, ALIGNED, false, 4, 1024, false>, (pieces + 127) / 128 * 32, 1);
}

template <int DT>
cudaError_t launch_norm_typed(int weight, const NormArgs &a, cudaStream_t s) {
    const bool eight = a.scales != nullptr;
    auto rows16 = [&](const void *p, long long row) {
        return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (a.tokens == 1 || row % 8 == 0);
    };
    const bool vector = a.cols % 8 == 0 && rows16(a.x, a.x_row) && (!a.residual || rows16(a.residual, a.residual_row)) &&
                        (!a.residual_out || rows16(a.residual_out, a.residual_out_row)) && rows16(a.weight, 0) &&
                        rows16(a.y, a.y_row);
    if (weight == 0) return vector ? run_norm<DT, 0, true, true>(a, s) : run_norm<DT, 0, true, false>(a, s);
    if (weight == 1)
        return eight ? (vector ? run_norm<DT, 1, true, true>(a, s) : run_norm<DT, 1, true, false>(a, s))
                     : (vector ? run_norm<DT, 1, false, true>(a, s) : run_norm<DT, 1, false, false>(a, s));
    return eight ? (vector ? run_norm<DT, 2, true, true>(a, s) : run_norm<DT, 2, true, false>(a, s))
                 : (vector ? run_norm<DT, 2, false, true>(a, s) : run_norm<DT, 2, false, false>(a, s));
}

}  // namespace qrk
