// qr_norm.cu -- rows in 8 bits and the root-mean-square norm with the
// residual's addition (qr_q8_quantize, qr_rms_norm, qr_rms_norm_q8).
#include "qr_device.cuh"
#include "qr_kv_device.cuh"
#include "qr_launch.h"
#include "qr_serving.h"

namespace qrk {

constexpr int kNormThreads = 256;

// W: weight none (0), in x's type (1), fp32 (2); EIGHT: rows in 8 bits.
template <int DT, int W, bool EIGHT>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(NormArgs a) {
    chain_entry();
    __shared__ float s_sum[kNormThreads / 32], s_max[kNormThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const auto *x = static_cast<const uint16_t *>(a.x), *res = static_cast<const uint16_t *>(a.residual);
    auto h_at = [&](long long t, int i) {
        float h = widen1<DT>(x[t * a.x_row + i]);
        if (res) h = __fadd_rn(h, widen1<DT>(res[t * a.residual_row + i]));
        return h;
    };
    auto w_at = [&](int i) {
        if (W == 2) return static_cast<const float *>(a.weight)[i];
        return W == 1 ? widen1<DT>(static_cast<const uint16_t *>(a.weight)[i]) : 1.0f;
    };
    for (long long t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        float sum = 0.0f, most = 0.0f;
        for (int i = tid; i < a.cols; i += kNormThreads) {
            const float h = h_at(t, i);
            if (W) sum = __fmaf_rn(h, h, sum);
            if (EIGHT) most = max_nan(most, fabsf(W ? __fmul_rn(h, w_at(i)) : h));
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            sum += __shfl_xor_sync(~0u, sum, d);
            most = max_nan(most, __shfl_xor_sync(~0u, most, d));
        }
        __syncthreads();
        if (lane == 0) s_sum[warp] = sum, s_max[warp] = most;
        __syncthreads();
        sum = 0.0f;
        for (int w = 0; w < kNormThreads / 32; ++w) sum += s_sum[w], most = max_nan(most, s_max[w]);
        const float rs = W ? __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(a.cols)), a.eps)) : 1.0f;
        float f = __fdiv_rn(127.0f, most);
        if (!(f < INFINITY)) f = 0.0f;
        if (EIGHT && tid == 0) a.scales[t] = __fmul_rn(__fdiv_rn(most, 127.0f), rs);
        for (int i = tid; i < a.cols; i += kNormThreads) {
            const float h = h_at(t, i);
            if (a.residual_out) static_cast<uint16_t *>(a.residual_out)[t * a.residual_out_row + i] = narrow1<DT>(h);
            if (EIGHT)
                static_cast<int8_t *>(a.y)[t * a.y_row + i] =
                    static_cast<int8_t>(__float2int_rn(__fmul_rn(W ? __fmul_rn(h, w_at(i)) : h, f)));
            else
                static_cast<uint16_t *>(a.y)[t * a.y_row + i] = narrow1<DT>(h * rs * w_at(i));
        }
    }
}

template <int DT>
static cudaError_t run_norm(int weight, const NormArgs &a, cudaStream_t s) {
    const bool eight = a.scales != nullptr;
    auto kern = weight == 0 ? norm_kernel<DT, 0, true>
                : weight == 1 ? (eight ? norm_kernel<DT, 1, true> : norm_kernel<DT, 1, false>)
                              : (eight ? norm_kernel<DT, 2, true> : norm_kernel<DT, 2, false>);
    const unsigned grid = static_cast<unsigned>(a.tokens < 65536 ? a.tokens : 65536);
    return launch_chained(kern, grid, kNormThreads, 0, s, a);
}

cudaError_t launch_norm(int dtype, int weight, const NormArgs &a, cudaStream_t s) {
    return dtype ? run_norm<1>(weight, a, s) : run_norm<0>(weight, a, s);
}

}  // namespace qrk
