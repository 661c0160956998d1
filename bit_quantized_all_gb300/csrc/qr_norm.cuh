// qr_norm.cuh -- rows in 8 bits and the root-mean-square norm with the
// residual's addition (qr_q8_quantize, qr_rms_norm, qr_rms_norm_q8);
// instantiated per type in qr_norm_f16.cu and qr_norm_bf16.cu.
//
// One pass: a row stays in registers between its sum of squares and largest
// magnitude and its output.  The 8-bit codes of (h rs w) do not depend on rs, a
// factor of the whole row, so that they come from h w, and rs goes into the
// scale; both reductions share one barrier.
//
// What bounds it: HBM (32768 x 8192 in 8 bits with the residual 272 to 276 us, 6.8 to
// 6.9 TB/s, a plain copy's rate; 8192 x 20480 without a norm 74 us, 6.8 TB/s); for few
// rows the launch and two round trips (16 x 8192 2.4 us); for a few thousand rows that do
// not begin on 16-byte boundaries a CTA's rows one after the other, load, barrier and
// store, with more instructions a piece (2049 x 5123 in 16 bits 14 us, 2049 x 5120 10; 55%
// of the issue slots and 22 warps an SM in use).
#pragma once

#include "qr_device.cuh"
#include "qr_kv_device.cuh"
#include "qr_launch.h"
#include "qr_serving.h"

namespace qrk {

// A piece is eight values of a row on a 16-byte boundary, from value i on.  Where
// rows do not begin on such boundaries (SHIFT), the first and the last piece of a
// row are partly outside it: they are read whole, as aligned words that hold a
// value of the row, and what is outside becomes zero when it is used (masking
// what a load has just asked for would wait for it).
__device__ __forceinline__ uint4 load_piece(const uint16_t *row, int i, int cols) {
    return i < cols ? *reinterpret_cast<const uint4 *>(row + i) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ bool edge_piece(int i, int cols) { return i < 0 || (i < cols && i + 8 > cols); }
// `mask`: of the row's first piece and of its last (one piece may be both).
__device__ __forceinline__ uint4 inside(uint4 r, int i, int cols, const uint4 *mask) {
    const uint4 a = i < 0 ? mask[0] : make_uint4(~0u, ~0u, ~0u, ~0u), b = i + 8 > cols ? mask[1] : make_uint4(~0u, ~0u, ~0u, ~0u);
    return make_uint4(r.x & a.x & b.x, r.y & a.y & b.y, r.z & a.z & b.z, r.w & a.w & b.w);
}

template <int DT, bool SHIFT>
__device__ __forceinline__ void store_piece(uint16_t *row, int i, int cols, const float (&v)[8]) {
    const uint32_t w[4] = {narrow2<DT>(v[0], v[1]), narrow2<DT>(v[2], v[3]), narrow2<DT>(v[4], v[5]), narrow2<DT>(v[6], v[7])};
    if (!SHIFT || !edge_piece(i, cols)) {
        *reinterpret_cast<uint4 *>(row + i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i + e >= 0 && i + e < cols) row[i + e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
    }
}

// W: weight none (0), in x's type (1), fp32 (2); of a piece, from aligned words
// or, SHIFT, value by value.
template <int DT, int W, bool SHIFT>
struct NormWeight {
    uint4 raw[W == 2 ? 2 : 1];

    __device__ __forceinline__ void load(const void *weight, int i, int cols) {
        if (W == 0 || i >= cols) return;
        if constexpr (SHIFT) {
            uint32_t v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = 0;
                if (i + e >= 0 && i + e < cols)
                    v[e] = W == 2 ? static_cast<const uint32_t *>(weight)[i + e] : static_cast<const uint16_t *>(weight)[i + e];
            }
            if constexpr (W == 2) {
                raw[0] = make_uint4(v[0], v[1], v[2], v[3]);
                raw[1] = make_uint4(v[4], v[5], v[6], v[7]);
            } else {
                raw[0] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
            }
        } else if constexpr (W == 1) {
            raw[0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(weight) + i);
        } else {
            const uint4 *const p = reinterpret_cast<const uint4 *>(static_cast<const float *>(weight) + i);
            raw[0] = p[0], raw[1] = p[1];
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

// A code (in the low byte), and the bytes of four, of v * f (|v f| is at most 127 (1 + 2^-23), or NaN,
// which gives what it gives): adding 1.5 * 2^23 rounds half to even and leaves
// the integer in the low bits.
__device__ __forceinline__ uint32_t row_code(float v, float f) {
    return __float_as_uint(__fadd_rn(__fmul_rn(v, f), 12582912.0f));
}
__device__ __forceinline__ uint32_t row_codes(const float *v, float f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = row_code(v[i], f);
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

// A row a CTA, or a warp (WARP); P pieces a thread, THREADS threads at most.
// AHEAD: the next row is on its way while this one is reduced, and the weights
// stay in registers from row to row: a CTA's (or warp's) rows are a multiple of
// eight apart, so that they all lie alike between 16-byte words.
//
// Shifted rows in 8 bits: codes begin on boundaries that the pieces do not, so
// that eight of them are a piece's last and the next lane's first; a warp's last
// lane has the piece that the next warp's first has too, and stores none.
template <int DT, int W, bool EIGHT, bool SHIFT, bool WARP, int P, int THREADS, bool AHEAD>
__global__ void __launch_bounds__(THREADS, WARP || (P == 2 && !EIGHT) || THREADS == 320 ? 2 : 1) norm_kernel(NormArgs a) {
    chain_entry();
    constexpr int kLanes = SHIFT && EIGHT ? 31 : 32;
    __shared__ float2 s_part[64];
    __shared__ uint4 s_mask[2];
    const int lane = threadIdx.x & 31, cols = a.cols;
    const int threads = WARP ? kLanes : (blockDim.x >> 5) * kLanes, me0 = WARP ? 0 : (threadIdx.x >> 5) * kLanes;
    const bool own = kLanes == 32 || lane < kLanes;
    const long long stride = WARP ? gridDim.x * (blockDim.x / 32ll) : gridDim.x;
    long long t = WARP ? blockIdx.x * (blockDim.x / 32ll) + (threadIdx.x >> 5) : blockIdx.x;
    const auto *const x = static_cast<const uint16_t *>(a.x), *const res = static_cast<const uint16_t *>(a.residual);
    const bool has_res = W && res != nullptr;

    // values between the 16-byte boundary at or before the rows and their first
    const int off = SHIFT ? static_cast<int>(reinterpret_cast<uintptr_t>(x + t * a.x_row) >> 1 & 7) : 0;
    auto place = [&](int p) { return (me0 + lane + p * threads) * 8 - off; };
    // whether the warp has a piece of the row in its p-th place
    auto any = [&](int p) { return (me0 + p * threads) * 8 - off < cols; };
    // (weights that are not held are read a group ahead of its stores)
    constexpr int kGroup = AHEAD ? P : P > 2 ? 2 : 1;
    NormWeight<DT, W, SHIFT> weight[kGroup];
    uint4 rx[P], rr[P];
    auto load = [&](long long row) {
        const uint16_t *const xr = x + row * a.x_row, *const sr = res + row * a.residual_row;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            rx[p] = load_piece(xr, place(p), cols);
            if (has_res) rr[p] = load_piece(sr, place(p), cols);
        }
    };
    auto weights = [&](int p, float (&w)[8]) {
        if (!AHEAD && p % kGroup == 0) {
#pragma unroll
            for (int k = 0; k < kGroup; ++k) weight[k].load(a.weight, place(p + k), cols);
        }
        weight[p % kGroup].get(w);
    };
    if constexpr (AHEAD) {
        if (t < a.tokens) load(t);
#pragma unroll
        for (int p = 0; p < P; ++p) weight[p].load(a.weight, place(p), cols);
    }
    // (the rows of a warp of its own lie as that warp's do: a mask each is not worth
    // its shared memory, it is worked out)
    if (SHIFT && !WARP && threadIdx.x < 16) {
        const int last = (cols + off) & 7, e = threadIdx.x & 7;
        const bool in = threadIdx.x < 8 ? e >= off : e < (last ? last : 8);
        reinterpret_cast<uint16_t *>(s_mask)[threadIdx.x] = in ? 0xffff : 0;
    }
    if (SHIFT && !WARP) __syncthreads();
    for (int turn = 0; t < a.tokens; t += stride, turn ^= 1) {
        float h[W ? P : 1][8];  // in 8 bits: h times the weight
        uint4 kept[P];          // x itself where there is no weight
        float sum = 0.0f, most = 0.0f;
        if (!AHEAD) load(t);
        // a warp's last lane reads what the next warp's first one may write, the
        // residual in place; rows ahead are read before the barrier of the row before
        if (kLanes < 32 && WARP) __syncwarp();
        if (kLanes < 32 && !WARP && !AHEAD) __syncthreads();
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if ((SHIFT || WARP) && !any(p)) break;
            const int i = place(p);
            float(&v)[8] = h[W ? p : 0];
            auto masked = [&](uint4 r) {
                if (!SHIFT || !edge_piece(i, cols)) return r;
                if constexpr (!WARP) return inside(r, i, cols, s_mask);
                uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (i + e < 0 || i + e >= cols) w[e >> 1] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
                return make_uint4(w[0], w[1], w[2], w[3]);
            };
            kept[p] = masked(rx[p]);
            widen8<DT>(kept[p], v);
            float w[8];
            if (W && EIGHT) weights(p, w);
            if (i >= cols) continue;
            if (has_res) {
                float r[8];
                widen8<DT>(masked(rr[p]), r);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __fadd_rn(v[e], r[e]);
                if (a.residual_out && own)
                    store_piece<DT, SHIFT>(static_cast<uint16_t *>(a.residual_out) + t * a.residual_out_row, i, cols, v);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (W && own) sum = __fmaf_rn(v[e], v[e], sum);
                if (W && EIGHT) v[e] = __fmul_rn(v[e], w[e]);
                if (EIGHT) most = max_nan(most, fabsf(v[e]));
            }
        }
        if (AHEAD && t + stride < a.tokens) load(t + stride);
        row_reduce<WARP, W != 0, EIGHT>(sum, most, s_part, turn);
        const float rs = W ? norm_factor(sum, a) : 1.0f;
        if constexpr (EIGHT) {
            const float f = row_factor(most);
            if (me0 + lane == 0) a.scales[t] = __fmul_rn(__fdiv_rn(most, 127.0f), rs);
            uint8_t *const to = static_cast<uint8_t *>(a.y) + t * a.y_row;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if ((SHIFT || WARP) && !any(p)) break;
                const int i = place(p);
                float(&v)[8] = h[W ? p : 0];
                if (!W) widen8<DT>(kept[p], v);
                const uint2 o = make_uint2(row_codes(v, f), row_codes(v + 4, f));
                if constexpr (!SHIFT) {
                    if (i < cols) *reinterpret_cast<uint2 *>(to + i) = o;
                } else {
                    unsigned long long mine = o.x | static_cast<unsigned long long>(o.y) << 32;
                    const unsigned long long next = __shfl_down_sync(~0u, mine, 1);
                    if (off) mine = mine >> (8 * off) | next << (64 - 8 * off);
                    const int have = cols - i - off;
                    if (own && have >= 8) {
                        *reinterpret_cast<unsigned long long *>(to + i + off) = mine;
                    } else if (own && have > 0) {
#pragma unroll 1
                        for (int e = 0; e < have; ++e) to[i + off + e] = static_cast<uint8_t>(mine >> (8 * e));
                    }
                }
            }
        } else {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if ((SHIFT || WARP) && !any(p)) break;
                const int i = place(p);
                float w[8], (&v)[8] = h[W ? p : 0];
                weights(p, w);
                if (i >= cols) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = v[e] * rs * w[e];
                store_piece<DT, SHIFT>(static_cast<uint16_t *>(a.y) + t * a.y_row, i, cols, v);
            }
        }
    }
}

// Rows longer than a CTA's registers, or on unlike boundaries: read twice, a value
// a thread at a time.
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
                static_cast<uint8_t *>(a.y)[t * a.y_row + i] =
                    static_cast<uint8_t>(row_code(W ? __fmul_rn(h, w_at(i)) : h, f));
            } else {
                static_cast<uint16_t *>(a.y)[t * a.y_row + i] = narrow1<DT>(h * rs * w_at(i));
            }
        }
    }
}

template <int DT, int W, bool EIGHT, bool SHIFT>
static cudaError_t run_norm(const NormArgs &a, cudaStream_t s) {
    cudaError_t err = cudaSuccess;
    const int sms = sm_count(&err);
    if (sms <= 0) return err;
    constexpr int kLanes = SHIFT && EIGHT ? 31 : 32;
    const int pieces = (a.cols + 7) / 8 + SHIFT;
    auto threads = [&](int p) { return (pieces + kLanes * p - 1) / (kLanes * p) * 32; };
    auto launch = [&](auto kern, int n, int rows) {
        const long long units = (a.tokens + rows - 1) / rows;
        int grid = grid_for(reinterpret_cast<const void *>(kern), n, units, 0, 1, &err);
        if (SHIFT && rows == 1 && grid < units) grid &= ~7;  // (a CTA's rows lie alike)
        return grid <= 0 ? err : launch_chained(kern, grid, n, 0, s, a);
    };
    // Times in us of bf16 rows: in 8 bits with the residual / norm in 16 bits / 8 bits
    // without a norm.
    //
    // A warp a row from eight rows an SM on (2432 x 1024: 3.2 / 2.7 / 2.4, a CTA a row 4.3 /
    // 3.8 / 2.8; 1300 x 1024 alike; 608 x 1024: 2.4 / 2.0 / 1.7 and 2.1 / 2.0 / 1.6).
    if (threads(4) <= 32 && a.tokens > 8 * sms) return launch(norm_kernel<DT, W, EIGHT, SHIFT, true, 4, 256, true>, 256, 8);
    // Few rows: one piece a thread, the fewest loads in turn, up to 640 threads (16 x 5120:
    // 2.0 / 1.8 / 1.5, four pieces a thread 2.1 / 2.0 / 1.6; 304 x 5120: 3.2 / 2.8 / 1.9 and 3.3 /
    // 2.6 / 1.9; past that 16 x 8192: 2.5 / 2.2 / 1.7 and 2.3 / 2.1 / 1.7; 304 x 5632: 3.4 / 2.9 /
    // 2.0 and 2.8 / 2.4 / 1.9), and wherever shifts make a piece dear (16 x 7001: 3.5 / 2.7 /
    // 2.0 and 5.8 / 3.4 / 2.1).  From two rows an SM on the other form has the next row on its
    // way (456 x 5120: 4.2 / 3.6 / 2.7 and 3.1 / 2.7 / 2.3).
    if (threads(1) <= (SHIFT ? 1024 : 640) && a.tokens <= 2 * sms)
        return launch(norm_kernel<DT, W, EIGHT, SHIFT, false, 1, 1024, false>, threads(1), 1);
    // Without a weight a row needs fewer registers: eight pieces a thread keep long rows
    // ahead (8192 x 24576: 98, four pieces of 1024 threads 127).  Up to 320 threads two such
    // CTAs fit an SM, with 96 registers a thread (8192 x 20480: 75, one CTA an SM 89).  (Up to
    // 384 with 80 registers: 8192 x 22528 81 for 94, 24576 92 for 98, not built.)
    if constexpr (W == 0) {
        if (threads(4) > 512)
            return threads(8) <= 320 ? launch(norm_kernel<DT, 0, EIGHT, SHIFT, false, 8, 320, true>, threads(8), 1)
                                     : launch(norm_kernel<DT, 0, EIGHT, SHIFT, false, 8, 512, true>, threads(8), 1);
    }
    // Shifted rows: two pieces a thread (2049 x 5123: 22.5 / 11.8 / -, four pieces 30.8 / 12.5;
    // aligned rows alike or slower: 32768 x 8192 310 / 177 / - and 276 / 180).
    if constexpr (SHIFT) {
        if (threads(2) <= 512) return launch(norm_kernel<DT, W, EIGHT, SHIFT, false, 2, 512, true>, threads(2), 1);
    }
    // Four pieces of up to 512 threads, the next row ahead (32768 x 8192: 276 / 180, 1024
    // threads without it 311 / 183); longer rows: 1024 threads (8192 x 20480: 212 / 168, read
    // twice 360 / 196).
    if (threads(4) <= 512) return launch(norm_kernel<DT, W, EIGHT, SHIFT, false, 4, 512, true>, threads(4), 1);
    if constexpr (!SHIFT) return launch(norm_kernel<DT, W, EIGHT, false, false, 4, 1024, false>, threads(4), 1);
    return cudaErrorInvalidValue;  // (pick_norm sends none)
}

template <int DT, int W, bool EIGHT>
static cudaError_t pick_norm(const NormArgs &a, cudaStream_t s) {
    // 16-byte words: rows that all begin on them, and a weight that does; or rows
    // that all lie alike between them
    auto at = [](const void *p) { return reinterpret_cast<uintptr_t>(p) & 15; };
    auto alike = [&](const void *p, long long row) {
        return !p || (at(p) == at(a.x) && (a.tokens == 1 || (row - a.x_row) % 8 == 0));
    };
    const bool like = alike(a.residual, a.residual_row) && alike(a.residual_out, a.residual_out_row) &&
                      (EIGHT || alike(a.y, a.y_row));
    const bool whole = a.cols % 8 == 0 && at(a.x) == 0 && (a.tokens == 1 || a.x_row % 8 == 0) && at(a.weight) == 0;
    if (like && whole && a.cols <= 32768) return run_norm<DT, W, EIGHT, false>(a, s);
    // Shifted rows as far as 512 threads hold them with the next row on its way.  Without
    // that, 1024 threads lost to the kernel that reads rows twice at every size (in 8 bits
    // with the residual 8192 x 20481 598 us, read twice 356; 16 x 16401 9.8 and 6.5).
    constexpr int kShifted = W == 0 ? 31 * 1024 : (EIGHT ? 31 : 32) * 512;
    if (like && a.cols <= kShifted - 8) return run_norm<DT, W, EIGHT, true>(a, s);
    cudaError_t err = cudaSuccess;
    const int grid = grid_for(reinterpret_cast<const void *>(norm_long_kernel<DT, W, EIGHT>), kNormLongThreads, a.tokens, 0, 1, &err);
    return grid <= 0 ? err : launch_chained(norm_long_kernel<DT, W, EIGHT>, grid, kNormLongThreads, 0, s, a);
}

template <int DT>
cudaError_t launch_norm_typed(int weight, const NormArgs &a, cudaStream_t s) {
    const bool eight = a.scales != nullptr;
    if (weight == 0) return pick_norm<DT, 0, true>(a, s);
    if (weight == 1) return eight ? pick_norm<DT, 1, true>(a, s) : pick_norm<DT, 1, false>(a, s);
    return eight ? pick_norm<DT, 2, true>(a, s) : pick_norm<DT, 2, false>(a, s);
}

}  // namespace qrk
