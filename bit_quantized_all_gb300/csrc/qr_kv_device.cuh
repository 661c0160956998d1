// qr_kv_device.cuh -- device-side pieces of the attention over the 8-bit
// paged cache: the cache's view, conversions of int8 codes into fp16 pairs,
// asynchronous 16-byte copies and the m16n8k16 fp16 product.
#pragma once

#include <cstdint>

#include "qr_device.cuh"
#include "qr_pipeline.cuh"
#include "qr_serving.h"

namespace qrk {

struct KvView {
    const int8_t *k, *v;
    const float *ks, *vs;
    long long k_block, k_head, v_block, v_head;  // bytes
    int blocks, heads, dim, shift;               // block_size = 1 << shift
};

inline KvView kv_view(const qr_kv_cache_t &c) {
    KvView v = {static_cast<const int8_t *>(c.k_codes), static_cast<const int8_t *>(c.v_codes), c.k_scales,
                c.v_scales, c.k_block_stride, c.k_head_stride, c.v_block_stride, c.v_head_stride,
                c.blocks, c.heads, c.head_dim, 0};
    while ((1 << v.shift) < c.block_size) ++v.shift;
    return v;
}

// int8 codes become fp16 exactly: a code's byte with its sign flipped (code +
// 128, 0..255) under the high byte 0x64 is the fp16 number 1024 + 128 + code,
// from which 1152 is subtracted (exact: every |code| <= 128).
constexpr uint32_t kFlip = 0x80808080u, kHigh = 0x64646464u;

// The scale of a block's values is split into a power of two and a rest of at
// most 1: 2^e with e in [kLeastExp, 129], scale <= 2^e.
constexpr int kLeastExp = -100;
__device__ __forceinline__ int scale_exp(float s) {
    return max(static_cast<int>((__float_as_uint(s) >> 23) & 255) - 126, kLeastExp);
}
// 2^n for -126 <= n <= 127
__device__ __forceinline__ float pow2i(int n) { return __uint_as_float(static_cast<uint32_t>(n + 127) << 23); }

__device__ __forceinline__ uint32_t minus_1152(uint32_t h2) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&h2), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Four codes of one word as two fp16 pairs, in order.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    w ^= kFlip;
    lo = minus_1152(__byte_perm(w, kHigh, 0x4140));
    hi = minus_1152(__byte_perm(w, kHigh, 0x4342));
}

// Four codes each of two words as pairs (a_i, b_i).
__device__ __forceinline__ void codes_f16_pairs(uint32_t a, uint32_t b, uint32_t (&out)[4]) {
    const uint32_t lo = __byte_perm(a, b, 0x5140) ^ kFlip, hi = __byte_perm(a, b, 0x7362) ^ kFlip;
    out[0] = minus_1152(__byte_perm(lo, kHigh, 0x4140));
    out[1] = minus_1152(__byte_perm(lo, kHigh, 0x4342));
    out[2] = minus_1152(__byte_perm(hi, kHigh, 0x4140));
    out[3] = minus_1152(__byte_perm(hi, kHigh, 0x4342));
}

// D = A B + C on fp16 operands with fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                        float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_f16_acc(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// What the rounding of y to the fp16 pair h left, as fp16.
__device__ __forceinline__ uint32_t rest_f16(float2 y, uint32_t h) {
    const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_f16(y.x - r.x, y.y - r.y);
}

// The transpose of an 8 x 8 matrix of 16-bit values, of which lane 4 g + t
// holds row g, columns 2t and 2t + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

// The larger value, NaN if either is: a query that is not finite gives NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace qrk
