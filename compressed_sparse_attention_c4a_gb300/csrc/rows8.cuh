// Rows in 8 bits: e4m3 codes with one fp32 scale per 128 consecutive values, as dsa_norm_q8, dsa_gemm_q8 and
// dsa_sparse_attn_q8 write them.
#pragma once

#include "common.cuh"

namespace dsa {

constexpr int kRowBlock = 128;  // values that share a scale

__host__ __device__ constexpr int row_blocks(int n) { return (n + kRowBlock - 1) / kRowBlock; }

// The scale of a block: amax / 448, at least 2^-126 (so that neither it nor its reciprocal leaves fp32's normal range), 1
// for a block of zeros.
__device__ __forceinline__ float block_scale8(float amax) { return amax > 0.f ? fmaxf(amax / 448.f, 0x1p-126f) : 1.f; }

// v / scale as correctly rounded division gives it: a product with the reciprocal and one correction by the remainder.
// An infinite scale (a block that holds an infinity) makes 0 of finite values and NaN of infinities, as division does.
struct BlockQuotient {
    float r, s;
    __device__ __forceinline__ explicit BlockQuotient(float scale)
        : r(1.f / scale), s(scale < INFINITY ? scale : 0.f) {}
    __device__ __forceinline__ float operator()(float v) const {
        const float q = v * r;
        return fmaf(fmaf(-q, s, v), r, q);
    }
};

// Four codes in a word, the first in the low byte; round to nearest even, saturating, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Two bf16 values in a word, the first in the low half, rounded to nearest even by one instruction.
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}

}  // namespace dsa
