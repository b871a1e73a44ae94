// Rows in 8 bits: e4m3 codes with one fp32 scale per 128 consecutive values, as dsa_norm_q8 and dsa_gemm_q8 write them.
#pragma once

#include "common.cuh"

namespace dsa {

constexpr int kRowBlock = 128;  // values that share a scale

__host__ __device__ constexpr int row_blocks(int n) { return (n + kRowBlock - 1) / kRowBlock; }

// The scale of a block: amax / 448, at least 2^-126 (so that neither it nor its reciprocal leaves fp32's normal range), 1
// for a block of zeros.
__device__ __forceinline__ float block_scale8(float amax) { return amax > 0.f ? fmaxf(amax / 448.f, 0x1p-126f) : 1.f; }

// v / scale as correctly rounded division gives it: a product with the reciprocal and one correction by the quotient's remainder
// (Markstein's).
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

// Two fp32 values in a register pair: packed arithmetic takes half the instructions, each rounded as its scalar form.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
// The two bf16 values of a word.
__device__ __forceinline__ uint64_t pair_of_bf16(uint32_t w) {
    return pair2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// BlockQuotient of two values at a time.
struct BlockQuotient2 {
    uint64_t r, minus_s;
    __device__ __forceinline__ explicit BlockQuotient2(float scale) {
        const BlockQuotient q(scale);
        r = pair2(q.r, q.r), minus_s = pair2(-q.s, -q.s);
    }
    __device__ __forceinline__ uint64_t operator()(uint64_t v) const {
        const uint64_t q = mul2(v, r);
        return fma2(fma2(q, minus_s, v), r, q);
    }
};

// 1 / v within 2^-23 of it, v and 1 / v normal.
__device__ __forceinline__ float near_reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Four codes in a word, the first in the low byte; round to nearest even, saturating, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t w;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(w)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return w;
}
__device__ __forceinline__ uint32_t e4m3x4(uint64_t ab, uint64_t cd) { return e4m3x4(lo_of(ab), hi_of(ab), lo_of(cd), hi_of(cd)); }

// Two bf16 values in a word, the first in the low half, rounded to nearest even by one instruction.
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}

}  // namespace dsa
