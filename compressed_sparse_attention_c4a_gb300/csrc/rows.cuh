// Cache rows in registers: loading bf16 rows and storing rows in every pool format.
#pragma once

#include "common.cuh"

namespace dsa {

// ---- rows of e2m1 codes with a scale per block of 16 (DSA_FP4_BLOCK, dim 512) ---------------------------------------
// value_d = s * bs_{d / 16} * e2m1(code_d).  s is a power of two, so x / s is exact; the block scale bs = e4m3(amax of
// the block / (6 s)) has 4 significant bits and a code 2, so a value has at most 6: exact in bf16.  For bf16 inputs
// every rounding below decides as exact arithmetic would: a quotient that is not itself a border between two codes
// differs from one by more than 2^-16 relative, and a quotient that is one is computed exactly.
constexpr int kFp4BlockRow = 288;  // bytes: 256 of codes, 32 of block scales

inline bool block_rows_ok(const dsa_pool_t* p) { return p->dtype != DSA_FP4_BLOCK || p->dim == 512; }

// Largest |v| as its bit pattern: patterns of magnitudes order as the magnitudes do, infinities and NaN above all.
template <int E>
__device__ __forceinline__ uint32_t lane_abs_max_bits(const float (&v)[E]) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < E; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
    return m;
}
__device__ __forceinline__ uint32_t warp_abs_max_bits(uint32_t m) { return __reduce_max_sync(0xffffffffu, m); }

// The row scale s = 2^e, e the least integer with amax <= 2688 * 2^e (2688 = 448 * 6 = 1.3125 * 2^11) and e >= -126,
// and 1 / s.  A zero row: s = 1.  A row with an infinity or a NaN: s = NaN and 1 / s = 0, so that its codes are zero
// and it reads back as NaN.
__device__ __forceinline__ void fp4_block_row_scale(uint32_t amax_bits, float* s, float* inv_s) {
    int e = (int)(amax_bits >> 23) - 127 - 11 + ((amax_bits & 0x7fffffu) > 0x280000u ? 1 : 0);
    e = max(e, -126);
    *s = __uint_as_float((uint32_t)(e + 127) << 23);
    *inv_s = __uint_as_float((uint32_t)(127 - e) << 23);
    if (amax_bits == 0u) *s = 1.f, *inv_s = 1.f;
    if (amax_bits >= 0x7f800000u) *s = __uint_as_float(0x7fc00000u), *inv_s = 0.f;
}

// Eight codes with every zero as code 0, whatever its sign: 7 added to a code's magnitude carries into the sign's place
// unless the magnitude is 0.
__device__ __forceinline__ uint32_t fp4_plain_zeros(uint32_t c) {
    return c & (((c & 0x77777777u) + 0x77777777u) | 0x77777777u);
}

// One block: its e4m3 scale (returned) and 16 codes (element 2j in the low nibble).  v / (s bs) is a reciprocal and one
// correction by the quotient's remainder (Markstein's), which gives the quotient itself wherever that is representable (the
// borders are).
__device__ __forceinline__ uint8_t fp4_block_codes(const float (&v)[kFp4Block], float block_amax, float inv_s,
                                                   uint32_t (&c)[2]) {
    const float a = inv_s == 0.f ? 0.f : block_amax * inv_s;
    const uint8_t bs8 = float_to_e4m3(a / 6.f);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(bs8, __NV_E4M3);
    const float bs = __half2float(*reinterpret_cast<const __half*>(&h));
    const float r = bs > 0.f ? 1.f / bs : 0.f;
    c[0] = c[1] = 0u;
#pragma unroll
    for (int k = 0; k < kFp4Block / 2; ++k) {
        float q[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float u = inv_s == 0.f ? 0.f : v[2 * k + e] * inv_s;
            const float q0 = u * r;
            q[e] = fmaf(fmaf(-q0, bs, u), r, q0);
        }
        c[k / 4] |= (uint32_t)float2_to_e2m1x2(q[0], q[1]) << (8 * (k % 4));
    }
    c[0] = fp4_plain_zeros(c[0]), c[1] = fp4_plain_zeros(c[1]);
    return bs8;
}

// The same for a row of bf16 values (the lane's block as packed words), row scale included, with half the instructions.
// A quotient q of a bf16 value (8 significant bits) by a scale (4) that is not one of the borders between two codes (3)
// differs from it by more than 2^-8 of it, at least 2^-10.  So q may be off by 2^-20 before it is rounded to a multiple of
// 2^-19, which every border is: the fused multiply-add adds 24, whose neighbours are 2^-19 apart, to v (1 / (s bs)), and
// 24 is taken off again.  The reciprocal's 2^-23 makes 2^-20.6 at the largest border, 5; from 8 on (a scale at the end of
// e4m3's range) the code is the largest either way.
__device__ __forceinline__ uint8_t fp4_block_codes_bf16(uint32_t (&u)[kFp4Block / 2], uint32_t (&c)[2], float* s) {
    uint32_t m2 = 0u;
#pragma unroll
    for (int k = 0; k < kFp4Block / 2; ++k) m2 = __vmaxu2(m2, u[k] & 0x7fff7fffu);
    const uint32_t m = max(m2 << 16, m2 & 0xffff0000u);
    float inv_s;
    fp4_block_row_scale(warp_abs_max_bits(m), s, &inv_s);
    float a = __uint_as_float(m) * inv_s;
    if (inv_s == 0.f) {  // the row holds an infinity or a NaN
        a = 0.f;
#pragma unroll
        for (int k = 0; k < kFp4Block / 2; ++k) u[k] = 0u;
    }
    const float a0 = a * (1.f / 6.f);  // and a correction by the remainder, which makes it the quotient
    const uint8_t bs8 = float_to_e4m3(fmaf(fmaf(-a0, 6.f, a), 1.f / 6.f, a0));
    const __half_raw h = __nv_cvt_fp8_to_halfraw(bs8, __NV_E4M3);
    const float bs = __half2float(*reinterpret_cast<const __half*>(&h));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(bs));
    r = bs > 0.f ? r : 0.f;
    if (inv_s > 0x1p100f) {  // a row of tiny values: r / s could leave fp32's range
#pragma unroll
        for (int k = 0; k < kFp4Block / 2; ++k) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(u[k]) : "r"(0x5F805F80u));  // 2^64
        inv_s *= 0x1p-64f;
    }
    r *= inv_s;
    c[0] = c[1] = 0u;
#pragma unroll
    for (int k = 0; k < kFp4Block / 2; ++k) {
        const float v[2] = {__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u)};
        uint64_t t;
        asm("{\n\t.reg .b64 v, k, c;\n\t"
            "mov.b64 v, {%1, %2};\n\tmov.b64 k, {%3, %3};\n\tmov.b64 c, {%4, %4};\n\t"
            "fma.rn.f32x2 v, v, k, c;\n\tmov.b64 c, {%5, %5};\n\tadd.rn.f32x2 %0, v, c;\n\t}"
            : "=l"(t)
            : "f"(v[0]), "f"(v[1]), "f"(r), "f"(24.f), "f"(-24.f));
        c[k / 4] |= (uint32_t)float2_to_e2m1x2(__uint_as_float((uint32_t)t), __uint_as_float((uint32_t)(t >> 32)))
                    << (8 * (k % 4));
    }
    c[0] = fp4_plain_zeros(c[0]), c[1] = fp4_plain_zeros(c[1]);
    return bs8;
}

// ---- rows ------------------------------------------------------------------------------------------------------
// A warp owns a row, each lane E = dim / 32 consecutive elements.
template <int E>
__device__ __forceinline__ void load_bf16_words(const uint16_t* row, int lane, uint32_t (&u)[E / 2], bool wide) {
    const uint16_t* p = row + lane * E;
    if constexpr (E == 16) {
        if (wide) {  // 32-byte aligned: one access (two of 16 bytes each touch half of every sector)
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                         : "l"(p)
                         : "memory");
            return;
        }
        const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 8);
        u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w, u[4] = b.x, u[5] = b.y, u[6] = b.z, u[7] = b.w;
    } else if constexpr (E == 4) {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        u[0] = a.x, u[1] = a.y;
    } else {
        static_assert(E == 2, "row width");
        u[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}
template <int E>
__device__ __forceinline__ void bf16_words(const uint32_t (&u)[E / 2], float (&v)[E]) {
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
        v[2 * k] = __uint_as_float(u[k] << 16);
        v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
}
template <int E>
__device__ __forceinline__ void load_bf16(const uint16_t* row, int lane, float (&v)[E]) {
    uint32_t u[E / 2];
    load_bf16_words<E>(row, lane, u, false);
    bf16_words<E>(u, v);
}

// N words to consecutive memory.
template <int N>
__device__ __forceinline__ void store_words(uint16_t* p, const uint32_t (&u)[N], bool wide) {
    if constexpr (N == 8) {
        if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                         "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                         : "memory");
            return;
        }
        reinterpret_cast<uint4*>(p)[0] = make_uint4(u[0], u[1], u[2], u[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(u[4], u[5], u[6], u[7]);
    } else if constexpr (N == 2) {
        *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
    } else {
        static_assert(N == 1, "words");
        *reinterpret_cast<uint32_t*>(p) = u[0];
    }
}

__device__ __forceinline__ void store_fp4_block_row(const dsa_pool_t& pool, long long prow, int lane, const uint32_t (&c)[2],
                                                    uint8_t bs, float s) {
    uint8_t* dst = reinterpret_cast<uint8_t*>(pool.data) + prow * kFp4BlockRow;
    *reinterpret_cast<uint2*>(dst + lane * 8) = make_uint2(c[0], c[1]);
    dst[256 + lane] = bs;
    if (lane == 0) pool.scale[prow] = s;
}

// Store one row (the warp's E values per lane) into a pool row: bf16, e4m3 + amax/448 scale, e2m1 + amax/6, or e2m1
// with a scale per block of 16 (rows of 512 only).  The 4-bit formats last: behind them the e4m3 store of the
// compressor takes longer (16 requests of c128a, entry and window row: 12.7 us against 12.3).
template <int E>
__device__ __forceinline__ void store_row(const dsa_pool_t& pool, long long prow, int lane, const float (&v)[E]) {
    if (pool.dtype == DSA_BF16) {
        uint32_t u[E / 2];
#pragma unroll
        for (int k = 0; k < E / 2; ++k)
            u[k] = (uint32_t)float_to_bf16(v[2 * k]) | ((uint32_t)float_to_bf16(v[2 * k + 1]) << 16);
        store_words<E / 2>(reinterpret_cast<uint16_t*>(pool.data) + prow * (E * 32) + lane * E, u, false);
    } else if (pool.dtype == DSA_FP8_E4M3) {
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < E; ++k) amax = fmaxf(amax, fabsf(v[k]));
        amax = warp_max(amax);
        const float scale = amax > 0.f ? amax / 448.f : 1.f;
        uint8_t* dst = reinterpret_cast<uint8_t*>(pool.data) + prow * (E * 32) + lane * E;
        uint32_t c[(E + 3) / 4] = {};  // the lane's E codes, little-endian in words
#pragma unroll
        for (int k = 0; k < E; ++k) c[k / 4] |= (uint32_t)float_to_e4m3(v[k] / scale) << (8 * (k % 4));
        if constexpr (E == 16) {
            *reinterpret_cast<uint4*>(dst) = make_uint4(c[0], c[1], c[2], c[3]);
        } else if constexpr (E == 4) {
            *reinterpret_cast<uint32_t*>(dst) = c[0];
        } else {
            *reinterpret_cast<uint16_t*>(dst) = (uint16_t)c[0];
        }
        if (lane == 0) pool.scale[prow] = scale;
    } else if (pool.dtype == DSA_FP4_E2M1) {  // e2m1 codes, two per byte, scale amax / 6
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < E; ++k) amax = fmaxf(amax, fabsf(v[k]));
        amax = warp_max(amax);
        const float scale = amax > 0.f ? amax / 6.f : 1.f;
        uint8_t* dst = reinterpret_cast<uint8_t*>(pool.data) + prow * (E * 16) + lane * (E / 2);
        uint32_t c[(E / 2 + 3) / 4] = {};  // the lane's E/2 code bytes, little-endian in words
#pragma unroll
        for (int k = 0; k < E / 2; ++k)
            c[k / 4] |= (uint32_t)float2_to_e2m1x2(v[2 * k] / scale, v[2 * k + 1] / scale) << (8 * (k % 4));
        if constexpr (E == 16) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
        } else if constexpr (E == 4) {
            *reinterpret_cast<uint16_t*>(dst) = (uint16_t)c[0];
        } else {
            *dst = (uint8_t)c[0];
        }
        if (lane == 0) pool.scale[prow] = scale;
    } else {
        if constexpr (E == kFp4Block) {  // a lane holds one block
            float inv_s, s;
            fp4_block_row_scale(warp_abs_max_bits(lane_abs_max_bits<E>(v)), &s, &inv_s);
            uint32_t c[2];
            const uint8_t bs = fp4_block_codes(v, __uint_as_float(lane_abs_max_bits<E>(v)), inv_s, c);
            store_fp4_block_row(pool, prow, lane, c, bs, s);
        }
    }
}

}  // namespace dsa
