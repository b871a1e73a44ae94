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

// One block: its e4m3 scale (returned) and 16 codes (element 2j in the low nibble).  v / (s bs) is a reciprocal and one
// correction step, which gives the quotient itself wherever that is representable (the borders are).
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
    return bs8;
}

// ---- rows ------------------------------------------------------------------------------------------------------
// A warp owns a row, each lane E = dim / 32 consecutive elements.
template <int E>
__device__ __forceinline__ void load_bf16(const uint16_t* row, int lane, float (&v)[E]) {
    const uint16_t* p = row + lane * E;
    if constexpr (E == 16) {
        uint4 a = *reinterpret_cast<const uint4*>(p);
        uint4 b = *reinterpret_cast<const uint4*>(p + 8);
        uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[2 * k] = __uint_as_float(u[k] << 16);
            v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
        }
    } else if constexpr (E == 4) {
        uint2 a = *reinterpret_cast<const uint2*>(p);
        v[0] = __uint_as_float(a.x << 16);
        v[1] = __uint_as_float(a.x & 0xffff0000u);
        v[2] = __uint_as_float(a.y << 16);
        v[3] = __uint_as_float(a.y & 0xffff0000u);
    } else {
        static_assert(E == 2, "row width");
        uint32_t a = *reinterpret_cast<const uint32_t*>(p);
        v[0] = __uint_as_float(a << 16);
        v[1] = __uint_as_float(a & 0xffff0000u);
    }
}

// Store one row (the warp's E values per lane) into a pool row: bf16, e4m3 + amax/448 scale, e2m1 + amax/6, or e2m1
// with a scale per block of 16 (rows of 512 only).
template <int E>
__device__ __forceinline__ void store_row(const dsa_pool_t& pool, long long prow, int lane, const float (&v)[E]) {
    if (pool.dtype == DSA_BF16) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(pool.data) + prow * (E * 32) + lane * E;
        uint32_t u[E / 2];
#pragma unroll
        for (int k = 0; k < E / 2; ++k)
            u[k] = (uint32_t)float_to_bf16(v[2 * k]) | ((uint32_t)float_to_bf16(v[2 * k + 1]) << 16);
        if constexpr (E == 16) {
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(u[0], u[1], u[2], u[3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(u[4], u[5], u[6], u[7]);
        } else if constexpr (E == 4) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[1]);
        } else {
            *reinterpret_cast<uint32_t*>(dst) = u[0];
        }
    } else if (pool.dtype == DSA_FP4_BLOCK) {
        if constexpr (E == kFp4Block) {  // a lane holds one block
            float inv_s, s;
            fp4_block_row_scale(warp_abs_max_bits(lane_abs_max_bits<E>(v)), &s, &inv_s);
            uint32_t c[2];
            const uint8_t bs = fp4_block_codes(v, __uint_as_float(lane_abs_max_bits<E>(v)), inv_s, c);
            uint8_t* dst = reinterpret_cast<uint8_t*>(pool.data) + prow * kFp4BlockRow;
            *reinterpret_cast<uint2*>(dst + lane * 8) = make_uint2(c[0], c[1]);
            dst[256 + lane] = bs;
            if (lane == 0) pool.scale[prow] = s;
        }
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
    }
}

}  // namespace dsa
