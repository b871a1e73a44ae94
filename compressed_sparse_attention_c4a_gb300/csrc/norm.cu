// dsa_norm_q8: the residual's addition, the RMS norm and the 8-bit rows that a projection reads, in one pass.
//
//     h = x + residual,   v = gamma h / sqrt(mean(h^2) + eps),   scale_b = max |v| of 128 values / 448,   code = e4m3(v / scale)
//
// [P2] "DeepSeek V4 稀疏注意力完全解剖" 融合点 1 names the norm of the layer, 第四层 the fusing of adjacent steps; the rows are
// those that the pages' fp8 projections take (融合点 2).  The sum h stays in fp32 for the norm and is rounded to bf16 once,
// for the residual stream.
//
// A row is read once and held in registers: eight consecutive values a thread and step, so that sixteen lanes hold a block
// and find its largest value by shuffles.  A warp takes a row of up to 1024 values, a CTA longer ones.  CTAs go from row to row,
// the next rows on their way into shared memory, each thread waiting for the pieces that it copied itself.
// The call has no status word: in the bounds-checked build a bad index leaves its access out, which the values show.
#include <algorithm>

#include "common.cuh"
#include "rows8.cuh"

namespace dsa {

struct NormArgs {
    int n, dim;
    const uint16_t* x;
    const uint16_t* residual;
    long long x_ld, residual_ld, sum_ld;
    const float* gamma;
    float eps;
    uint16_t* sum;
    uint8_t* out;
    float* out_scale;
};

// Sum over the CTA's warps (W == 1: over the warp).  `red`: two sets of W slots, taken in turn so that one barrier a sum
// is enough.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red, int warp, int lane) {
    v = warp_sum(v);
    if constexpr (W == 1) return v;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) t += red[i];
    return t;
}

constexpr int kNormAhead = 2;  // rows on their way

// W warps to a row, V steps of 8 values a thread, C CTAs to an SM.  W == 1: eight rows to a CTA of eight warps.
template <int W, int V, int C, bool RES>
__global__ void __launch_bounds__(W == 1 ? 256 : 32 * W, C) norm_q8_kernel(NormArgs a) {
    extern __shared__ uint4 ring[];  // [warps or 1][kNormAhead][x, residual][vecs]
    __shared__ float red[3][W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = W == 1 ? lane : (int)threadIdx.x;
    const int vecs = a.dim / 8, blocks = row_blocks(a.dim), slot_vecs = vecs * (RES ? 2 : 1);
    const long long step = (long long)gridDim.x * (W == 1 ? 8 : 1);
    uint4* const mine = ring + (W == 1 ? warp * kNormAhead * slot_vecs : 0);
    uint64_t g[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = t + i * 32 * W;
        if (c < vecs && a.gamma) {
            const float4 p = __ldg(reinterpret_cast<const float4*>(a.gamma) + 2 * c);
            const float4 q = __ldg(reinterpret_cast<const float4*>(a.gamma) + 2 * c + 1);
            g[i][0] = pair2(p.x, p.y), g[i][1] = pair2(p.z, p.w), g[i][2] = pair2(q.x, q.y), g[i][3] = pair2(q.z, q.w);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) g[i][k] = pair2(1.f, 1.f);
        }
    }
    const auto request = [&](long long row, int slot) {  // a group of copies, empty behind the last row
        if (row < a.n) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = t + i * 32 * W;
                if (c < vecs && DSA_IDX_OK(slot * slot_vecs + (RES ? vecs : 0) + c, kNormAhead * slot_vecs, nullptr)) {
                    cp_async16_nc(smem_u32(mine + slot * slot_vecs + c), reinterpret_cast<const uint4*>(a.x + row * a.x_ld) + c, 16);
                    if constexpr (RES)
                        cp_async16_nc(smem_u32(mine + slot * slot_vecs + vecs + c),
                                      reinterpret_cast<const uint4*>(a.residual + row * a.residual_ld) + c, 16);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    pdl_wait();
    pdl_launch_dependents();
    long long row = W == 1 ? (long long)blockIdx.x * 8 + warp : (long long)blockIdx.x;
#pragma unroll
    for (int i = 0; i < kNormAhead; ++i) request(row + i * step, i);
    int turn = 0, slot = 0;
    for (; row < a.n; row += step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kNormAhead - 1) : "memory");
        uint64_t h[V][4], s2 = 0ull;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = t + i * 32 * W;
            const uint4 u = c < vecs ? mine[slot * slot_vecs + c] : make_uint4(0, 0, 0, 0);
            h[i][0] = pair_of_bf16(u.x), h[i][1] = pair_of_bf16(u.y), h[i][2] = pair_of_bf16(u.z), h[i][3] = pair_of_bf16(u.w);
            if constexpr (RES) {
                const uint4 r = c < vecs ? mine[slot * slot_vecs + vecs + c] : make_uint4(0, 0, 0, 0);
                h[i][0] = add2(h[i][0], pair_of_bf16(r.x)), h[i][1] = add2(h[i][1], pair_of_bf16(r.y));
                h[i][2] = add2(h[i][2], pair_of_bf16(r.z)), h[i][3] = add2(h[i][3], pair_of_bf16(r.w));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) s2 = fma2(h[i][k], h[i][k], s2);
        }
        request(row + kNormAhead * step, slot);
        if (++slot == kNormAhead) slot = 0;
        if (a.sum) {
            uint4* to = reinterpret_cast<uint4*>(a.sum + row * a.sum_ld);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = t + i * 32 * W;
                if (c < vecs)
                    to[c] = make_uint4(bf16x2(lo_of(h[i][0]), hi_of(h[i][0])), bf16x2(lo_of(h[i][1]), hi_of(h[i][1])),
                                       bf16x2(lo_of(h[i][2]), hi_of(h[i][2])), bf16x2(lo_of(h[i][3]), hi_of(h[i][3])));
            }
        }
        const float ss = row_sum<W>(lo_of(s2) + hi_of(s2), red[turn], warp, lane);
        turn ^= 1;
        // The norm's factor is one for the row: a block's codes are those of gamma h whatever it is, its scale has it.  Rows of
        // huge or tiny values (an infinity, a NaN) take it first: gamma times them could leave fp32 where the norm does not.
        float rs = 1.f / sqrtf(ss / (float)a.dim + a.eps);
        if (!(rs > 0x1p-20f && rs < 0x1p20f)) {
            if (!(ss < INFINITY)) {  // squares beyond fp32: those of h 2^-80, beside which eps is nothing
                s2 = 0ull;
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint64_t u = mul2(h[i][k], pair2(0x1p-80f, 0x1p-80f));
                        s2 = fma2(u, u, s2);
                        h[i][k] = mul2(h[i][k], pair2(0x1p-40f, 0x1p-40f));  // the rest is rs's: small values keep their bits
                    }
                const float again = row_sum<W>(lo_of(s2) + hi_of(s2), red[2], warp, lane);
                if constexpr (W > 1) __syncthreads();  // red[2] is free again
                rs = 0x1p-40f / sqrtf(again / (float)a.dim);
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) h[i][k] = mul2(h[i][k], pair2(rs, rs));
            rs = 1.f;
        }
        uint8_t* codes = a.out + row * a.dim;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = t + i * 32 * W;
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h[i][k] = mul2(h[i][k], g[i][k]);
                amax = fmaxf(amax, fmaxf(fabsf(lo_of(h[i][k])), fabsf(hi_of(h[i][k]))));
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            float scale;
            if (amax > 0x1p-60f && amax < 0x1p60f) {  // the scale is above 2^-89
                const float r = 448.f * near_reciprocal(amax);
                scale = amax * rs * (1.f / 448.f);
#pragma unroll
                for (int k = 0; k < 4; ++k) h[i][k] = mul2(h[i][k], pair2(r, r));
            } else {  // parts of which could leave fp32's normal range; NaN and infinities
                amax = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    h[i][k] = mul2(h[i][k], pair2(rs, rs));
                    amax = fmaxf(amax, fmaxf(fabsf(lo_of(h[i][k])), fabsf(hi_of(h[i][k]))));
                }
                const unsigned half = lane < 16 ? 0xffffu : 0xffff0000u;
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(half, amax, o));
                scale = block_scale8(amax);
                const BlockQuotient2 q(scale);
#pragma unroll
                for (int k = 0; k < 4; ++k) h[i][k] = q(h[i][k]);
            }
            if (c < vecs && DSA_IDX_OK(row * vecs + c, (long long)a.n * vecs, nullptr)) {
                reinterpret_cast<uint2*>(codes)[c] = make_uint2(e4m3x4(h[i][0], h[i][1]), e4m3x4(h[i][2], h[i][3]));
                if ((lane & 15) == 0 && DSA_IDX_OK(c / 16, blocks, nullptr)) a.out_scale[row * blocks + c / 16] = scale;
            }
        }
    }
}

template <int W, int V, int C, bool RES>
static cudaError_t launch_rows(const NormArgs& a, cudaStream_t st) {
    const int rows = W == 1 ? 8 : 1, smem = rows * kNormAhead * a.dim * 2 * (RES ? 2 : 1);
    if (smem > 48 * 1024 &&  // what a kernel may have unasked
        cudaFuncSetAttribute(norm_q8_kernel<W, V, C, RES>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return cudaErrorInvalidValue;
    const long long grid = std::min<long long>((a.n + rows - 1ll) / rows, (long long)sm_count() * C);
    return launch_pdl(norm_q8_kernel<W, V, C, RES>, dim3((unsigned)grid), dim3(W == 1 ? 256 : 32 * W), smem, st, a);
}

// What bounds it: HBM with a residual (7 bytes a value: 8,192 rows of 8,192 in 73.1 us, 6.5 TB/s, 0.96 of the copy rate; of
// 4,096 38.0, 16,384 of 2,048 39.3, 32,768 of 512 21.5).  Without one (3 bytes a value: 40.2, 22.9, 22.5, 12.2) neither HBM (51 %
// at 8,192 values a row) nor the issue slots (56 %): sixteen warps an SM (their rows in 116 registers a thread) wait for shuffles
// and shared memory (1.8 of 6.9 cycles a warp's instruction) and for results of fixed latency (1.6).  Warps to a row, steps and
// CTAs an SM were chosen at these sizes: rows of 8,192 with a residual by eight warps in two CTAs took 83.7 us where sixteen in
// one took 72.2; without one 41.3 and 51.4.  Loaded into registers instead of copied ahead, the first took 106.
template <bool RES>
static cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
    if (a.dim <= 256) return launch_rows<1, 1, 4, RES>(a, st);
    if (a.dim <= 512) return launch_rows<1, 2, 3, RES>(a, st);
    if (a.dim <= 1024) return launch_rows<1, 4, 2, RES>(a, st);
    if (a.dim <= 2048) return launch_rows<RES ? 8 : 4, RES ? 1 : 2, RES ? 4 : 6, RES>(a, st);
    if (a.dim <= 4096) return launch_rows<8, 2, RES ? 2 : 3, RES>(a, st);
    if (a.dim <= 8192) return launch_rows<RES ? 16 : 8, RES ? 2 : 4, RES ? 1 : 2, RES>(a, st);
    return launch_rows<16, 4, 1, RES>(a, st);
}

}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_norm_q8(int32_t n, int32_t dim, const void* x, int64_t x_ld, const void* residual,
                                    int64_t residual_ld, const float* gamma, float eps, void* sum, int64_t sum_ld,
                                    uint8_t* out, float* out_scale, void* stream) {
    if (n < 0 || dim <= 0) return DSA_ERR_INVALID_ARG;
    if (n == 0) return DSA_OK;
    if (dim % 16 || dim > 16384) return DSA_ERR_UNSUPPORTED;
    const auto rows_ok = [&](const void* p, int64_t ld) {
        return aligned(p, 16) && ld % 8 == 0 && (ld >= dim || n == 1) && ld >= 0 && ld <= (1ll << 40);
    };
    if (!x || !rows_ok(x, x_ld) || (residual && !rows_ok(residual, residual_ld)) || (sum && !rows_ok(sum, sum_ld)) ||
        !aligned(gamma, 16) || !(eps > 0.f) || !(eps < __builtin_inff()) || !out || !aligned(out, 16) || !out_scale ||
        !aligned(out_scale, 4))
        return DSA_ERR_INVALID_ARG;
    const NormArgs a{n, dim, static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(residual), x_ld, residual_ld,
                     sum_ld, gamma, eps, static_cast<uint16_t*>(sum), out, out_scale};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((residual ? launch_norm<true>(a, st) : launch_norm<false>(a, st)) != cudaSuccess) return DSA_ERR_CUDA;
    return launch_status();
}
