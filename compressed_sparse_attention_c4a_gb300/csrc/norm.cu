// dsa_norm_q8: the residual's addition, the RMS norm and the 8-bit rows that a projection reads, in one pass.
//
//     h = x + residual,   v = gamma h / sqrt(mean(h^2) + eps),   scale_b = max |v| of 128 values / 448,   code = e4m3(v / scale)
//
// [P2] "DeepSeek V4 稀疏注意力完全解剖" 融合点 1 names the norm of the layer, 第四层 the fusing of adjacent steps; the rows are
// those that the pages' fp8 projections take (融合点 2).  The sum h stays in fp32 for the norm and is rounded to bf16 once,
// for the residual stream.
//
// A row is read once and held in registers: eight consecutive values a thread and step, so that sixteen lanes hold a block
// and find its largest value by shuffles.  A warp takes a row of up to 1024 values, a CTA longer ones.
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

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}

// W warps to a row, V steps of 8 values a thread.  W == 1: eight rows to a CTA of eight warps.
template <int W, int V, bool RES>
__global__ void __launch_bounds__(W == 1 ? 256 : 32 * W) norm_q8_kernel(NormArgs a) {
    __shared__ float red[3][W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = W == 1 ? lane : (int)threadIdx.x;
    const int vecs = a.dim / 8, blocks = row_blocks(a.dim);
    const long long step = (long long)gridDim.x * (W == 1 ? 8 : 1);
    float g[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = t + i * 32 * W;
        if (c < vecs && a.gamma) {
            const float4 p = __ldg(reinterpret_cast<const float4*>(a.gamma) + 2 * c);
            const float4 q = __ldg(reinterpret_cast<const float4*>(a.gamma) + 2 * c + 1);
            g[i][0] = p.x, g[i][1] = p.y, g[i][2] = p.z, g[i][3] = p.w;
            g[i][4] = q.x, g[i][5] = q.y, g[i][6] = q.z, g[i][7] = q.w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) g[i][k] = 1.f;
        }
    }
    pdl_wait();
    pdl_launch_dependents();
    int turn = 0;
    for (long long row = W == 1 ? (long long)blockIdx.x * 8 + warp : (long long)blockIdx.x; row < a.n; row += step) {
        const uint4* xr = reinterpret_cast<const uint4*>(a.x + row * a.x_ld);
        uint4 ux[V], ur[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = t + i * 32 * W;
            ux[i] = c < vecs ? xr[c] : make_uint4(0, 0, 0, 0);
            if constexpr (RES)
                ur[i] = c < vecs ? reinterpret_cast<const uint4*>(a.residual + row * a.residual_ld)[c] : make_uint4(0, 0, 0, 0);
        }
        float h[V][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            unpack8(ux[i], h[i]);
            if constexpr (RES) {
                float r[8];
                unpack8(ur[i], r);
#pragma unroll
                for (int k = 0; k < 8; ++k) h[i][k] += r[k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) ss = fmaf(h[i][k], h[i][k], ss);
        }
        if (a.sum) {
            uint4* to = reinterpret_cast<uint4*>(a.sum + row * a.sum_ld);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = t + i * 32 * W;
                if (c < vecs)
                    to[c] = make_uint4(bf16x2(h[i][0], h[i][1]), bf16x2(h[i][2], h[i][3]), bf16x2(h[i][4], h[i][5]),
                                       bf16x2(h[i][6], h[i][7]));
            }
        }
        ss = row_sum<W>(ss, red[turn], warp, lane);
        turn ^= 1;
        float rs;
        if (ss < INFINITY) {
            rs = 1.f / sqrtf(ss / (float)a.dim + a.eps);
        } else {  // squares beyond fp32 (or an infinity, a NaN): the same of h 2^-80, beside which eps is nothing
            float s2 = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    h[i][k] *= 0x1p-80f;
                    s2 = fmaf(h[i][k], h[i][k], s2);
                }
            s2 = row_sum<W>(s2, red[2], warp, lane);
            if constexpr (W > 1) __syncthreads();  // red[2] is free again
            rs = 1.f / sqrtf(s2 / (float)a.dim);
        }
        uint8_t* codes = a.out + row * a.dim;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = t + i * 32 * W;
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                h[i][k] = h[i][k] * rs * g[i][k];
                amax = fmaxf(amax, fabsf(h[i][k]));
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const float scale = block_scale8(amax);
            const BlockQuotient q(scale);
            if (c < vecs) {
                reinterpret_cast<uint2*>(codes)[c] = make_uint2(e4m3x4(q(h[i][0]), q(h[i][1]), q(h[i][2]), q(h[i][3])),
                                                                e4m3x4(q(h[i][4]), q(h[i][5]), q(h[i][6]), q(h[i][7])));
                if ((lane & 15) == 0) a.out_scale[row * blocks + c / 16] = scale;
            }
        }
    }
}

template <bool RES>
static cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
    const long long sms = sm_count();
    const auto grid = [&](long long rows, long long per_sm) {
        return dim3((unsigned)(rows < sms * per_sm ? rows : sms * per_sm));
    };
    if (a.dim <= 1024) {
        const dim3 g = grid((a.n + 7ll) / 8, 8), b(256);
        return a.dim <= 256   ? launch_pdl(norm_q8_kernel<1, 1, RES>, g, b, 0, st, a)
               : a.dim <= 512 ? launch_pdl(norm_q8_kernel<1, 2, RES>, g, b, 0, st, a)
                              : launch_pdl(norm_q8_kernel<1, 4, RES>, g, b, 0, st, a);
    }
    if (a.dim <= 2048) return launch_pdl(norm_q8_kernel<8, 1, RES>, grid(a.n, 8), dim3(256), 0, st, a);
    if (a.dim <= 4096) return launch_pdl(norm_q8_kernel<8, 2, RES>, grid(a.n, 4), dim3(256), 0, st, a);
    if (a.dim <= 8192) return launch_pdl(norm_q8_kernel<8, 4, RES>, grid(a.n, 2), dim3(256), 0, st, a);
    return launch_pdl(norm_q8_kernel<16, 4, RES>, grid(a.n, 1), dim3(512), 0, st, a);
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
