// dsa_gemm_q8: products of 8-bit rows with 8-bit weights, both with a scale per block of 128, on the tensor cores.
//
//     out[i][g][j] = sum_b sa[i][g][b] sw[g][j / 128][b] * (sum_{k in block b} a[i][g][k] w[g][j][k])
//
// [P2] "DeepSeek V4 稀疏注意力完全解剖" 全景图 (the projections around the attention) and 融合点 2 (the attention's output goes
// in fp8 into a batched product, one matrix per group of heads).
//
// The inner sums run in kind::f8f6f4 (fp32 accumulation in TMEM), one accumulator per block of 128; the epilogue warps
// read each, multiply by the two scales' product and add it to sums in fp32 registers.
#include <algorithm>

#include "common.cuh"
#include "rows8.cuh"

namespace dsa {

constexpr int kFeat = 128;       // weight rows of a tile (the MMA's M)
constexpr int kChunk = 8;        // blocks of 128 whose scales are staged together
constexpr int kFewThreads = 192; // warp 0: copies, warp 1: MMA, warps 2-5: sums

enum { kOutF32 = DSA_FP32, kOutBf16 = DSA_BF16, kOutQ8 = DSA_FP8_E4M3 };

struct GemmArgs {
    int m, n, k, groups;
    int nkb, nnb;      // blocks of 128 along k and n
    const float* a_scale;
    long long a_scale_ld;
    const float* w_scale;
    void* out;
    long long out_ld;  // elements between rows
    float* out_scale;
    int format;
    int vec;           // four consecutive outputs may be stored at once
    int splits;        // CTAs of a cluster that share a tile's blocks
    int tiles_n, tiles_m;
    int stages;
    int32_t* status;
    unsigned long long wait_ns;
    int withhold;      // test hook: no copy is issued
};

// 3-D tiled tensor copy global -> shared with the tensor map's swizzle.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// K-major operand of 128-byte rows in the 128-byte swizzle (8-row atoms, 1024 bytes apart).
__device__ __forceinline__ uint64_t rows128_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// kind::f8f6f4, D fp32, A and B e4m3 and K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// A wait of at most wait_ns; when it expires, or another role has given up, false.
__device__ __forceinline__ bool wait_or_stop(uint64_t* bar, uint32_t parity, volatile int* stop, const GemmArgs& a) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*stop) return false;
        if (global_ns() - t0 > a.wait_ns) {
            *stop = 1;
            report(a.status, DSA_ERR_TIMEOUT);
            return false;
        }
    }
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Four consecutive outputs (features j0 + 4 lane ..) of row i, group g, by a warp that holds the 128 features of a block.
__device__ __forceinline__ void store_block(const GemmArgs& a, int i, int g, int nb, int lane, float4 v) {
    const int j = nb * kFeat + 4 * lane, left = a.n - j;
    const long long at = (long long)i * a.out_ld + (long long)g * a.n + j;
    if (a.format == kOutQ8) {
        float x[4] = {v.x, v.y, v.z, v.w}, amax = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, e < left ? fabsf(x[e]) : 0.f);
        amax = warp_max(amax);
        const float scale = block_scale8(amax);
        const BlockQuotient q(scale);
        const uint32_t c = e4m3x4(q(x[0]), q(x[1]), q(x[2]), q(x[3]));
        uint8_t* to = static_cast<uint8_t*>(a.out) + at;
        if (a.vec && left >= 4) *reinterpret_cast<uint32_t*>(to) = c;
        else
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left) to[e] = (uint8_t)(c >> (8 * e));
        if (lane == 0) a.out_scale[((long long)i * a.groups + g) * a.nnb + nb] = scale;
    } else if (a.format == kOutBf16) {
        uint16_t* to = static_cast<uint16_t*>(a.out) + at;
        const uint2 u = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
        if (a.vec && left >= 4) *reinterpret_cast<uint2*>(to) = u;
        else {
            if (left > 0) to[0] = (uint16_t)u.x;
            if (left > 1) to[1] = (uint16_t)(u.x >> 16);
            if (left > 2) to[2] = (uint16_t)u.y;
            if (left > 3) to[3] = (uint16_t)(u.y >> 16);
        }
    } else {
        float* to = static_cast<float*>(a.out) + at;
        if (a.vec && left >= 4) *reinterpret_cast<float4*>(to) = v;
        else {
            if (left > 0) to[0] = v.x;
            if (left > 1) to[1] = v.y;
            if (left > 2) to[2] = v.z;
            if (left > 3) to[3] = v.w;
        }
    }
}

template <int BN>
__host__ __device__ constexpr int few_stage_bytes() { return kFeat * 128 + BN * 128; }
template <int BN>
__host__ __device__ constexpr int few_accumulators() { return BN >= 128 ? 2 : 4; }

// Tile: 128 weight rows x BN rows of a.  The MMA's M is the weights' side, so that few rows of a cost few columns.  A tile's
// blocks of 128 along k are shared by the CTAs of a cluster, whose sums are added in rank order.
template <int BN>
__global__ void __launch_bounds__(kFewThreads) gemm_q8_few_kernel(const __grid_constant__ CUtensorMap wmap,
                                                                  const __grid_constant__ CUtensorMap amap, const GemmArgs a) {
    constexpr int NA = few_accumulators<BN>();
    constexpr uint32_t kStage = few_stage_bytes<BN>();
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    float* part = reinterpret_cast<float*>(base);  // [BN][128], in the stages once they are done with
    float* scales = reinterpret_cast<float*>(base + a.stages * kStage);  // [2][kChunk][BN]
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + 2 * kChunk * BN);
    uint64_t* empty = full + a.stages;
    uint64_t* acc_full = empty + a.stages;
    uint64_t* acc_empty = acc_full + NA;
    uint64_t* drained = acc_empty + NA;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
    volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x % a.splits);
    int tile = (int)(blockIdx.x / a.splits);
    const int tm = tile % a.tiles_m;
    tile /= a.tiles_m;
    const int nb = tile % a.tiles_n, g = tile / a.tiles_n;
    const int row0 = tm * BN;
    const int kb0 = (int)((long long)a.nkb * rank / a.splits), kb1 = (int)((long long)a.nkb * (rank + 1) / a.splits);

    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        mbar_init(drained, 1);
        *stop = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, NA * BN < 32 ? 32 : NA * BN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // Copies.  The weights do not come from the preceding kernel: those of the first stages are requested before the wait.
        if (lane == 0 && !a.withhold) {
            const int ahead = min(a.stages, kb1 - kb0);
            for (int i = 0; i < ahead; ++i) {
                const uint32_t st = smem_u32(base) + i * kStage;
                mbar_arrive_expect_tx(&full[i], kStage);
                tma_load_3d(st, &wmap, (kb0 + i) * 128, nb * kFeat, g, smem_u32(&full[i]));
            }
            pdl_wait();
            pdl_launch_dependents();
            for (int i = 0; i < ahead; ++i)
                tma_load_3d(smem_u32(base) + i * kStage + kFeat * 128, &amap, (kb0 + i) * 128, g, row0, smem_u32(&full[i]));
            int s = 0;
            uint32_t ph = 0;
            int issued = ahead;
            for (int kb = kb0 + ahead; kb < kb1; ++kb) {
                if (!wait_or_stop(&empty[s], ph, stop, a)) break;
                const uint32_t st = smem_u32(base) + s * kStage;
                mbar_arrive_expect_tx(&full[s], kStage);
                tma_load_3d(st, &wmap, kb * 128, nb * kFeat, g, smem_u32(&full[s]));
                tma_load_3d(st + kFeat * 128, &amap, kb * 128, g, row0, smem_u32(&full[s]));
                ++issued;
                if (++s == a.stages) s = 0, ph ^= 1;
            }
            // no copy is left in flight: the last fill of each stage has landed (an expired wait must not leave one behind)
            for (int i = max(0, issued - a.stages); i < issued; ++i)
                mbar_wait_bounded(&full[i % a.stages], (uint32_t)(i / a.stages) & 1, kWaitLimitNs);
        } else {
            pdl_wait();
        }
    } else if (warp == 1) {
        pdl_wait();
        constexpr uint32_t idesc = idesc_e4m3(kFeat, BN);
        int s = 0, b = 0;
        uint32_t ph = 0, aph = 1;
        for (int kb = kb0; kb < kb1; ++kb) {
            const bool ok = wait_or_stop(&full[s], ph, stop, a) && wait_or_stop(&acc_empty[b], aph, stop, a);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const uint32_t st = smem_u32(base) + s * kStage;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_f8_elect(tmem + b * BN, rows128_desc(st + ks * 32), rows128_desc(st + kFeat * 128 + ks * 32), idesc,
                             ks > 0 ? 1u : 0u);
            mma_commit_elect(&empty[s]);
            mma_commit_elect(&acc_full[b]);
            if (++s == a.stages) s = 0, ph ^= 1;
            if (++b == NA) b = 0, aph ^= 1;
        }
        mma_commit_elect(drained);
        mbar_wait_bounded(drained, 0, kWaitLimitNs);
        __syncwarp();
    } else {
        pdl_wait();
        const int t = threadIdx.x - 64;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        float acc[BN];
#pragma unroll
        for (int j = 0; j < BN; ++j) acc[j] = 0.f;
        // the products of scales of block kb0 + chunk * 8 + e % 8 and row e / 8, e = t, t + 128 ..
        constexpr int PER = BN * kChunk / 128;
        float next[PER];
        const float* sa = a.a_scale + (long long)g * a.nkb;
        const float* sw = a.w_scale + ((long long)g * a.nnb + nb) * a.nkb;
        const auto fetch = [&](int kb) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = t + 128 * i, row = row0 + e / kChunk, b = kb + e % kChunk;
                next[i] = row < a.m && b < kb1 ? sa[(long long)row * a.a_scale_ld + b] * __ldg(sw + b) : 0.f;
            }
        };
        fetch(kb0);
        int b = 0;
        uint32_t aph = 0;
        bool live = true;  // a warp whose wait expired still takes part in the barriers below
        for (int kb = kb0; kb < kb1; ++kb) {
            const int c = (kb - kb0) % kChunk;
            float* sc = scales + ((kb - kb0) / kChunk & 1) * kChunk * BN;
            if (c == 0) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int e = t + 128 * i;
                    sc[(e % kChunk) * BN + e / kChunk] = next[i];
                }
                named_bar_sync(1, 128);
                fetch(kb + kChunk);
            }
            live = live && __all_sync(0xffffffffu, wait_or_stop(&acc_full[b], aph, stop, a));
            if (!live) continue;
            tc_fence_after();
            const float4* s4 = reinterpret_cast<const float4*>(sc + c * BN);
#pragma unroll
            for (int j0 = 0; j0 < BN; j0 += 16) {
                float p[16];
                tmem_ld16(tmem + b * BN + lanes + j0, p);
                if (j0 + 16 == BN) {
                    tc_fence_before();
                    if (lane == 0) mbar_arrive(&acc_empty[b]);
                }
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 f = s4[(j0 + j) / 4];
                    acc[j0 + j] = fmaf(p[j], f.x, acc[j0 + j]);
                    acc[j0 + j + 1] = fmaf(p[j + 1], f.y, acc[j0 + j + 1]);
                    acc[j0 + j + 2] = fmaf(p[j + 2], f.z, acc[j0 + j + 2]);
                    acc[j0 + j + 3] = fmaf(p[j + 3], f.w, acc[j0 + j + 3]);
                }
            }
            if (++b == NA) b = 0, aph ^= 1;
        }
        // the last accumulator was complete, so the stages have been read
        const int feat = 32 * (warp & 3) + lane;
#pragma unroll
        for (int j = 0; j < BN; ++j) part[j * 128 + feat] = acc[j];
    }
    __syncwarp();
    if (a.splits > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    bool failed = false;
    for (int r = 0; r < a.splits; ++r) failed |= ld_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(stop)), r)) != 0u;
    for (int j = rank + a.splits * warp; j < BN && row0 + j < a.m; j += a.splits * (kFewThreads / 32)) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        const uint32_t at = smem_u32(part + j * 128 + 4 * lane);
        for (int r = 0; r < a.splits; ++r) {
            const float4 p = ld_cluster_v4(mapa_shared(at, r));
            v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
        }
        if (failed) v = make_float4(0.f, 0.f, 0.f, 0.f);
        store_block(a, row0 + j, g, nb, lane, v);
    }
    if (a.splits > 1) {  // the others may still read this CTA's sums
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == 1) tmem_dealloc(tmem, NA * BN < 32 ? 32 : NA * BN);
}

// ---- host ----------------------------------------------------------------------------------------------------------
struct GemmPlan {
    int rows;    // rows of a in a tile
    int splits;  // CTAs that share a tile's blocks of k
};

static GemmPlan plan_gemm(int m, int n, int k, int groups) {
    GemmPlan p{};
    p.rows = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
    const long long tiles = (long long)groups * row_blocks(n) * ((m + p.rows - 1) / p.rows);
    const int nkb = row_blocks(k);
    p.splits = 1;
    while (p.splits < 8 && tiles * p.splits * 2 <= 2ll * sm_count() && nkb >= 4 * p.splits) p.splits *= 2;
    return p;
}

// Codes [z][y][x] (x contiguous) in boxes of 128 x values and `rows` of the dimension `box_dim`, one of the other.
static bool make_codes_map(CUtensorMap* map, const void* base, long long x, long long y, long long z, long long y_stride,
                           long long z_stride, int box_y, int box_z) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t dim[3] = {(cuuint64_t)x, (cuuint64_t)y, (cuuint64_t)z};
    const cuuint64_t stride[2] = {(cuuint64_t)y_stride, (cuuint64_t)z_stride};
    const cuuint32_t box[3] = {128, (cuuint32_t)box_y, (cuuint32_t)box_z}, one[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dim, stride, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN>
static dsa_status_t launch_few(const CUtensorMap& wmap, const CUtensorMap& amap, GemmArgs a, cudaStream_t st) {
    // two CTAs an SM where their accumulators and a few stages fit
    constexpr int extra = 1024 + 2 * kChunk * BN * 4 + 512;
    constexpr int budget = BN <= 32 ? 228 * 1024 / 2 - 1024 : 227 * 1024;
    a.stages = std::max(2, std::min(12, (budget - extra) / few_stage_bytes<BN>()));
    const int smem = extra + a.stages * few_stage_bytes<BN>();
    static_assert(2 * few_stage_bytes<BN>() >= BN * 512 || BN == 128, "the sums fit into the stages");
    if (cudaFuncSetAttribute(gemm_q8_few_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return DSA_ERR_CUDA;
    const long long grid = (long long)a.groups * a.tiles_n * a.tiles_m * a.splits;
    if (grid > 0x7fffffff) return DSA_ERR_UNSUPPORTED;
    if (launch_pdl_cluster(gemm_q8_few_kernel<BN>, dim3((unsigned)grid), dim3(kFewThreads), smem, st, a.splits, wmap, amap,
                           a) != cudaSuccess)
        return DSA_ERR_CUDA;
    return launch_status();
}

static dsa_status_t check_gemm(int32_t m, int32_t n, int32_t k, int32_t groups) {
    if (m < 0 || n <= 0 || k <= 0 || groups <= 0) return DSA_ERR_INVALID_ARG;
    if (k % 16 || (long long)n * k >= (1ll << 40) || n > 0x7fffff00 || k > 0x7fffff00 || m > 0x7fffff00)
        return DSA_ERR_UNSUPPORTED;
    return DSA_OK;
}

static dsa_status_t gemm_q8(int32_t m, int32_t n, int32_t k, int32_t groups, const uint8_t* a, int64_t a_ld,
                            const float* a_scale, int64_t a_scale_ld, const uint8_t* w, const float* w_scale,
                            int32_t out_format, void* out, int64_t out_ld, float* out_scale, uint64_t wait_ns, int withhold,
                            int32_t* dev_status, void* stream) {
    const dsa_status_t e = check_gemm(m, n, k, groups);
    if (e != DSA_OK) return e;
    if (out_format != kOutF32 && out_format != kOutBf16 && out_format != kOutQ8) return DSA_ERR_INVALID_ARG;
    if (m == 0) return DSA_OK;
    const int size = out_format == kOutF32 ? 4 : out_format == kOutBf16 ? 2 : 1;
    const int nkb = row_blocks(k), nnb = row_blocks(n);
    if (!a || !a_scale || !w || !w_scale || !out || !aligned(a, 16) || !aligned(w, 16) || !aligned(a_scale, 4) ||
        !aligned(w_scale, 4) || !aligned(out, size) || (out_format == kOutQ8 && (!out_scale || !aligned(out_scale, 4))))
        return DSA_ERR_INVALID_ARG;
    if (a_ld % 16 || a_ld < (long long)groups * k || a_scale_ld < (long long)groups * nkb ||
        out_ld < (long long)groups * n)
        return DSA_ERR_INVALID_ARG;
    if (a_ld >= (1ll << 40) || a_scale_ld >= (1ll << 40) || out_ld >= (1ll << 40)) return DSA_ERR_UNSUPPORTED;
    const GemmPlan p = plan_gemm(m, n, k, groups);
    GemmArgs args{};
    args.m = m, args.n = n, args.k = k, args.groups = groups, args.nkb = nkb, args.nnb = nnb;
    args.a_scale = a_scale, args.a_scale_ld = a_scale_ld, args.w_scale = w_scale;
    args.out = out, args.out_ld = out_ld, args.out_scale = out_scale, args.format = out_format;
    args.vec = aligned(out, 4 * size) && out_ld % 4 == 0 && (groups == 1 || n % 4 == 0);
    args.splits = p.splits, args.tiles_n = nnb, args.tiles_m = (m + p.rows - 1) / p.rows;
    args.status = dev_status, args.wait_ns = wait_ns, args.withhold = withhold;
    CUtensorMap wmap, amap;
    if (!make_codes_map(&wmap, w, k, n, groups, k, (long long)n * k, kFeat, 1) ||
        !make_codes_map(&amap, a, k, groups, m, k, a_ld, 1, p.rows))
        return DSA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (p.rows) {
        case 16: return launch_few<16>(wmap, amap, args, st);
        case 32: return launch_few<32>(wmap, amap, args, st);
        case 64: return launch_few<64>(wmap, amap, args, st);
        default: return launch_few<128>(wmap, amap, args, st);
    }
}

}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_gemm_q8(int32_t m, int32_t n, int32_t k, int32_t groups, const uint8_t* a, int64_t a_ld,
                                    const float* a_scale, int64_t a_scale_ld, const uint8_t* w, const float* w_scale,
                                    int32_t out_format, void* out, int64_t out_ld, float* out_scale, int32_t* dev_status,
                                    void* stream) {
    return gemm_q8(m, n, k, groups, a, a_ld, a_scale, a_scale_ld, w, w_scale, out_format, out, out_ld, out_scale, kWaitLimitNs,
                   0, dev_status, stream);
}

extern "C" dsa_status_t dsa_debug_gemm_q8_stalled(int32_t m, int32_t n, int32_t k, int32_t groups, const uint8_t* a,
                                                  int64_t a_ld, const float* a_scale, int64_t a_scale_ld, const uint8_t* w,
                                                  const float* w_scale, int32_t out_format, void* out, int64_t out_ld,
                                                  float* out_scale, uint64_t wait_limit_ns, int32_t* dev_status,
                                                  void* stream) {
    if (wait_limit_ns < 1 || wait_limit_ns > 2000000000ull) return DSA_ERR_INVALID_ARG;
    return gemm_q8(m, n, k, groups, a, a_ld, a_scale, a_scale_ld, w, w_scale, out_format, out, out_ld, out_scale, wait_limit_ns,
                   1, dev_status, stream);
}

extern "C" dsa_status_t dsa_gemm_q8_plan(int32_t m, int32_t n, int32_t k, int32_t groups, int32_t* plan) {
    if (!plan || m == 0) return DSA_ERR_INVALID_ARG;
    const dsa_status_t e = check_gemm(m, n, k, groups);
    if (e != DSA_OK) return e;
    const GemmPlan p = plan_gemm(m, n, k, groups);
    plan[0] = kFeat, plan[1] = p.rows, plan[2] = p.splits;
    return DSA_OK;
}
