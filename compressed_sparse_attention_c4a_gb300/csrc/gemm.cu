// dsa_gemm_q8: products of 8-bit rows with 8-bit weights, both with a scale per block of 128, on the tensor cores.
//
//     out[i][g][j] = sum_b sa[i][g][b] sw[g][j / 128][b] * (sum_{k in block b} a[i][g][k] w[g][j][k])
//
// [P2] "DeepSeek V4 稀疏注意力完全解剖" 全景图 (the projections around the attention) and 融合点 2 (the attention's output goes
// in fp8 into a batched product, one matrix per group of heads).
//
// The inner sums run in kind::f8f6f4 (fp32 accumulation in TMEM), one accumulator per block of 128; warps of sums read each,
// multiply by the two scales' product and add it to sums in fp32 registers.  (The tensor cores can scale by themselves only by
// powers of two per 32 values; these scales are any fp32 number.)
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "rows8.cuh"

namespace dsa {

constexpr int kFeat = 128;       // weight rows of a tile (the MMA's M)
constexpr int kChunk = 8;        // blocks of 128 whose scales are staged together

enum { kOutF32 = DSA_FP32, kOutBf16 = DSA_BF16, kOutQ8 = DSA_FP8_E4M3 };

struct GemmArgs {
    int m, n, k, groups;
    int nkb, nnb;      // blocks of 128 along k and n
    const float* a_scale;
    long long a_scale_ld;
    int a_scale_vec;   // four consecutive scales of a row may be read at once, from multiples of four blocks on
    const float* w_scale;
    void* out;
    long long out_ld;  // elements between rows
    float* out_scale;
    int format;
    int vec;           // 1: four consecutive outputs may be stored at once, 2: 16 bytes
    int whole;         // a row's outputs end on 16 bytes
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
// A descriptor like d with this low word (address, leading offset): an offset within shared memory carries nothing upwards.
__device__ __forceinline__ uint64_t desc_lo(uint64_t d, uint32_t lo) { return (d & 0xffffffff00000000ull) | lo; }
// kind::f8f6f4, D fp32, A and B e4m3 and K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// A wait of at most wait_ns; when it expires, or another role has given up, false.
__device__ __forceinline__ bool wait_or_stop(uint64_t* bar, uint32_t parity, volatile int* stop, const GemmArgs& a) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
#pragma unroll 1
    do {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
    } while (!*stop && global_ns() - t0 <= a.wait_ns);
    if (!*stop) report(a.status, DSA_ERR_TIMEOUT);
    *stop = 1;
    return false;
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

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
        "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// After tmem_wait_ld(): no use of the registers is scheduled before the wait.
__device__ __forceinline__ void regs_after_wait(uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                     "+r"(r[i + 6]), "+r"(r[i + 7]));
}
// acc (two sums) += p (two products) * s (twice the same scale)
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t p0, uint32_t p1, uint64_t s) {
    asm("{\n\t.reg .b64 p;\n\tmov.b64 p, {%1, %2};\n\tfma.rn.f32x2 %0, p, %3, %0;\n\t}" : "+l"(acc) : "r"(p0), "r"(p1), "l"(s));
}

// Four consecutive outputs (features j0 + 4 lane ..) of row i, group g, by a warp that holds the 128 features of a block.
__device__ __forceinline__ void store_block(const GemmArgs& a, int i, int g, int nb, int lane, float4 v) {
    const int j = nb * kFeat + 4 * lane, left = a.n - j;
    const long long at = (long long)i * a.out_ld + (long long)g * a.n + j;
    if (!DSA_IDX_OK(i, a.m, a.status) || !DSA_IDX_OK(nb, a.nnb, a.status) || !DSA_IDX_OK(g, a.groups, a.status)) return;
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
constexpr int kFewThreads = 192;
constexpr int kFewAcc = 4;  // accumulators

// The sums of S CTAs for up to R = 4 / S rows j, j + step .. of the tile, four loads in flight before the first is added (in
// rank order).  What is loaded is added, so no load from another CTA is left in flight.
template <int S>
__device__ __forceinline__ void join_rows(const GemmArgs& a, const float* part, int j, int step, int rows, int row0, int g, int nb,
                                          int lane, bool failed) {
    constexpr int Q = S < 4 ? S : 4, R = 4 / Q;
    const uint32_t at = smem_u32(part + j * 128 + 4 * lane);
    float4 sum[R];
#pragma unroll
    for (int r0 = 0; r0 < S; r0 += Q) {
        float4 v[R][Q];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int r = 0; r < Q; ++r)
                if (i < rows) v[i][r] = ld_cluster_v4(mapa_shared(at + i * step * 512, r0 + r));
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i < rows)
#pragma unroll
                for (int r = 0; r < Q; ++r) {
                    if (r0 + r == 0) sum[i] = v[i][r];
                    else sum[i].x += v[i][r].x, sum[i].y += v[i][r].y, sum[i].z += v[i][r].z, sum[i].w += v[i][r].w;
                }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < rows) store_block(a, row0 + j + i * step, g, nb, lane, failed ? make_float4(0.f, 0.f, 0.f, 0.f) : sum[i]);
}

// Tile: 128 weight rows x BN rows of a.  The MMA's M is the weights' side, so that few rows of a cost few columns.  A tile's
// blocks of 128 along k are shared by the CTAs of a cluster, whose sums are added in rank order (no workspace, and the same
// bits every time).
// Warp 0: copies, warp 1: products, warps 2-5: sums, a thread a weight row's.
// What bounds it: the weights' bytes where there are many (32 rows x 32,768 x 4,096: 23.2 us for 134 MB, 5.9 TB/s; they stream
// at 6.5, the rest is the launch, the first copies and the end), else the chain of steps: set-up 1,100 cycles (under the first
// copies), first copy 1,400 to 1,700, 150 to 600 a block, barrier and loads of the join 2,500 (1 x 520 x 4,096: 3.8 us; 32
// rows in eight groups of 1,024 x 4,096, 34 MB: 9.6).
// Two CTAs an SM: a sub-partition then holds four of their warps, of at most 128 registers.
template <int BN>
__global__ void __launch_bounds__(kFewThreads, 2) gemm_q8_few_kernel(const __grid_constant__ CUtensorMap wmap,
                                                                        const __grid_constant__ CUtensorMap amap,
                                                                        const __grid_constant__ GemmArgs a) {
    constexpr int NA = kFewAcc;
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
    const int count = (a.nkb - rank + a.splits - 1) / a.splits;  // blocks rank, rank + splits ..
    const int ahead = min(a.stages, count);

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
        // The weights do not come from the preceding kernel: those of the first stages are requested before anything else.
        if (!a.withhold)
            for (int i = 0; i < ahead; ++i) {
                mbar_arrive_expect_tx(&full[i], kStage);
                tma_load_3d(smem_u32(base) + i * kStage, &wmap, (rank + i * a.splits) * 128, nb * kFeat, g, smem_u32(&full[i]));
            }
    }
    if (warp == 1) tmem_alloc(tmem_slot, NA * BN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        pdl_wait();
        if (lane == 0 && !a.withhold) {
            pdl_launch_dependents();
            for (int i = 0; i < ahead; ++i)
                tma_load_3d(smem_u32(base) + i * kStage + kFeat * 128, &amap, (rank + i * a.splits) * 128, g, row0,
                            smem_u32(&full[i]));
            int s = 0, issued = ahead;
            uint32_t ph = 0;
            for (int i = ahead; i < count; ++i) {
                if (!wait_or_stop(&empty[s], ph, stop, a)) break;
                const uint32_t st = smem_u32(base) + s * kStage;
                const int x = (rank + i * a.splits) * 128;
                mbar_arrive_expect_tx(&full[s], kStage);
                tma_load_3d(st, &wmap, x, nb * kFeat, g, smem_u32(&full[s]));
                tma_load_3d(st + kFeat * 128, &amap, x, g, row0, smem_u32(&full[s]));
                ++issued;
                if (++s == a.stages) s = 0, ph ^= 1;
            }
            // no copy is left in flight: the last fill of each stage has landed (an expired wait must not leave one behind)
            for (int i = max(0, issued - a.stages); i < issued; ++i)
                mbar_wait_bounded(&full[i % a.stages], (uint32_t)(i / a.stages) & 1, kWaitLimitNs);
        }
    } else if (warp == 1) {
        pdl_wait();
        constexpr uint32_t idesc = idesc_e4m3(kFeat, BN);
        const uint64_t desc = rows128_desc(smem_u32(base));
        int s = 0, b = 0;
        uint32_t ph = 0, aph = 1;
        for (int i = 0; i < count; ++i) {
            const bool ok = wait_or_stop(&full[s], ph, stop, a) && wait_or_stop(&acc_empty[b], aph, stop, a);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const uint32_t lo = __shfl_sync(0xffffffffu, (uint32_t)desc + s * (kStage >> 4), 0);
            const uint32_t d = __shfl_sync(0xffffffffu, tmem + b * BN, 0);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_f8_elect(d, desc_lo(desc, lo + 2 * ks), desc_lo(desc, lo + (kFeat * 128 >> 4) + 2 * ks), idesc, ks > 0 ? 1u : 0u);
            mma_commit_elect(&acc_full[b]);
            mma_commit_elect(&empty[s]);
            if (++s == a.stages) s = 0, ph ^= 1;
            if (++b == NA) b = 0, aph ^= 1;
        }
        mma_commit_elect(drained);
        mbar_wait_bounded(drained, 0, kWaitLimitNs);
    } else {
        pdl_wait();
        const int t = threadIdx.x - 64;
        const uint32_t column = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        uint64_t acc[BN / 2];
#pragma unroll
        for (int j = 0; j < BN / 2; ++j) acc[j] = 0ull;
        // the products of scales of the CTA's block chunk * 8 + e % 8 and row e / 8, e = t, t + 128 ..
        constexpr int PER = BN * kChunk / 128;
        float next[PER];
        const float* sa = a.a_scale + (long long)g * a.nkb;
        const float* sw = a.w_scale + ((long long)g * a.nnb + nb) * a.nkb;
        const auto fetch = [&](int i0) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = t + 128 * i, row = row0 + e / kChunk, j = i0 + e % kChunk, kb = rank + j * a.splits;
                next[i] = row < a.m && j < count && DSA_IDX_OK(kb, a.nkb, a.status) ? sa[(long long)row * a.a_scale_ld + kb] * __ldg(sw + kb) : 0.f;
            }
        };
        fetch(0);
        int b = 0;
        uint32_t aph = 0;
        bool live = true;  // a warp whose wait expired still takes part in the barriers below
        for (int j = 0; j < count; ++j) {
            const int c = j % kChunk;
            float* sc = scales + (j / kChunk & 1) * kChunk * BN;
            if (c == 0) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int e = t + 128 * i;
                    sc[(e % kChunk) * BN + e / kChunk] = next[i];
                }
                named_bar_sync(1, 128);
                fetch(j + kChunk);
            }
            live = live && __all_sync(0xffffffffu, wait_or_stop(&acc_full[b], aph, stop, a));
            if (!live) continue;
            tc_fence_after();
            const ulonglong2* s2 = reinterpret_cast<const ulonglong2*>(sc + c * BN);  // four rows' scales each
            const uint32_t from = column + b * BN;
            uint32_t p[BN];
            if constexpr (BN == 16) tmem_ld_nowait<16>(from, reinterpret_cast<float(&)[16]>(p));
            else tmem_ld32_nowait(from, p);
            tmem_wait_ld();
            if constexpr (BN == 16) tmem_regs_after_wait<16>(reinterpret_cast<float(&)[16]>(p));
            else regs_after_wait(p);
            tc_fence_before();
            if (lane == 0) mbar_arrive(&acc_empty[b]);
#pragma unroll
            for (int q = 0; q < BN / 4; ++q) {
                const ulonglong2 f = s2[q];
                fma2(acc[2 * q], p[4 * q], p[4 * q + 1], f.x);
                fma2(acc[2 * q + 1], p[4 * q + 2], p[4 * q + 3], f.y);
            }
            if (++b == NA) b = 0, aph ^= 1;
        }
        // every product has ended, so the stages are free
        float* to = part + 32 * (warp & 3) + lane;
#pragma unroll
        for (int j = 0; j < BN / 2; ++j) {
            to[2 * j * 128] = __uint_as_float((uint32_t)acc[j]);
            to[(2 * j + 1) * 128] = __uint_as_float((uint32_t)(acc[j] >> 32));
        }
    }
    __syncwarp();
    if (a.splits > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    bool failed = false;  // a wait expired in one of the CTAs: zeros
    for (int r = 0; r < a.splits; ++r) failed |= ld_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(stop)), r)) != 0u;
    failed = __any_sync(0xffffffffu, failed);
    const int end = min(BN, a.m - row0), step = a.splits * (kFewThreads / 32);
    for (int j = rank + a.splits * warp; j < end;) {
        const int rows = min((end - j + step - 1) / step, a.splits >= 4 ? 1 : 4 / a.splits);
        if (a.splits == 1) join_rows<1>(a, part, j, step, rows, row0, g, nb, lane, failed);
        else if (a.splits == 2) join_rows<2>(a, part, j, step, rows, row0, g, nb, lane, failed);
        else if (a.splits == 4) join_rows<4>(a, part, j, step, rows, row0, g, nb, lane, failed);
        else join_rows<8>(a, part, j, step, rows, row0, g, nb, lane, failed);
        j += rows * step;
    }
    // The others may still read this CTA's sums.  What a thread has read it has used, so nothing needs to be released (a
    // release here waits for the outputs: 2 us).
    if (a.splits > 1) {
        cluster_arrive_relaxed();
        cluster_wait();
    }
    if (warp == 1) tmem_dealloc(tmem, NA * BN);
}

// ---- many rows -------------------------------------------------------------------------------------------------------
// Tile: 256 rows of a x 256 outputs, by a pair of CTAs whose tensor cores work as one (cta_group::2): each CTA copies its 128
// rows of a and its 128 weight rows, the even one issues the products, and each has its rows' sums over all 256 outputs in its
// TMEM, two accumulators of 256 columns in turn.  Pairs go from tile to tile; the products of the next tile's first two blocks
// run while a tile is stored.  Where the tiles leave pairs idle and the blocks are many, two pairs share a tile (SPLIT, below).
//
// Warp 0: copies; warp 1: products (even CTA); warps 2, 3: the scales' products, kChunk blocks at a time; warps 4-11: sums, four
// for each half of the outputs, a thread holding a row's 128 sums.
//
// What bounds it: the sums.  8,192 rows x 32,768 x 4,096 take 853 us (2.58 PFLOP/s, 1.37 times the measured bf16 rate; 735 to
// 780 in short runs, before the clocks fall under the power limit), 2,048 rows in eight groups of 1,024 x 4,096 59 to 63 (256
// tiles are 3.4 rounds of 76 pairs).  A block takes ~700 cycles, of which the products take 512 and the packed FMAs of both warps
// of sums on a scheduler 384 (three register operands make one 3 cycles); the rest of a warp's turn is its wait, its factor and
// its first load, one after the other.  Timed without the sums the kernel ran at the tensor cores' rate (562 us), timed without the
// products no faster than with them.  Tried, in the same runs: sixteen warps of 64 sums 920 against 812; products and barriers for
// each half of the outputs 919; TMEM loads of 16 columns 863; two loads in flight instead of one 850 against 790; scalar FMAs 850
// against 780; last tiles cut into halves of 128 outputs: a block of a half takes 0.9 of a whole one's time; six stages as four;
// bands of 4, 8 or 16 row tiles alike.  Registers: 136 a thread for the first four warps and 184 for the sums spill nothing (SPLIT:
// 44 bytes of stores, 84 of loads); with 64 and 216 it was the first four that spilled whenever a line changed (2,048 rows x 8,192 x
// 4,096: 57.4 us against 62 to 86).
constexpr int kWideThreads = 384;
constexpr int kWideStages = 4;
static_assert(kWideStages % 2 == 0, "a stage meets the same accumulator every round");
constexpr uint32_t kWideStage = 2 * 128 * 128;             // the CTA's rows of a, then its weight rows
constexpr int kBandRows = 8;                               // row tiles that pass over the weights together
constexpr int kOutBytes = 2 * 4096;                        // a warp's outputs on their way
constexpr int kWideSmem = 1024 + kWideStages * (int)kWideStage + 8 * kOutBytes + 2 * kChunk * 256 * 4 + 512;

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_f8_pair_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                  uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives at the barrier in the cluster's CTAs of `mask` once the products issued so far are complete.
__device__ __forceinline__ void mma_commit_pair_elect(uint64_t* bar, uint16_t mask) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            smem_u32(bar)),
        "h"(mask)
        : "memory");
}
// Only TMEM has been read before it, which has ended: no release at cluster scope, whose fence took most of the kernel's time.
__device__ __forceinline__ void mbar_arrive_cluster_elect(uint32_t bar) {
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t@e mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
struct WideTile {
    int g, n0, m0;  // group, first output, first row
};
// Tile t: bands of kBandRows row tiles; within a band all outputs, the band's row tiles next to one another.
__device__ __forceinline__ WideTile wide_tile(const GemmArgs& a, int t) {
    const int per_group = a.tiles_m * a.tiles_n, g = t / per_group;
    t -= g * per_group;
    const int band = t / (kBandRows * a.tiles_n), first = band * kBandRows;
    const int high = min(kBandRows, a.tiles_m - first);
    t -= band * kBandRows * a.tiles_n;
    return WideTile{g, (t / high) * 256, (first + t % high) * 256};
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y),
                 "r"(z), "r"(src)
                 : "memory");
}

// A warp's 32 rows of 128 outputs, a thread a row's.  Through shared memory, 128 bytes of each row at a time in the tensor
// map's swizzle (eight lanes' 16 bytes lie in different banks), and from there by one bulk copy: stored by the threads
// themselves, 32 lines an instruction, the outputs took a fifth of the kernel's time.  The copy leaves out what lies beyond
// the matrix, but by 16 bytes: the last outputs of rows that end within 16 bytes, and outputs whose alignment admits no tensor
// map, are stored by the threads, a lane an output.
__device__ __forceinline__ void store_wide(const GemmArgs& a, const CUtensorMap& omap, uint8_t* stage, long long row, int g,
                                           int j0, int lane, const uint64_t (&acc)[64]) {
    const int left = min(128, a.n - j0), row0 = (int)row - lane;
    if (!DSA_IDX_OK(j0 / 128, a.nnb, a.status) || !DSA_IDX_OK(g, a.groups, a.status)) return;
    float r = 1.f, s = 0.f;  // an 8-bit row's quotients: see BlockQuotient
    if (a.format == kOutQ8) {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 64; ++j) {
            amax = fmaxf(amax, 2 * j < left ? fabsf(lo_of(acc[j])) : 0.f);
            amax = fmaxf(amax, 2 * j + 1 < left ? fabsf(hi_of(acc[j])) : 0.f);
        }
        const float scale = block_scale8(amax);
        const BlockQuotient q(scale);
        r = q.r, s = q.s;
        if (row < a.m) a.out_scale[(row * a.groups + g) * a.nnb + j0 / 128] = scale;
    }
    const auto quotient = [&](float v) {
        const float q = v * r;
        return fmaf(fmaf(-q, s, v), r, q);
    };
    // word w of the row's outputs, of B bytes each
    const auto word = [&](auto bytes, int w) -> uint32_t {
        constexpr int B = decltype(bytes)::value;
        if constexpr (B == 4) return (uint32_t)(acc[w / 2] >> (32 * (w % 2)));
        else if constexpr (B == 2) return bf16x2(lo_of(acc[w]), hi_of(acc[w]));
        else return e4m3x4(quotient(lo_of(acc[2 * w])), quotient(hi_of(acc[2 * w])), quotient(lo_of(acc[2 * w + 1])),
                           quotient(hi_of(acc[2 * w + 1])));
    };
    const bool bulk = a.vec == 2 && (left == 128 || a.whole);
    const auto pieces = [&](auto bytes) {  // bytes an output
        constexpr int B = decltype(bytes)::value, PER = 128 / B;  // outputs in 128 bytes
#pragma unroll
        for (int piece = 0; piece < B; ++piece) {
            uint8_t* to = stage + (piece & 1) * 4096;
            if (lane == 0) {
                // The copy that went through this half of the stage has left it: the one before the last, or (8-bit outputs, one
                // piece a tile) the last tile's.  Halves that alternate from tile to tile instead cost every format a twentieth
                // (8,192 rows x 32,768 x 4,096 862 us against 816, eight groups of 1,024 x 4,096 64.8 against 62.2).
                if (bulk && B > 1) bulk_wait_read<1>();
                else bulk_wait_read<0>();
            }
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int w = piece * 32 + c * 4;
                *reinterpret_cast<uint4*>(to + lane * 128 + ((c ^ (lane & 7)) * 16)) =
                    make_uint4(word(bytes, w), word(bytes, w + 1), word(bytes, w + 2), word(bytes, w + 3));
            }
            if (bulk) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (piece * PER < left) tma_store_3d(&omap, j0 + piece * PER, g, row0, smem_u32(to));
                    bulk_commit();
                }
            } else {  // row by row, a lane an output
                using T = std::conditional_t<B == 4, uint32_t, std::conditional_t<B == 2, uint16_t, uint8_t>>;
                __syncwarp();
                T* out = static_cast<T*>(a.out) + row0 * a.out_ld + (long long)g * a.n + j0 + piece * PER;
#pragma unroll 1
                for (int r = 0; r < min(32, a.m - row0); ++r, out += a.out_ld)
#pragma unroll 1
                    for (int e = lane; e < min(PER, left - piece * PER); e += 32)
                        out[e] = *reinterpret_cast<const T*>(to + r * 128 + ((e * B / 16) ^ (r & 7)) * 16 + e * B % 16);
                __syncwarp();
            }
        }
    };
    if (a.format == kOutF32) pieces(std::integral_constant<int, 4>());
    else if (a.format == kOutBf16) pieces(std::integral_constant<int, 2>());
    else pieces(std::integral_constant<int, 1>());
}

// SPLIT: a cluster of two pairs shares a tile, each with half of its blocks; the first pair ends up with the first 128 outputs and
// the second with the others, whose sums they get from one another through distributed shared memory (500 rows x 4,096 x 8,192:
// 22.0 us against 28.9; the exchange and the two barriers around it take ~2.5).
template <bool SPLIT>
__global__ void __launch_bounds__(kWideThreads, 1) gemm_q8_wide_kernel(const __grid_constant__ CUtensorMap wmap,
                                                                       const __grid_constant__ CUtensorMap amap,
                                                                       const __grid_constant__ CUtensorMap omap,
                                                                       const __grid_constant__ GemmArgs a) {
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint8_t* stage_out = base + kWideStages * kWideStage;  // two pieces of 32 rows x 128 bytes for each warp of sums
    float* scales = reinterpret_cast<float*>(stage_out + 8 * kOutBytes);  // [2][kChunk][half][128 rows]
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + 2 * kChunk * 256);      // the even CTA's: both CTAs' copies
    uint64_t* empty = full + kWideStages;
    uint64_t* acc_full = empty + kWideStages;
    uint64_t* acc_empty = acc_full + 2;  // the even CTA's: both CTAs' warps
    uint64_t* drained = acc_empty + 2;
    uint64_t* sc_full = drained + 1;  // [2]: scales written
    uint64_t* sc_empty = sc_full + 2; // [2]: and read
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sc_empty + 2);
    volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank() & 1, even = cluster_ctarank() & ~1u;  // in the pair; the pair's even CTA
    const int part = SPLIT ? (int)even / 2 : 0, share = SPLIT ? 4 : 2;            // the pair's part of the blocks; CTAs of a tile
    const int pairs = (int)(gridDim.x / share), pair = (int)(blockIdx.x / share);
    const int middle = (a.nkb + 7) / 8 * 4;  // a multiple of 4: scales are read four at a time
    const int kb0 = part == 0 ? 0 : middle, kb1 = SPLIT && part == 0 ? middle : a.nkb;
    const int tiles = a.groups * a.tiles_m * a.tiles_n;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kWideStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 16);
            mbar_init(&sc_full[i], 2);
            mbar_init(&sc_empty[i], 8);
        }
        mbar_init(drained, 1);
        *stop = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 136;");
        if (warp == 0 && lane == 0 && !a.withhold) {
            int s = 0;
            uint32_t ph = 1;
            bool live = true;
            for (int t = pair; t < tiles && live; t += pairs) {
                const WideTile x = wide_tile(a, t);
                const int row = x.m0 + 128 * (int)rank, feat = x.n0 + 128 * (int)rank;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wait_or_stop(&empty[s], ph, stop, a)) {
                        live = false;
                        break;
                    }
                    const uint32_t st = smem_u32(base) + s * kWideStage, bar = mapa_shared(smem_u32(&full[s]), even);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kWideStage);
                    tma_load_3d_pair(st, &amap, kb * 128, x.g, row, bar);
                    tma_load_3d_pair(st + 128 * 128, &wmap, kb * 128, feat, x.g, bar);
                    if (++s == kWideStages) s = 0, ph ^= 1;
                }
            }
            // every stage is read before the CTA ends (a stage never filled passes at once)
            for (int i = 0; i < kWideStages && live; ++i) {
                live = wait_or_stop(&empty[s], ph, stop, a);
                if (++s == kWideStages) s = 0, ph ^= 1;
            }
        } else if (warp == 1 && rank == 0) {
            // Products need no tile: block after block, in a loop unrolled over the stages so that every address is a constant
            // beside one uniform word.
            constexpr uint32_t idesc = idesc_e4m3(256, 256);
            const uint64_t desc = rows128_desc(smem_u32(base));
            const uint32_t first = __shfl_sync(0xffffffffu, (uint32_t)desc, 0), d = __shfl_sync(0xffffffffu, tmem, 0);
            long long left = (long long)((tiles - pair + pairs - 1) / pairs) * (kb1 - kb0);
            for (uint32_t ph = 0; left > 0; ph ^= 1) {
#pragma unroll
                for (int s = 0; s < kWideStages; ++s) {
                    if (left <= 0) break;
                    // the accumulator's (round * kWideStages / 2 + s / 2)-th use; ph is the round's parity
                    const uint32_t use = (kWideStages / 2 % 2 ? ph : 0u) + s / 2;
                    const bool ok = wait_or_stop(&full[s], ph, stop, a) && wait_or_stop(&acc_empty[s & 1], (use & 1) ^ 1, stop, a);
                    if (!__all_sync(0xffffffffu, ok)) {
                        left = 0;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t lo = first + s * (kWideStage >> 4);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f8_pair_elect(d + (s & 1) * 256, desc_lo(desc, lo + 2 * ks), desc_lo(desc, lo + (128 * 128 >> 4) + 2 * ks),
                                          idesc, ks > 0 ? 1u : 0u);
                    mma_commit_pair_elect(&acc_full[s & 1], (uint16_t)(3u << even));
                    mma_commit_pair_elect(&empty[s], (uint16_t)(3u << even));
                    --left;
                }
            }
            mma_commit_pair_elect(drained, (uint16_t)(1u << even));
            mbar_wait_bounded(drained, 0, kWaitLimitNs);
        } else if (warp >= 2) {
            // Each lane two rows: their scales of kChunk blocks (32 bytes of each row), times those of the two halves' weights.
            const int r0 = 64 * (warp - 2) + lane;
            const bool vec = a.a_scale_vec != 0;
            int c = 0;
            uint32_t ph = 1;
            bool live = true;
            for (int t = pair; t < tiles && live; t += pairs) {
                const WideTile x = wide_tile(a, t);
                const float* sw = a.w_scale + ((long long)x.g * a.nnb + x.n0 / 128) * a.nkb;
                const bool second = x.n0 / 128 + 1 < a.nnb;
                for (int kb = kb0; kb < kb1; kb += kChunk) {
                    float s[2][kChunk];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int row = x.m0 + 128 * (int)rank + r0 + 32 * i;
                        const float* sa = a.a_scale + (long long)row * a.a_scale_ld + (long long)x.g * a.nkb + kb;
                        if (vec && row < a.m && kb + kChunk <= a.nkb) {
                            const float4 u = *reinterpret_cast<const float4*>(sa), v = *reinterpret_cast<const float4*>(sa + 4);
                            s[i][0] = u.x, s[i][1] = u.y, s[i][2] = u.z, s[i][3] = u.w;
                            s[i][4] = v.x, s[i][5] = v.y, s[i][6] = v.z, s[i][7] = v.w;
                        } else {
#pragma unroll
                            for (int j = 0; j < kChunk; ++j) s[i][j] = row < a.m && kb + j < a.nkb ? sa[j] : 0.f;
                        }
                    }
                    float w0[kChunk], w1[kChunk];
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) {
                        w0[j] = kb + j < a.nkb ? __ldg(sw + kb + j) : 0.f;
                        w1[j] = second && kb + j < a.nkb ? __ldg(sw + a.nkb + kb + j) : 0.f;
                    }
                    live = __all_sync(0xffffffffu, wait_or_stop(&sc_empty[c], ph, stop, a));
                    if (!live) break;
                    float* to = scales + c * kChunk * 256 + r0;
#pragma unroll
                    for (int j = 0; j < kChunk; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            to[j * 256 + 32 * i] = s[i][j] * w0[j];
                            to[j * 256 + 128 + 32 * i] = s[i][j] * w1[j];
                        }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sc_full[c]);
                    c ^= 1;
                    ph ^= c == 0 ? 1u : 0u;
                }
            }
        }
        __syncwarp();
        if constexpr (SPLIT) {  // as the warps of sums
            cluster_arrive_relaxed();
            cluster_wait();
            cluster_arrive();
            cluster_wait();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int half = (warp - 4) >> 2;
        const int mine = 128 * (int)rank + 32 * (warp & 3) + lane;  // the thread's row of the tile
        const uint32_t column = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + half * 128;
        const uint32_t drained_to = mapa_shared(smem_u32(acc_empty), even);
        const uint32_t factor = smem_u32(scales) + (half * 128 + 32 * (warp & 3) + lane) * 4;
        uint32_t b = 0, c = 0, aph = 0, cph = 0;  // the accumulator, the scales' buffer, and their parities
        bool live = true;
        for (int t = pair; t < tiles; t += pairs) {
            uint64_t acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = 0ull;
            int left = kb1 - kb0;
#pragma unroll 1
            while (left > 0 && live) {
                live = __all_sync(0xffffffffu, wait_or_stop(&sc_full[c], cph, stop, a));
                uint32_t at = factor + c * kChunk * 1024;
                const int until = max(left - kChunk, 0);
#pragma unroll 1
                for (; left > until && live; --left) {
                    const float f = ld_shared_f32(at);
                    at += 1024;
                    if (!__all_sync(0xffffffffu, mbar_try_wait(&acc_full[b], aph))) {
                        live = __all_sync(0xffffffffu, wait_or_stop(&acc_full[b], aph, stop, a));
                        if (!live) break;
                    }
                    tc_fence_after();
                    uint64_t f2;
                    asm("mov.b64 %0, {%1, %1};" : "=l"(f2) : "f"(f));
                    uint32_t p[32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        tmem_ld32_nowait(column + b * 256 + 32 * q, p);
                        tmem_wait_ld();
                        regs_after_wait(p);
                        if (q == 3) {
                            tc_fence_before();
                            mbar_arrive_cluster_elect(drained_to + 8 * b);
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) fma2(acc[16 * q + j], p[2 * j], p[2 * j + 1], f2);
                    }
                    b ^= 1;
                    aph ^= b ^ 1;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_empty[c]);
                c ^= 1;
                cph ^= c ^ 1;
            }
            if constexpr (SPLIT) {  // one tile a cluster
                cluster_arrive_relaxed();
                cluster_wait();  // every product of the four CTAs has ended: the stages are free
                const int at = (32 * (warp & 3) + lane) * 16;
                if (half != part) {
                    const uint32_t to = mapa_shared(smem_u32(base), cluster_ctarank() ^ 2) + at;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        st_cluster_v4(to + j * 2048, lo_of(acc[2 * j]), hi_of(acc[2 * j]), lo_of(acc[2 * j + 1]), hi_of(acc[2 * j + 1]));
                }
                cluster_arrive();
                cluster_wait();
                if (half != part) continue;
                for (int r = 0; r < 4; ++r) live = live && ld_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(stop)), r)) == 0u;
                live = __all_sync(0xffffffffu, live);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float4 v = *reinterpret_cast<const float4*>(base + at + j * 2048);
                    acc[2 * j] = add2(acc[2 * j], pair2(v.x, v.y)), acc[2 * j + 1] = add2(acc[2 * j + 1], pair2(v.z, v.w));
                }
            }
            const WideTile x = wide_tile(a, t);
            if (!live) {  // a wait expired: this tile and the ones after it are zeros
#pragma unroll
                for (int j = 0; j < 64; ++j) acc[j] = 0ull;
            }
            const int j0 = x.n0 + 128 * half;
            if (j0 < a.n && x.m0 + 128 * (int)rank + 32 * (warp & 3) < a.m)
                store_wide(a, omap, stage_out + (warp - 4) * kOutBytes, x.m0 + mine, x.g, j0, lane, acc);
        }
        if (lane == 0) bulk_wait_read<0>();  // shared memory is left; the kernel's end waits for the rest
    }
    if (*stop) {  // copies that the other CTA asked for may still be on their way: they take microseconds
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 2000000ull) {}
    }
    tc_fence_before();
    cluster_arrive_relaxed();  // no data: each thread's loads have ended, and a release would wait for the outputs
    cluster_wait();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ---- host ----------------------------------------------------------------------------------------------------------
struct GemmPlan {
    int feat;    // outputs of a tile: 128, or 256 by a pair of CTAs
    int rows;    // rows of a in a tile
    int splits;  // CTAs that share a tile: its blocks of k, or its rows by a pair (2), both by two pairs (4)
};

constexpr int kFewCtasPerSm = 2;

// The form with the least estimated time.  A round of CTAs takes a fixed time and one for each block of k; both were fitted to
// in-graph times over cold weights on 152 SMs (us).  Outputs x k, rows: the best forms (rows of a tile x CTAs that share it),
// and what they were taken for:
//   4,096 x 4,096       1: 16x8 6.0, 16x4 6.1, 16x1 9.7;  64: 32x4 7.3, 32x2 8.5, pairs 16.6;  256: 32x1 13.5, two pairs 14.3,
//                       pairs 17.1;  500: two pairs 15.5, pairs 17.2, 32x1 26.4
//   4,096 x 8,192       160: two pairs 20.7, 32x1 22.9, pairs 28.7;  500: two pairs 22.0, pairs 28.9, 32x1 45.6
//   4,096 x 16,384      32: 32x8 14.2, 32x4 16.0;  64: 32x4 15.7, 32x2 21.1, pairs 52.0
//   8 x 1,024 x 4,096   32: 32x4 9.1, 32x2 10.7;  100: 32x1 13.7, pairs 17.6;  160: two pairs 16.2, pairs 17.9, 32x1 24.5
//   32,768 x 4,096      32: 32x1 23.8, 32x2 27.5, 16x1 28.0;  64: 32x1 30.3, pairs 33.8;  100: pairs 35.0
//   1,000 x 1,040       500: 32x1 5.7, pairs 8.2, two pairs 10.1;  2,048: pairs 8.6, two pairs 11.2, 32x1 14.0
// The bytes of the weights bound every form; among those that they bound alike the one with the least work of its own is taken.
// Tiles of 64 and 128 rows (one CTA an SM, a block 0.3 and 0.53 us) were best nowhere but at 160 to 256 rows of 4,096 x 16,384
// (128x2 39.8 us, 32x1 42.6), and are not built.
static GemmPlan plan_gemm(int m, int n, int k, int groups) {
    const long long sms = sm_count();
    const int nkb = row_blocks(k);
    const double bytes_us = 3.5 + ((double)groups * n * k + (double)groups * m * k) / 6.0e6;
    const long long wide_tiles = (long long)groups * ((m + 255ll) / 256) * ((n + 255ll) / 256);
    const auto rounds = [](long long items, long long at_once) { return (double)((items + at_once - 1) / at_once); };
    const auto cost = [&](double work) { return std::max(work, bytes_us) + 0.02 * work; };
    GemmPlan best{256, 256, 2};
    double least = cost(3.2 + rounds(wide_tiles, sms / 2) * (2.0 + 0.365 * nkb));
    if (4 * wide_tiles <= sms * 27 / 32 && nkb >= 16) {  // all clusters at once
        const double us = cost(7.8 + 0.40 * ((nkb + 7) / 8 * 4));
        if (us < least) best = GemmPlan{256, 256, 4}, least = us;
    }
    for (int rows = 16; rows <= 32; rows *= 2) {
        const long long tiles = (long long)groups * row_blocks(n) * ((m + rows - 1ll) / rows);
        for (int splits = 1; splits <= 8 && (splits == 1 || nkb >= 2 * splits); splits *= 2) {
            // clusters of eight leave some SMs of a GPC out
            const long long at_once = (splits == 8 ? sms * 27 / 32 : sms) * kFewCtasPerSm;
            const double us = cost(rounds(tiles * splits, at_once) *
                                   (4.5 + (splits > 1 ? 0.7 : 0.0) + (rows == 16 ? 0.16 : 0.235) * ((nkb + splits - 1) / splits)));
            if (us < least) best = GemmPlan{kFeat, rows, splits}, least = us;
        }
    }
    return best;
}

// Codes [z][y][x] (x contiguous) in boxes of 128 x box_y x box_z.
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
    constexpr int extra = 1024 + 2 * kChunk * BN * 4 + 512;
    constexpr int budget = 228 * 1024 / kFewCtasPerSm - 1024;
    a.stages = std::min(12, (budget - extra) / few_stage_bytes<BN>());
    const int smem = extra + a.stages * few_stage_bytes<BN>();
    static_assert((budget - extra) / few_stage_bytes<BN>() * few_stage_bytes<BN>() >= BN * 512, "the sums fit into the stages");
    if (cudaFuncSetAttribute(gemm_q8_few_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return DSA_ERR_CUDA;
    const long long grid = (long long)a.groups * a.tiles_n * a.tiles_m * a.splits;
    if (grid > 0x7fffffff) return DSA_ERR_UNSUPPORTED;
    if (launch_pdl_cluster(gemm_q8_few_kernel<BN>, dim3((unsigned)grid), dim3(kFewThreads), smem, st, a.splits, wmap,
                           amap, a) != cudaSuccess)
        return DSA_ERR_CUDA;
    return launch_status();
}

static dsa_status_t launch_wide(const CUtensorMap& wmap, const CUtensorMap& amap, GemmArgs a, cudaStream_t st) {
    CUtensorMap omap = wmap;
    if (a.vec == 2) {
        auto fn = tensor_map_encoder();
        const int size = a.format == kOutF32 ? 4 : a.format == kOutBf16 ? 2 : 1;
        const cuuint64_t dim[3] = {(cuuint64_t)a.n, (cuuint64_t)a.groups, (cuuint64_t)a.m};
        // one group: its stride is never used, but has to be a multiple of 16
        const cuuint64_t stride[2] = {((cuuint64_t)a.n * size + 15) / 16 * 16, (cuuint64_t)a.out_ld * size};
        const cuuint32_t box[3] = {(cuuint32_t)(128 / size), 1, 32}, one[3] = {1, 1, 1};
        if (!fn || fn(&omap,
                      a.format == kOutF32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                      : a.format == kOutBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                      3, a.out, dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return DSA_ERR_CUDA;
    }
    const long long tiles = (long long)a.groups * a.tiles_n * a.tiles_m;
    if (tiles > 0x3fffffff) return DSA_ERR_UNSUPPORTED;
    const bool split = a.splits == 4;
    const auto kernel = split ? gemm_q8_wide_kernel<true> : gemm_q8_wide_kernel<false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWideSmem) != cudaSuccess) return DSA_ERR_CUDA;
    const long long grid = split ? 4 * tiles : 2 * std::min<long long>(tiles, sm_count() / 2);
    if (launch_pdl_cluster(kernel, dim3((unsigned)grid), dim3(kWideThreads), kWideSmem, st, a.splits, wmap, amap, omap, a) !=
        cudaSuccess)
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
    if (a_ld >= (1ll << 40) || a_scale_ld >= (1ll << 40) || out_ld >= (1ll << 38)) return DSA_ERR_UNSUPPORTED;  // the tensor maps' strides
    const GemmPlan p = plan_gemm(m, n, k, groups);
    GemmArgs args{};
    args.m = m, args.n = n, args.k = k, args.groups = groups, args.nkb = nkb, args.nnb = nnb;
    args.a_scale = a_scale, args.a_scale_ld = a_scale_ld;
    args.a_scale_vec = aligned(a_scale, 16) && a_scale_ld % 4 == 0 && (groups == 1 || nkb % 4 == 0);
    args.w_scale = w_scale;
    args.out = out, args.out_ld = out_ld, args.out_scale = out_scale, args.format = out_format;
    args.vec = aligned(out, 4 * size) && out_ld % 4 == 0 && (groups == 1 || n % 4 == 0) ? 1 : 0;
    if (args.vec && aligned(out, 16) && out_ld * size % 16 == 0 && (groups == 1 || (long long)n * size % 16 == 0)) args.vec = 2;
    args.whole = (long long)n * size % 16 == 0;
    args.splits = p.splits, args.tiles_n = (n + p.feat - 1) / p.feat, args.tiles_m = (m + p.rows - 1) / p.rows;
    args.status = dev_status, args.wait_ns = wait_ns, args.withhold = withhold;
    CUtensorMap wmap, amap;
    if (!make_codes_map(&wmap, w, k, n, groups, k, (long long)n * k, kFeat, 1) ||
        !make_codes_map(&amap, a, k, groups, m, k, a_ld, 1, std::min(p.rows, 128)))
        return DSA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p.feat == 256) return launch_wide(wmap, amap, args, st);
    return p.rows == 16 ? launch_few<16>(wmap, amap, args, st) : launch_few<32>(wmap, amap, args, st);
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
    plan[0] = p.feat, plan[1] = p.rows, plan[2] = p.splits;
    return DSA_OK;
}
