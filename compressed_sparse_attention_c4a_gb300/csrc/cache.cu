// dsa_cache_write / dsa_cache_read: rows into a paged cache in its storage format, and back as values; dsa_cache_append:
// rows normed and rotated by their positions on the way.
//
// [P1] "DeepSeek DSA、DeepSeek V4与vLLM Hybrid KV Cache详解" §2.2 (logical rows of a request through its block table),
// [P2] "DeepSeek V4 稀疏注意力完全解剖" 设计 1 (256 raw positions per logical block) and 第三层 (prefill keeps the cache
// in bf16, decode quantises it row by row): the caches that a prefill hands over are stored row by row in the decode
// format, and stored rows can be had back as bf16 values.
#include <algorithm>

#include "common.cuh"
#include "rows.cuh"
#include "rows8.cuh"

namespace dsa {

constexpr int kRowThreads = 256;  // 8 warps, a row each, or four in turn

// What bounds both, from about 30,000 rows on: the rows in flight.  A warp requests nothing of its next rows before its own are
// stored, and its waits for HBM lead the stalls (131,072 rows, 1,316 or 1,324 bytes each: stored in 36.5 us, 4.7 TB/s, and read
// in 35.7, with DRAM 50 and 39 % busy and the issue slots 57 and 51 %; 65,536 rows 20.3 and 20.1).  Below that the chain of loads
// from the schedule to the row.  Storing takes 200 instructions a row for a warp, reading 100.  The other formats, 131,072 rows
// of 512 stored and read: bf16 51.8 and 44.4 us (floor 40.1), e4m3 56.9 and 36.7 (30.1), e2m1 53.8 and 35.2 (25.1); their stores
// divide every element by the row scale.
//
// Rows per warp: four consecutive ones, whose addresses four lanes find side by side and whose loads are in flight
// together, when there are enough rows for two blocks of such warps on every SM.  Measured over one input again and again
// (up to 65,536 rows it stays in the L2), four against one, stored and read: 131,072 rows 35.8 and 35.5 us against 38.0 and 44.3, 65,536 rows 14.3 and 15.5 against 18.4 and 18.6, 16,384 rows
// 5.1 and 5.0 against 5.3 and 5.4; 8,192 rows level, 5,000 rows 2.9 and 3.6 against 2.5 and 3.4.
static int rows_per_warp(long long n) { return n >= 2ll * 4 * 8 * sm_count() ? 4 : 1; }

struct CacheWriteArgs {
    int batch, n;
    const int32_t* cu_new;
    const int32_t* start_row;
    const uint16_t* x;
    dsa_pool_t pool;
    dsa_block_table_t bt;
    int32_t* status;
    bool wide;  // x 32-byte aligned
};

// The request of new row j: the largest r with cu_new[r] <= j, by a search of 32 probes a step (one for up to 32
// requests, two for up to 1024).
__device__ __forceinline__ int request_of(const int32_t* cu_new, int batch, int j, int lane) {
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int p = lo + step * lane;
        const unsigned le = __ballot_sync(0xffffffffu, p < hi && (lane == 0 || __ldg(cu_new + p) <= j));
        lo += step * (31 - __clz(le));
        hi = min(hi, lo + step);
    }
    return lo;
}

// physical_row() of a row below 2^32: a 32-bit division.
__device__ __forceinline__ long long pool_row(const dsa_block_table_t& bt, int r, uint32_t row, const dsa_pool_t& pool) {
    const uint32_t lb = row / (uint32_t)pool.rows_per_block;
    if (lb >= (uint32_t)bt.max_blocks) return -1;
    const int pb = __ldg(bt.table + (long long)r * bt.max_blocks + lb);
    if (pb < 0 || pb >= pool.num_blocks) return -1;
    return (long long)pb * pool.rows_per_block + (row - lb * (uint32_t)pool.rows_per_block);
}

__device__ __forceinline__ long long pool_rows(const dsa_pool_t& p) { return (long long)p.num_blocks * p.rows_per_block; }

// A warp takes R consecutive rows.  BLOCK: a pool of DSA_FP4_BLOCK, else any other.  The schedule and the block table are
// read before waiting for the preceding kernel.
template <int DIM, int R, bool BLOCK>
__global__ void __launch_bounds__(kRowThreads) cache_write_kernel(CacheWriteArgs a) {
    constexpr int E = DIM / 32;
    const int lane = threadIdx.x & 31;
    const long long j0 = ((long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * R;
    const int total = min(a.n, __ldg(a.cu_new + a.batch));
    const int live = (int)min((long long)R, total - j0);
    long long prow = -1;  // lane i < live: of row j0 + i
    if (live > 0) {
        int r = request_of(a.cu_new, a.batch, (int)j0, lane);
        if constexpr (R > 1) {
            const int last = request_of(a.cu_new, a.batch, (int)j0 + live - 1, lane);
            for (int hi = last + 1; hi - r > 1;) {  // between the two
                const int mid = (r + hi) / 2;
                if (__ldg(a.cu_new + mid) <= j0 + lane) r = mid;
                else hi = mid;
            }
        }
        if (lane < live) {
            const long long row = (long long)__ldg(a.start_row + r) + (j0 + lane - __ldg(a.cu_new + r));
            if (row >= 0 && DSA_IDX_OK(r, a.batch, a.status)) prow = pool_row(a.bt, r, (uint32_t)row, a.pool);
            if (prow >= 0 && !DSA_IDX_OK(prow, pool_rows(a.pool), a.status)) prow = -1;
        }
    }
    pdl_wait();
    pdl_launch_dependents();
    if (live <= 0) return;
    if (lane < live && prow < 0) report(a.status, DSA_ERR_DEVICE_FAULT);
    uint32_t u[R][E / 2];
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < live && DSA_IDX_OK(j0 + i, a.n, a.status)) load_bf16_words<E>(a.x + (j0 + i) * DIM, lane, u[i], a.wide);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const long long to = __shfl_sync(0xffffffffu, prow, i);
        if (i >= live || to < 0) continue;
        if constexpr (BLOCK) {
            uint32_t c[2];
            float s;
            const uint8_t bs = fp4_block_codes_bf16(u[i], c, &s);
            store_fp4_block_row(a.pool, to, lane, c, bs, s);
        } else {
            float v[E];
            bf16_words<E>(u[i], v);
            store_row<E>(a.pool, to, lane, v);
        }
    }
}

struct CacheReadArgs {
    int n;
    const int32_t* req;
    const int32_t* ids;
    dsa_pool_t pool;
    dsa_block_table_t bt;
    uint16_t* out;
    int32_t* status;
    bool wide;  // out 32-byte aligned
};

// A lane's part of a stored row as it lies in memory: E elements, the row's scale, the block's.
template <int E>
struct StoredRow {
    uint32_t w[E / 2];
    float scale;
    uint32_t block;
};

template <int E>
__device__ __forceinline__ void fetch_row(const dsa_pool_t& pool, long long prow, int lane, StoredRow<E>& row) {
    const uint8_t* base = static_cast<const uint8_t*>(pool.data);
    if (pool.dtype == DSA_BF16) {
        load_bf16_words<E>(reinterpret_cast<const uint16_t*>(base) + prow * (E * 32), lane, row.w, false);
        return;
    }
    row.scale = pool.scale[prow];
    if (pool.dtype == DSA_FP8_E4M3) {
        const uint8_t* src = base + prow * (E * 32) + lane * E;
        if constexpr (E == 16) {
            const uint4 u = *reinterpret_cast<const uint4*>(src);
            row.w[0] = u.x, row.w[1] = u.y, row.w[2] = u.z, row.w[3] = u.w;
        } else if constexpr (E == 4) {
            row.w[0] = *reinterpret_cast<const uint32_t*>(src);
        } else {
            row.w[0] = *reinterpret_cast<const uint16_t*>(src);
        }
        return;
    }
    // two e2m1 codes a byte, with a scale per row, or per row and block
    const bool block = pool.dtype == DSA_FP4_BLOCK;
    const uint8_t* src = base + prow * (block ? kFp4BlockRow : E * 16);
    if constexpr (E == 16) {
        if (block) row.block = src[kFp4BlockRow - 32 + lane];
        const uint2 u = *reinterpret_cast<const uint2*>(src + lane * 8);
        row.w[0] = u.x, row.w[1] = u.y;
    } else if constexpr (E == 4) {
        row.w[0] = *reinterpret_cast<const uint16_t*>(src + lane * 2);
    } else {
        row.w[0] = src[lane];
    }
}

template <int E>
__device__ __forceinline__ void row_values(int dtype, const StoredRow<E>& row, float (&v)[E]) {
    if (dtype == DSA_FP8_E4M3) {
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((uint16_t)(row.w[k / 2] >> (16 * (k & 1))), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            v[2 * k] = row.scale * f.x;
            v[2 * k + 1] = row.scale * f.y;
        }
        return;
    }
    float unit = row.scale;
    if constexpr (E == kFp4Block) {
        if (dtype == DSA_FP4_BLOCK) {
            const __half_raw h = __nv_cvt_fp8_to_halfraw((uint8_t)row.block, __NV_E4M3);
            unit = row.scale * __half2float(*reinterpret_cast<const __half*>(&h));
        }
    }
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((uint8_t)(row.w[k / 4] >> (8 * (k & 3))), __NV_E2M1);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[2 * k] = unit * f.x;
        v[2 * k + 1] = unit * f.y;
    }
}

// A warp takes R consecutive rows.
template <int DIM, int R>
__global__ void __launch_bounds__(kRowThreads) cache_read_kernel(CacheReadArgs a) {
    constexpr int E = DIM / 32;
    const int lane = threadIdx.x & 31;
    const long long j0 = ((long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * R;
    pdl_wait();
    pdl_launch_dependents();
    const int live = (int)min((long long)R, a.n - j0);
    if (live <= 0) return;
    long long prow = -1;  // lane i < live: of row j0 + i
    if (lane < live) {
        const int id = __ldg(a.ids + j0 + lane), r = __ldg(a.req + j0 + lane);
        if (id >= 0 && r >= 0 && r < a.bt.batch)
            prow = pool_row(a.bt, r, (uint32_t)id, a.pool);
        if (prow >= 0 && !DSA_IDX_OK(prow, pool_rows(a.pool), a.status)) prow = -1;
        if (prow < 0 && id != -1) report(a.status, DSA_ERR_DEVICE_FAULT);
    }
    StoredRow<E> row[R];
    long long from[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        from[i] = __shfl_sync(0xffffffffu, prow, i);
        if (from[i] >= 0) fetch_row<E>(a.pool, from[i], lane, row[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (i >= live) break;
        uint32_t u[E / 2] = {};
        if (from[i] >= 0) {
            if (a.pool.dtype == DSA_BF16) {
#pragma unroll
                for (int k = 0; k < E / 2; ++k) u[k] = row[i].w[k];
            } else {
                float v[E];
                row_values<E>(a.pool.dtype, row[i], v);
#pragma unroll
                for (int k = 0; k < E / 2; ++k)
                    u[k] = (uint32_t)float_to_bf16(v[2 * k]) | ((uint32_t)float_to_bf16(v[2 * k + 1]) << 16);
            }
        }
        store_words<E / 2>(a.out + (j0 + i) * DIM + lane * E, u, a.wide);
    }
}

// ---- dsa_cache_append ------------------------------------------------------------------------------------------------
struct CacheAppendArgs {
    int batch, n;
    const int32_t* cu_new;
    const int32_t* start_pos;
    const uint16_t* x;
    long long x_ld;
    const float* gamma;
    float eps;
    RopeTable rope;
    dsa_pool_t pool;
    dsa_block_table_t bt;
    int32_t* status;
    bool wide;  // rows of x 32-byte aligned
};

// The lane's frequency as a table's first, kept in registers: a kernel argument indexed by the lane is fetched lane by lane, and
// the compiler would fetch it again for every row (131,072 rows: 71 us against 42).
__device__ __forceinline__ void own_frequency(const RopeTable& all, int lane, RopeTable& own) {
    own.f_hi[0] = all.f_hi[lane], own.f_lo[0] = all.f_lo[lane];
    asm volatile("" : "+f"(own.f_hi[0]), "+f"(own.f_lo[0]));
}

// Rotates the pairs of the last rope_dim dims by R_pos.  A lane finds the angle of one pair, whatever lanes hold it: the
// E / 2 pairs of a lane one after the other would leave the lanes without pairs idle (rows of 512: four lanes hold them all).
// own: a table whose first frequency is the lane's.
template <int E>
__device__ __forceinline__ void rotate_row(float (&v)[E], int lane, const RopeTable& own, int rope_dim, long long pos) {
    const int pairs = rope_dim / 2, first = E * 32 - rope_dim;
    float c = 1.f, s = 0.f;
    if (lane < pairs) rope_cos_sin(pos, own, 0, &c, &s);
#pragma unroll
    for (int k = 0; k < E; k += 2) {
        const int d = lane * E + k, j = (d - first) / 2;
        const float cj = __shfl_sync(0xffffffffu, c, j & 31), sj = __shfl_sync(0xffffffffu, s, j & 31);
        if (d >= first) {
            const float x0 = v[k], x1 = v[k + 1];
            v[k] = x0 * cj - x1 * sj;
            v[k + 1] = x0 * sj + x1 * cj;
        }
    }
}

// The pool row (-1: none) and position of new row j0 + lane * apart, for the `live` rows of a warp.
__device__ __forceinline__ void append_places(const CacheAppendArgs& a, long long j0, long long apart, int live, int lane,
                                              long long* prow, uint32_t* pos) {
    *prow = -1, *pos = 0;
    if (live <= 0) return;
    int r = request_of(a.cu_new, a.batch, (int)j0, lane);
    const long long j = j0 + lane * apart;
    if (lane >= live) return;
    if (live > 1)
        for (int hi = a.batch; hi - r > 1;) {
            const int mid = (r + hi) / 2;
            if (__ldg(a.cu_new + mid) <= j) r = mid;
            else hi = mid;
        }
    const int start = __ldg(a.start_pos + r);
    *pos = (uint32_t)start + (uint32_t)(j - __ldg(a.cu_new + r));  // below 2^32
    if (start >= 0 && DSA_IDX_OK(r, a.batch, a.status)) *prow = pool_row(a.bt, r, *pos, a.pool);
    if (*prow >= 0 && !DSA_IDX_OK(*prow, pool_rows(a.pool), a.status)) *prow = -1;
}

// Rows of 512 into bf16 or e4m3 pools.  Lane l holds dims 128 i + 4 l .. + 3, so that the 32 pairs of the rotation lie two to
// a lane in sixteen lanes.  The warps take the rows in turn, the next one or two of a warp's on their way into shared memory
// while it works on one; the places of a warp's next eight rows are found by eight lanes side by side.  131,072 rows normed into
// e4m3 (1,540 bytes each) take 40.1 us, 5.0 TB/s, into bf16 (2,048 bytes) 46.1, 5.8 TB/s, without the norm into e4m3 36.6.  What
// bounds the first: a row is one chain (sum, factor, rotation, largest value, codes) of about 250 instructions, and 24 warps an
// SM do not cover it: the issue slots are 70 % busy and DRAM 49 %, 45 instructions a row less (angles of consecutive rows turned
// from the first one's) took longer, two rows to a warp, sixteen lanes each, 36.6 us against 39.6, but longer for few rows (6,000
// rows 5.2 us against 4.2, 32 rows 3.0 against 2.3).  One row on its way against two: with the norm 39.6 against 40.3 us and,
// into bf16, 45.7 against 50.1, without it 42.2 against 36.4.
template <bool NORM, bool FP8>
__global__ void __launch_bounds__(kRowThreads) cache_append_wide_kernel(const __grid_constant__ CacheAppendArgs a) {
    constexpr int kAppendAhead = NORM ? 1 : 2;  // rows of a warp on their way
    const int lane = threadIdx.x & 31;
    const int total = min(a.n, __ldg(a.cu_new + a.batch));
    uint64_t g[8];
    if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float* src = a.gamma + 128 * (i / 2) + 4 * lane + 2 * (i % 2);
            g[i] = a.gamma ? pair2(__ldg(src), __ldg(src + 1)) : pair2(1.f, 1.f);
        }
    }
    const int pairs = a.rope.rope_dim / 2;
    RopeTable own;
    own_frequency(a.rope, lane, own);
    const int p0 = 2 * lane - 64 + pairs;  // the first of the lane's two pairs among the rotated ones
    __shared__ alignas(16) uint4 ring[kRowThreads / 32][kAppendAhead][64];
    uint4(*mine)[64] = ring[threadIdx.x >> 5];
    const auto request = [&](long long j, int slot) {  // a group of copies, empty behind the last row
        if (j < total && DSA_IDX_OK(j, a.n, a.status)) {
            const uint16_t* src = a.x + j * a.x_ld + 8 * lane;
            cp_async16_nc(smem_u32(&mine[slot][lane]), src, 16);
            cp_async16_nc(smem_u32(&mine[slot][lane + 32]), src + 256, 16);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    constexpr int kTogether = 8;  // rows whose places are found together
    const long long warps = (long long)gridDim.x * (kRowThreads / 32);
    long long j0 = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5), prow;
    const auto rows_from = [&](long long j) { return j < total ? (int)min((long long)kTogether, (total - 1 - j) / warps + 1) : 0; };
    uint32_t pos;
    int live = rows_from(j0);
    append_places(a, j0, warps, live, lane, &prow, &pos);
    pdl_wait();
    pdl_launch_dependents();
#pragma unroll
    for (int i = 0; i < kAppendAhead; ++i) request(j0 + i * warps, i);
    int slot = 0;
    while (live > 0) {
        if (lane < live && prow < 0) report(a.status, DSA_ERR_DEVICE_FAULT);
#pragma unroll 1
        for (int i = 0; i < live; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kAppendAhead - 1) : "memory");
            __syncwarp();
            uint2 u[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) u[c] = reinterpret_cast<const uint2*>(mine[slot])[32 * c + lane];
            __syncwarp();
            request(j0 + (i + kAppendAhead) * warps, slot);
            if (++slot == kAppendAhead) slot = 0;
            const long long to = __shfl_sync(0xffffffffu, prow, i);
            const uint32_t at = __shfl_sync(0xffffffffu, pos, i);
            if (to < 0) continue;
            uint64_t v[8];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[2 * c] = pair_of_bf16(u[c].x), v[2 * c + 1] = pair_of_bf16(u[c].y);
            float rs = 1.f;  // the norm's factor: taken into the end, as it is one for the row
            if constexpr (NORM) {
                uint64_t s2 = mul2(v[0], v[0]);
#pragma unroll
                for (int k = 1; k < 8; ++k) s2 = fma2(v[k], v[k], s2);
                const float ss = warp_sum(lo_of(s2) + hi_of(s2));
                rs = rsqrtf(ss / 512.f + a.eps);
                if (!(ss < INFINITY)) {  // squares beyond fp32: those of the values times 2^-80, beside which eps is nothing
                    s2 = 0ull;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint64_t w = mul2(v[k], pair2(0x1p-80f, 0x1p-80f));
                        s2 = fma2(w, w, s2);
                        v[k] = mul2(v[k], pair2(0x1p-40f, 0x1p-40f));  // the rest is rs's: small values keep their bits
                    }
                    rs = 0x1p-40f * rsqrtf(warp_sum(lo_of(s2) + hi_of(s2)) / 512.f);
                }
                // A row of huge or tiny values, an infinity or a NaN: gamma times them could leave fp32 where the norm does not
                if (FP8 && !(rs > 0x1p-20f && rs < 0x1p20f)) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = mul2(v[k], pair2(rs, rs));
                    rs = 1.f;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = mul2(FP8 ? v[k] : mul2(v[k], pair2(rs, rs)), g[k]);
            }
            if (pairs > 0) {
                float c = 1.f, s = 0.f;
                if (lane < pairs) rope_cos_sin((long long)at, own, 0, &c, &s);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float ck = __shfl_sync(0xffffffffu, c, (p0 + k) & 31), sk = __shfl_sync(0xffffffffu, s, (p0 + k) & 31);
                    const float x0 = lo_of(v[6 + k]), x1 = hi_of(v[6 + k]);
                    if (p0 + k >= 0) v[6 + k] = pair2(x0 * ck - x1 * sk, x0 * sk + x1 * ck);
                }
            }
            if constexpr (!FP8) {
                uint16_t* dst = static_cast<uint16_t*>(a.pool.data) + to * 512 + 4 * lane;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint2*>(dst + 128 * c) =
                        make_uint2(bf16x2(lo_of(v[2 * c]), hi_of(v[2 * c])), bf16x2(lo_of(v[2 * c + 1]), hi_of(v[2 * c + 1])));
            } else {
                float m = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) m = fmaxf(m, fmaxf(fabsf(lo_of(v[k])), fabsf(hi_of(v[k]))));
                const float amax = __uint_as_float(warp_abs_max_bits(__float_as_uint(m)));  // (fmaxf passes over NaN)
                float scale;
                if (amax > 0x1p-60f && amax < 0x1p60f) {
                    const float q = amax * (1.f / 448.f);  // amax / 448: a reciprocal, a correction by the remainder (Markstein's)
                    scale = fmaf(fmaf(-q, 448.f, amax), 1.f / 448.f, q);
                    if constexpr (NORM) {  // the values are rounded already: a product with the reciprocal is near enough
                        const float r = near_reciprocal(scale);
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = mul2(v[k], pair2(r, r));
                    } else {
                        const BlockQuotient2 quotient(scale);
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = quotient(v[k]);
                    }
                } else {  // parts of which could leave fp32's normal range, the norm's factor not yet taken in
                    if constexpr (NORM) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = mul2(v[k], pair2(rs, rs));
                    }
                    const float most = amax * rs;
                    rs = 1.f;
                    scale = most > 0.f ? most / 448.f : 1.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = pair2(lo_of(v[k]) / scale, hi_of(v[k]) / scale);
                }
                uint8_t* dst = static_cast<uint8_t*>(a.pool.data) + to * 512 + 4 * lane;
#pragma unroll
                for (int c = 0; c < 4; ++c) *reinterpret_cast<uint32_t*>(dst + 128 * c) = e4m3x4(v[2 * c], v[2 * c + 1]);
                if (lane == 0) a.pool.scale[to] = amax > 0.f ? scale * rs : 1.f;
            }
        }
        j0 += live * warps;
        live = rows_from(j0);
        append_places(a, j0, warps, live, lane, &prow, &pos);
    }
}

// Any pool of rows of DIM.  A warp takes R consecutive rows, one after the other from the registers that their loads, in flight
// together, fill.
template <int DIM, int R, bool NORM>
__global__ void __launch_bounds__(kRowThreads) cache_append_kernel(const __grid_constant__ CacheAppendArgs a) {
    constexpr int E = DIM / 32;
    const int lane = threadIdx.x & 31;
    const long long j0 = ((long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * R;
    const int total = min(a.n, __ldg(a.cu_new + a.batch));
    const int live = (int)min((long long)R, total - j0);
    long long prow;
    uint32_t pos;
    append_places(a, j0, 1, live, lane, &prow, &pos);
    float g[E];
    if constexpr (NORM) {
#pragma unroll
        for (int k = 0; k < E; ++k) g[k] = a.gamma ? __ldg(a.gamma + lane * E + k) : 1.f;
    }
    pdl_wait();
    pdl_launch_dependents();
    if (live <= 0) return;
    if (lane < live && prow < 0) report(a.status, DSA_ERR_DEVICE_FAULT);
    RopeTable own;
    own_frequency(a.rope, lane, own);
    uint32_t u[R][E / 2];
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < live && DSA_IDX_OK(j0 + i, a.n, a.status)) load_bf16_words<E>(a.x + (j0 + i) * a.x_ld, lane, u[i], a.wide);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const long long to = __shfl_sync(0xffffffffu, prow, i);
        const uint32_t at = __shfl_sync(0xffffffffu, pos, i);
        if (i >= live || to < 0) continue;
        float v[E];
        bf16_words<E>(u[i], v);
        if constexpr (NORM) {
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < E; ++k) ss = fmaf(v[k], v[k], ss);
            ss = warp_sum(ss);
            float rs = rsqrtf(ss / (float)DIM + a.eps);
            if (!(ss < INFINITY)) {  // as above
                ss = 0.f;
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const float w = v[k] * 0x1p-80f;
                    ss = fmaf(w, w, ss);
                    v[k] *= 0x1p-40f;
                }
                rs = 0x1p-40f * rsqrtf(warp_sum(ss) / (float)DIM);
            }
#pragma unroll
            for (int k = 0; k < E; ++k) v[k] = v[k] * rs * g[k];
        }
        rotate_row<E>(v, lane, own, a.rope.rope_dim, (long long)at);
        store_row<E>(a.pool, to, lane, v);
    }
}

template <int DIM, bool NORM>
static cudaError_t launch_append(const CacheAppendArgs& a, cudaStream_t st) {
    const dim3 block(kRowThreads);
    if (DIM == 512 && (a.pool.dtype == DSA_BF16 || a.pool.dtype == DSA_FP8_E4M3)) {
        const dim3 grid((unsigned)std::min<long long>((a.n + 7ll) / 8, 3ll * sm_count()));
        return a.pool.dtype == DSA_FP8_E4M3 ? launch_pdl(cache_append_wide_kernel<NORM, true>, grid, block, 0, st, a)
                                            : launch_pdl(cache_append_wide_kernel<NORM, false>, grid, block, 0, st, a);
    }
    const bool four = rows_per_warp(a.n) == 4;
    const dim3 grid((unsigned)((a.n + (four ? 31ll : 7ll)) / (four ? 32 : 8)));
    return launch_pdl(four ? cache_append_kernel<DIM, 4, NORM> : cache_append_kernel<DIM, 1, NORM>, grid, block, 0, st, a);
}

static dsa_status_t check_rows(const dsa_pool_t* pool, const dsa_block_table_t* bt) {
    if (!pool_ok(pool) || !bt || !bt->table || bt->max_blocks <= 0 || bt->batch <= 0) return DSA_ERR_INVALID_ARG;
    if (pool->dim != 64 && pool->dim != 128 && pool->dim != 512) return DSA_ERR_UNSUPPORTED;
    return block_rows_ok(pool) ? DSA_OK : DSA_ERR_UNSUPPORTED;
}

}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_cache_write(int32_t batch, const int32_t* cu_new, const int32_t* start_row, int32_t n,
                                        const void* x, const dsa_pool_t* pool, const dsa_block_table_t* bt,
                                        int32_t* dev_status, void* stream) {
    if (batch < 0 || n < 0) return DSA_ERR_INVALID_ARG;
    if (batch == 0 || n == 0) return DSA_OK;
    const dsa_status_t e = check_rows(pool, bt);
    if (e != DSA_OK) return e;
    if (!cu_new || !start_row || !x || !aligned(x, 16) || bt->batch < batch) return DSA_ERR_INVALID_ARG;
    const CacheWriteArgs a{batch, n, cu_new, start_row, static_cast<const uint16_t*>(x), *pool, *bt, dev_status, aligned(x, 32)};
    const bool four = rows_per_warp(n) == 4;
    const dim3 grid((unsigned)((n + (four ? 31ll : 7ll)) / (four ? 32 : 8))), block(kRowThreads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t err =
        pool->dtype == DSA_FP4_BLOCK
            ? launch_pdl(four ? cache_write_kernel<512, 4, true> : cache_write_kernel<512, 1, true>, grid, block, 0, st, a)
        : pool->dim == 64
            ? launch_pdl(four ? cache_write_kernel<64, 4, false> : cache_write_kernel<64, 1, false>, grid, block, 0, st, a)
        : pool->dim == 128
            ? launch_pdl(four ? cache_write_kernel<128, 4, false> : cache_write_kernel<128, 1, false>, grid, block, 0, st, a)
            : launch_pdl(four ? cache_write_kernel<512, 4, false> : cache_write_kernel<512, 1, false>, grid, block, 0, st, a);
    if (err != cudaSuccess) return DSA_ERR_CUDA;
    return launch_status();
}

extern "C" dsa_status_t dsa_cache_read(const dsa_pool_t* pool, const dsa_block_table_t* bt, int32_t n,
                                       const int32_t* req, const int32_t* ids, void* out, int32_t* dev_status,
                                       void* stream) {
    if (n < 0) return DSA_ERR_INVALID_ARG;
    if (n == 0) return DSA_OK;
    const dsa_status_t e = check_rows(pool, bt);
    if (e != DSA_OK) return e;
    if (!req || !ids || !out || !aligned(out, 16)) return DSA_ERR_INVALID_ARG;
    const CacheReadArgs a{n, req, ids, *pool, *bt, static_cast<uint16_t*>(out), dev_status, aligned(out, 32)};
    const bool four = rows_per_warp(n) == 4;
    const dim3 grid((unsigned)((n + (four ? 31ll : 7ll)) / (four ? 32 : 8))), block(kRowThreads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t err =
        pool->dim == 64    ? launch_pdl(four ? cache_read_kernel<64, 4> : cache_read_kernel<64, 1>, grid, block, 0, st, a)
        : pool->dim == 128 ? launch_pdl(four ? cache_read_kernel<128, 4> : cache_read_kernel<128, 1>, grid, block, 0, st, a)
                           : launch_pdl(four ? cache_read_kernel<512, 4> : cache_read_kernel<512, 1>, grid, block, 0, st, a);
    if (err != cudaSuccess) return DSA_ERR_CUDA;
    return launch_status();
}

extern "C" dsa_status_t dsa_cache_append(int32_t batch, const int32_t* cu_new, const int32_t* start_pos, int32_t n,
                                         const void* x, int64_t x_ld, int32_t norm, const float* rms_gamma, float rms_eps,
                                         const dsa_rope_t* rope, const dsa_pool_t* pool, const dsa_block_table_t* bt,
                                         int32_t* dev_status, void* stream) {
    if (batch < 0 || n < 0) return DSA_ERR_INVALID_ARG;
    if (batch == 0 || n == 0) return DSA_OK;
    const dsa_status_t e = check_rows(pool, bt);
    if (e != DSA_OK) return e;
    if (!cu_new || !start_pos || !x || !aligned(x, 16) || x_ld % 8 || x_ld < pool->dim || x_ld >= (1ll << 40) ||
        bt->batch < batch || !rope || rope->rope_dim < 0 || rope->rope_dim > pool->dim || (rope->rope_dim & 1) ||
        !(rope->theta > 0.0) || (norm && !(rms_eps > 0.f)) || !aligned(rms_gamma, 4))
        return DSA_ERR_INVALID_ARG;
    if (rope->rope_dim > 64) return DSA_ERR_UNSUPPORTED;  // the frequency table holds 32 pairs
    const CacheAppendArgs a{batch,   n,    cu_new, start_pos,  static_cast<const uint16_t*>(x),
                            x_ld,    rms_gamma, rms_eps, make_rope_table(rope->rope_dim, rope->theta),
                            *pool,   *bt,  dev_status, aligned(x, 32) && x_ld % 16 == 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t err = pool->dim == 64    ? norm ? launch_append<64, true>(a, st) : launch_append<64, false>(a, st)
                            : pool->dim == 128 ? norm ? launch_append<128, true>(a, st) : launch_append<128, false>(a, st)
                                               : norm ? launch_append<512, true>(a, st) : launch_append<512, false>(a, st);
    if (err != cudaSuccess) return DSA_ERR_CUDA;
    return launch_status();
}
