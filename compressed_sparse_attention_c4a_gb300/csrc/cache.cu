// dsa_cache_write / dsa_cache_read: rows into a paged cache in its storage format, and back as values.
//
// [P1] "DeepSeek DSA、DeepSeek V4与vLLM Hybrid KV Cache详解" §2.2 (logical rows of a request through its block table),
// [P2] "DeepSeek V4 稀疏注意力完全解剖" 设计 1 (256 raw positions per logical block) and 第三层 (prefill keeps the cache
// in bf16, decode quantises it row by row): the caches that a prefill hands over are stored row by row in the decode
// format, and stored rows can be had back as bf16 values.
#include "common.cuh"
#include "rows.cuh"

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
