// dsa_cache_write / dsa_cache_read: rows into a paged cache in its storage format, and back as values.
//
// [P1] "DeepSeek DSA、DeepSeek V4与vLLM Hybrid KV Cache详解" §2.2 (logical rows of a request through its block table),
// [P2] "DeepSeek V4 稀疏注意力完全解剖" 设计 1 (256 raw positions per logical block) and 第三层 (prefill keeps the cache
// in bf16, decode quantises it row by row): the caches that a prefill hands over are stored row by row in the decode
// format, and stored rows can be had back as bf16 values.
#include "common.cuh"
#include "rows.cuh"

namespace dsa {

constexpr int kRowThreads = 256;  // 8 warps, a row each

struct CacheWriteArgs {
    int batch, n;
    const int32_t* cu_new;
    const int32_t* start_row;
    const uint16_t* x;
    dsa_pool_t pool;
    dsa_block_table_t bt;
    int32_t* status;
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

// One warp per row.  The schedule and the block table are read before waiting for the preceding kernel.
template <int DIM>
__global__ void __launch_bounds__(kRowThreads) cache_write_kernel(CacheWriteArgs a) {
    constexpr int E = DIM / 32;
    const int lane = threadIdx.x & 31;
    const long long j = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    long long prow = -1;
    bool live = false;
    if (j < a.n && j < __ldg(a.cu_new + a.batch)) {
        const int r = request_of(a.cu_new, a.batch, (int)j, lane);
        const long long row = (long long)__ldg(a.start_row + r) + (j - __ldg(a.cu_new + r));
        live = true;
        prow = physical_row(a.bt, r, row, a.pool.rows_per_block, a.pool.num_blocks);
    }
    pdl_wait();
    pdl_launch_dependents();
    if (!live) return;
    if (prow < 0) {
        if (lane == 0) report(a.status, DSA_ERR_DEVICE_FAULT);
        return;
    }
    float v[E];
    load_bf16<E>(a.x + j * DIM, lane, v);
    store_row<E>(a.pool, prow, lane, v);
}

struct CacheReadArgs {
    int n;
    const int32_t* req;
    const int32_t* ids;
    dsa_pool_t pool;
    dsa_block_table_t bt;
    uint16_t* out;
    int32_t* status;
};

// The stored row `prow` as the warp's E values per lane.
template <int E>
__device__ __forceinline__ void load_row(const dsa_pool_t& pool, long long prow, int lane, float (&v)[E]) {
    const uint8_t* base = static_cast<const uint8_t*>(pool.data);
    if (pool.dtype == DSA_BF16) {
        load_bf16<E>(reinterpret_cast<const uint16_t*>(base) + prow * (E * 32), lane, v);
        return;
    }
    const float s = pool.scale[prow];
    if (pool.dtype == DSA_FP8_E4M3) {
        const uint8_t* src = base + prow * (E * 32) + lane * E;
        uint16_t c[E / 2];
        if constexpr (E == 16) {
            const uint4 u = *reinterpret_cast<const uint4*>(src);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) c[k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
        } else {
#pragma unroll
            for (int k = 0; k < E / 2; ++k) c[k] = reinterpret_cast<const uint16_t*>(src)[k];
        }
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(c[k], __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            v[2 * k] = s * f.x;
            v[2 * k + 1] = s * f.y;
        }
        return;
    }
    // two e2m1 codes a byte, with a scale per row, or per row and block
    const bool block = pool.dtype == DSA_FP4_BLOCK;
    const uint8_t* row = base + prow * (block ? kFp4BlockRow : E * 16);
    float unit = s;
    if constexpr (E == kFp4Block) {
        if (block) {
            const __half_raw h = __nv_cvt_fp8_to_halfraw(row[256 + lane], __NV_E4M3);
            unit = s * __half2float(*reinterpret_cast<const __half*>(&h));
        }
    }
    uint8_t c[E / 2];
    if constexpr (E == 16) {
        const uint2 u = *reinterpret_cast<const uint2*>(row + lane * 8);
#pragma unroll
        for (int k = 0; k < 8; ++k) c[k] = (uint8_t)((k < 4 ? u.x : u.y) >> (8 * (k & 3)));
    } else {
#pragma unroll
        for (int k = 0; k < E / 2; ++k) c[k] = row[lane * (E / 2) + k];
    }
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(c[k], __NV_E2M1);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[2 * k] = unit * f.x;
        v[2 * k + 1] = unit * f.y;
    }
}

// One warp per row.
template <int DIM>
__global__ void __launch_bounds__(kRowThreads) cache_read_kernel(CacheReadArgs a) {
    constexpr int E = DIM / 32;
    const int lane = threadIdx.x & 31;
    const long long j = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (j >= a.n) return;
    const int id = __ldg(a.ids + j), r = __ldg(a.req + j);
    long long prow = -1;
    if (id >= 0 && r >= 0 && r < a.bt.batch)
        prow = physical_row(a.bt, r, id, a.pool.rows_per_block, a.pool.num_blocks);
    if (prow < 0 && id != -1 && lane == 0) report(a.status, DSA_ERR_DEVICE_FAULT);
    float v[E] = {};
    if (prow >= 0) load_row<E>(a.pool, prow, lane, v);
    uint32_t u[E / 2];
#pragma unroll
    for (int k = 0; k < E / 2; ++k)
        u[k] = (uint32_t)float_to_bf16(v[2 * k]) | ((uint32_t)float_to_bf16(v[2 * k + 1]) << 16);
    uint16_t* dst = a.out + j * DIM + lane * E;
    if constexpr (E == 16) {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(u[0], u[1], u[2], u[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(u[4], u[5], u[6], u[7]);
    } else if constexpr (E == 4) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[1]);
    } else {
        *reinterpret_cast<uint32_t*>(dst) = u[0];
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
    const CacheWriteArgs a{batch, n, cu_new, start_row, static_cast<const uint16_t*>(x), *pool, *bt, dev_status};
    const dim3 grid((unsigned)((n + 7ll) / 8)), block(kRowThreads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t err = pool->dim == 64    ? launch_pdl(cache_write_kernel<64>, grid, block, 0, st, a)
                            : pool->dim == 128 ? launch_pdl(cache_write_kernel<128>, grid, block, 0, st, a)
                                               : launch_pdl(cache_write_kernel<512>, grid, block, 0, st, a);
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
    const CacheReadArgs a{n, req, ids, *pool, *bt, static_cast<uint16_t*>(out), dev_status};
    const dim3 grid((unsigned)((n + 7ll) / 8)), block(kRowThreads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t err = pool->dim == 64    ? launch_pdl(cache_read_kernel<64>, grid, block, 0, st, a)
                            : pool->dim == 128 ? launch_pdl(cache_read_kernel<128>, grid, block, 0, st, a)
                                               : launch_pdl(cache_read_kernel<512>, grid, block, 0, st, a);
    if (err != cudaSuccess) return DSA_ERR_CUDA;
    return launch_status();
}
