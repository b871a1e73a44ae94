// Shared by the attention kernels over bf16 / e4m3 rows (attention.cu) and over 4-bit rows (attention_fp4.cu): their
// arguments, small PTX wrappers, the merge of a cluster's partial outputs and the store.
#pragma once

#include "common.cuh"
#include "rows.cuh"
#include "topk_cluster.cuh"

namespace dsa {

constexpr int kD = 512;
constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
    int rows, heads, hg_count, nsplit, cps;   // cps = the kernel's key tiles per split
    const uint16_t* q;
    const int32_t* q_pos;
    const int32_t* q_req;                     // NULL: row r belongs to request r
    int kind_w, kind_s;
    const int32_t* topk;                      // NULL: every visible entry
    int k;
    dsa_pool_t main;
    dsa_block_table_t main_bt;
    dsa_pool_t swa;
    dsa_block_table_t swa_bt;
    int window;
    float scale_log2;                         // sm_scale * log2(e)
    RopeTable rope;
    uint16_t* out;                            // bf16 output, or NULL with out8
    uint8_t* out8;                            // e4m3 output [rows][heads][512] (with out_scale), or NULL
    float* out_scale;                         // [rows][heads][4]: amax / 448 of each 128-dim block
    float* lse;
    float* ws_o;                              // [rows][nsplit][heads][512]
    float* ws_ml;                             // [rows][nsplit][heads][4]: M, L (bf16 P), E (fp32 P), 0
    const float* scores;                      // fused top-k: indexer scores [rows][score_ld]
    int score_ld;
    const int32_t* n_valid;                   // fused top-k: [rows] valid scores of a row
    int32_t* topk_out;                        // fused top-k: the selected entries [rows][k]
    int nans;                                 // a sum that is NaN makes the row NaN (4-bit rows), else it counts as empty
    int stall_row;                            // test hook: this row's last CTAs never see their queries arrive (-1: none)
    int32_t* status;
};

// ---- PTX wrappers ---------------------------------------------------------------------
__device__ __forceinline__ void cp_async16_hint(uint32_t dst, const void* src, uint32_t src_bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(src_bytes),
                 "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_group() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return (uint32_t)float_to_bf16(lo) | ((uint32_t)float_to_bf16(hi) << 16);
}
// {lo, hi} -> bf16x2 in one conversion (round to nearest even, as pack_bf16), lo in the low half.
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// 2^x on the special-function unit (PTX ex2.approx.ftz: a few ulp, 2^-inf = 0); for softmax
// probabilities, which enter the product rounded to bf16.
__device__ __forceinline__ float ex2_sfu(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr int kClThreads = 512;             // 16 warps: 4 softmax, MW issuing MMAs, the rest gathering
constexpr float kLazyLog2 = 8.f;            // the running maximum moves when exceeded by more than this
constexpr int kBtCache = 1024;              // main block tables up to this many blocks are cached in shared memory
constexpr int kFusedK = 512;                // the fused top-k + attention kernel: k up to this
constexpr int kFusedVpt = 8;                // ... scores per thread: rows up to 4 * 512 * 8 = 16,384 entries
static_assert(kClThreads == 512, "16 warps");

// Byte offset of element (row r, element e) in a tile of 128B-swizzled atoms whose rows are 128 bytes
// (64 bf16) long: atoms of 8 rows are 1024 bytes apart, 64-element chunks `chunk_stride` apart.
__device__ __forceinline__ uint32_t sw128_offset(int r, int e, int chunk_stride) {
    const int c = e >> 6, in = e & 63;
    return (uint32_t)(c * chunk_stride + (r >> 3) * 1024 + (r & 7) * 128 + ((((in >> 3) ^ (r & 7))) << 4) +
                      ((in & 7) << 1));
}

// ---- merge across the cluster and store, after a CTA's last product ----------------------------------------------------
// O^T of the CTA sits in TMEM at tO ([4 tiles of 128 dims][NH heads]), its (m, l, e) per head at L::kOffOwn.  Tile t
// belongs to CTA t mod csize: each CTA sends the tiles that others own, the owner weighs every CTA's partial by
// 2^(m_c - M), divides by L, rotates by R_m^-1 and stores (or writes an fp32 partial when the row has several splits).
// SCALE_LOG2: O^T is 2^-SCALE_LOG2 of the output.  NANS: a sum that is NaN makes the row's output and lse NaN (else such a
// partial counts as empty).  Called by all 512 threads; frees the TMEM columns.
template <int NH, class L, bool FUSED, int SCALE_LOG2 = 0, bool NANS = false>
__device__ __forceinline__ void attn_finish(const AttnArgs& a, const CUtensorMap* omap, uint8_t* smem, uint32_t tmem,
                                            uint32_t tO, int row, int split, int hg, int crank, int csize, int n_mine,
                                            bool ok) {
    constexpr float kOScale = (float)(1 << SCALE_LOG2);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int* s_vote = reinterpret_cast<int*>(smem + L::kOffVote);
    float* s_own = reinterpret_cast<float*>(smem + L::kOffOwn);
    float* s_fac = reinterpret_cast<float*>(smem + L::kOffFac);  // [4][NH]: weight of each CTA's partial
    float* s_inv = s_fac + 4 * NH;
    float* s_M = s_inv + NH;
    float* s_L = s_M + NH;
    float* s_E = s_L + NH;
    float* s_rc = reinterpret_cast<float*>(smem + L::kOffRope);
    uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + L::kOffXfull);  // [3] each received tile slot loaded
    volatile int* s_fault = reinterpret_cast<volatile int*>(smem + L::kOffFault);
    auto some = [](float x) { return NANS ? !(x <= 0.f) : x > 0.f; };
    tc_fence_before();
    const bool all_ok = __syncthreads_and(ok);  // O^T complete (the softmax warps waited for it); s_own set
    tc_fence_after();
    if (tid == 0) DSA_STAMP(8);
    const bool have = n_mine > 0 && all_ok;
    constexpr int G = NH / 4;                    // heads per finishing thread (a TMEM load of G columns)
    const int quad = warp & 3, quarter = warp >> 2;
    const int d = quad * 32 + lane, h0 = quarter * G;  // thread: dim d of a 128-dim tile, heads h0 .. h0 + G
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int tiles_per = 4 / csize;
    auto tmem_cols = [&](int t, float (&v)[G]) {
        if constexpr (G == 16) tmem_ld16(tO + t * NH + lane_off + h0, v);
        else if constexpr (G == 8) tmem_ld8(tO + t * NH + lane_off + h0, v);
        else tmem_ld4(tO + t * NH + lane_off + h0, v);
    };
    auto tmem_cols_nowait = [&](int t, float (&v)[G]) { tmem_ld_nowait<G>(tO + t * NH + lane_off + h0, v); };
    // Tiles this CTA sends sit at [0, 3 tiles) of shared memory (the query rows, idle now), the tiles it
    // receives at [3, 6 tiles) (query rows and key stages); each as [NH / 4 head quads][128 dims] x 4 bf16.
    uint8_t* xout = smem + L::kOffQ;
    uint8_t* xin = smem + L::kOffQ + 3 * L::kTile;
    if (csize > 1) {
        // 1. the tiles other CTAs own, unscaled (the owner applies this CTA's factor), staged as bf16 (half the bytes of
        // fp32, in shared memory as between the CTAs, for 2^-8 of each partial: a rounding like the output's own); only this
        // CTA's own accumulators are needed, so no CTA waits for another here
        float v[4][G];  // static register indices; the sent tiles' columns in flight together
        if (have) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t % csize != crank) tmem_cols_nowait(t, v[t]);
            tmem_wait_ld();
#pragma unroll
            for (int t = 0; t < 4; ++t) tmem_regs_after_wait<G>(v[t]);
        }
        if (tid == 0) DSA_STAMP(15);
        int sl = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t % csize == crank) continue;
#pragma unroll
            for (int q4 = 0; q4 < G / 4; ++q4)
                *reinterpret_cast<uint2*>(xout + sl * L::kTile + ((h0 / 4 + q4) * 128 + d) * 8) =
                    have ? make_uint2(bf16x2_rn(v[t][4 * q4], v[t][4 * q4 + 1]), bf16x2_rn(v[t][4 * q4 + 2], v[t][4 * q4 + 3]))
                         : make_uint2(0u, 0u);
            ++sl;
        }
        if (tid == 0) DSA_STAMP(16);
        fence_proxy_async_smem();  // staged tiles -> async proxy (the bulk copies after the cluster barrier)
    }
    if (tid == 0) DSA_STAMP(9);
    // 2. (m, l, e, fault) per head to every CTA of the cluster
    if constexpr (!FUSED)
        if (csize > 1) cluster_wait();  // phase 0: every CTA of the cluster has started (fused: waited above)
    if (tid == 0) DSA_STAMP(17);
    if (csize > 1 && tid == 0)  // before any peer can push (pushes follow phase 1)
        for (int b = 0; b < (csize - 1) * tiles_per; ++b) mbar_arrive_expect_tx(&xfull[b], (uint32_t)L::kTile);
    // this CTA met a device fault, or a wait of its ran out: the whole row is written as zeros
    const float fo = *s_fault || !all_ok ? 1.f : 0.f;
    for (int h = tid; h < NH; h += kClThreads) {
        const uint32_t dst = smem_u32(smem + L::stat(crank, h));
        const float mo = have ? s_own[h] : -INFINITY, lo = have ? s_own[NH + h] : 0.f,
                    eo = have ? s_own[2 * NH + h] : 0.f;
        if (csize == 1)
            *reinterpret_cast<float4*>(smem + L::stat(0, h)) = make_float4(mo, lo, eo, fo);
        else
            for (int q = 0; q < csize; ++q)
                st_cluster_v4(mapa_shared(dst, (uint32_t)q), mo, lo, eo, fo);
    }
    if (tid == 0) DSA_STAMP(18);
    if (csize > 1) {
        cluster_arrive();  // phase 1: statistics delivered, sent tiles staged, every CTA's products complete
        cluster_wait();
    } else {
        __syncthreads();  // one CTA: the statistics in its own shared memory, its products complete
    }
    if (tid == 0) DSA_STAMP(10);
    // 3. push: one bulk copy per sent tile, all from lane 0 of the last warp (the first warps compute the
    // factors meanwhile), the next CTA's tiles first, then the one after: every owner receives one CTA's tiles at
    // a time, each tile signalling its own slot, so the owner adds the first arrivals while the rest stream in
    const bool pusher = csize > 1 && warp == 15 && lane == 0;
    if (pusher) {
        for (int k = 1; k < csize; ++k) {
            const int o = (crank + k) % csize;
            for (int t = 0, sl = 0; t < 4; ++t) {
                if (t % csize == crank) continue;
                if (t % csize == o) {
                    const int slot = ((crank - o - 1 + csize) % csize) * tiles_per + t / csize;  // in the owner's xin
                    bulk_s2cluster(mapa_shared(smem_u32(xin + slot * L::kTile), (uint32_t)o),
                                   smem_u32(xout + sl * L::kTile), L::kTile,
                                   mapa_shared(smem_u32(&xfull[slot]), (uint32_t)o));
                }
                ++sl;
            }
        }
        bulk_commit();
    }
    // 4. per head: the cluster maximum M, each CTA's weight 2^(m_c - M), 1 / L; one thread per (head, CTA),
    // the four of a head in neighbouring lanes
    if (tid < NH * 4) {
        const int h = tid >> 2, qq = tid & 3;
        const bool in = qq < csize;
        const float4 st = in ? *reinterpret_cast<const float4*>(smem + L::stat(qq, h))
                             : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        float M = fmaxf(st.x, __shfl_xor_sync(0xffffffffu, st.x, 1));
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 2));
        int fault = st.w != 0.f;
        fault |= __shfl_xor_sync(0xffffffffu, fault, 1);
        fault |= __shfl_xor_sync(0xffffffffu, fault, 2);
        const float fq = (st.x == -INFINITY || fault) ? 0.f : exp2f(st.x - M);
        float Ls = fq != 0.f ? st.y * fq : 0.f, Es = fq != 0.f ? st.z * fq : 0.f;
        Ls += __shfl_xor_sync(0xffffffffu, Ls, 1);
        Es += __shfl_xor_sync(0xffffffffu, Es, 1);
        Ls += __shfl_xor_sync(0xffffffffu, Ls, 2);
        Es += __shfl_xor_sync(0xffffffffu, Es, 2);
        if (in) s_fac[qq * NH + h] = fq;
        if (qq == 0) {
            s_inv[h] = some(Ls) ? kOScale / Ls : 0.f;
            s_M[h] = fault ? -INFINITY : M;
            s_L[h] = Ls;
            s_E[h] = Es;
            if (h == 0) s_vote[0] = fault;  // (the softmax votes are done) the row's fault flag for the partials
        }
    }
    if (tid == 0) DSA_STAMP(19);
    if (csize > 1) {
        // the factors reach every thread; the pushing warp (15, still issuing its copies one after another)
        // joins through a barrier of its own with the factor threads, so that the others need not wait for it
        static_assert(kClThreads == 512, "warps 0-14 and warp 15");
        if (tid < NH * 4) named_bar_arrive(4, NH * 4 + 32);
        if (warp == 15) {
            __syncwarp();  // lane 0 has issued the pushes
            named_bar_sync(4, NH * 4 + 32);
        } else {
            named_bar_sync(3, kClThreads - 32);
        }
    } else {
        __syncthreads();
    }
    if (tid == 0) DSA_STAMP(11);
    // this CTA's first owned tile leaves TMEM while the other CTAs' tiles are still arriving
    float v_first[G];
    if (have) tmem_cols(crank, v_first);
    if (tid == 0) DSA_STAMP(12);
    // ---- owner: finish each owned tile; bf16 output staged as [NH][128] in the P^T buffers and stored
    // with 16-byte writes, or fp32 split partials ------------------------------------------------------
    float inv[G], fown[G];
#pragma unroll
    for (int e = 0; e < G; e += 4) {
        const float4 b4 = *reinterpret_cast<const float4*>(s_inv + h0 + e);
        const float4 a4 = *reinterpret_cast<const float4*>(s_fac + crank * NH + h0 + e);
        inv[e] = b4.x, inv[e + 1] = b4.y, inv[e + 2] = b4.z, inv[e + 3] = b4.w;
        fown[e] = a4.x, fown[e + 1] = a4.y, fown[e + 2] = a4.z, fown[e + 3] = a4.w;
    }
    // output staging: a buffer of [NH][128] bf16 for each owned tile (the P^T buffers, and key stages that no received
    // tile uses, idle by now), each stored by one TMA box
    uint8_t* const ob0 = smem + L::kOffP;
    uint8_t* const ob1 = smem + L::kOffOut1;
    static_assert(L::kOffOut1 + 3 * NH * 256 <= L::kOffP, "the other tiles' buffers end before the P^T buffers");
    const int firstd = kD - a.rope.rope_dim;
    const bool odd = lane & 1;
    float v_next[G];  // the next owned tile's columns, loaded from TMEM while this one is finished and stored
#pragma unroll 1
    for (int j = 0; j < tiles_per; ++j) {
        const int t = crank + csize * j;
        const int D = t * 128 + d;
        float v[G];
        if (have) {
            if (j == 0) {
#pragma unroll
                for (int e = 0; e < G; ++e) v[e] = v_first[e];
            } else {
                tmem_wait_ld();
                tmem_regs_after_wait<G>(v_next);
#pragma unroll
                for (int e = 0; e < G; ++e) v[e] = v_next[e];
            }
            if (j + 1 < tiles_per) tmem_cols_nowait(t + csize, v_next);
        }
        if (tid == 0 && j == 0) DSA_STAMP(20);
#pragma unroll
        for (int e = 0; e < G; ++e) v[e] = have && (!NANS || fown[e] != 0.f) ? v[e] * fown[e] : 0.f;
        // received tiles in the order they arrive: slot si holds CTA crank + 1 + si's, and CTA crank - 1 (the
        // last si) sends to this CTA first
#pragma unroll
        for (int sr = 0; sr < 3; ++sr) {
            const int si = csize - 2 - sr;
            if (si >= 0) {
                const int src = (crank + 1 + si) % csize;
                const float* fsrc = s_fac + src * NH + h0;
                const uint8_t* p = xin + (si * tiles_per + j) * L::kTile;
                const bool landed = mbar_wait_bounded(&xfull[si * tiles_per + j], 0, kWaitLimitNs);
                if (!landed && tid == 0) report(a.status, DSA_ERR_TIMEOUT);
                ok = ok && landed;
#pragma unroll
                for (int q4 = 0; q4 < G / 4; ++q4) {
                    uint2 w = *reinterpret_cast<const uint2*>(p + ((h0 / 4 + q4) * 128 + d) * 8);
                    const float4 f4 = *reinterpret_cast<const float4*>(fsrc + 4 * q4);
                    if constexpr (NANS) {  // a partial without weight may hold NaN
                        if (f4.x == 0.f) w.x &= 0xFFFF0000u;
                        if (f4.y == 0.f) w.x &= 0x0000FFFFu;
                        if (f4.z == 0.f) w.y &= 0xFFFF0000u;
                        if (f4.w == 0.f) w.y &= 0x0000FFFFu;
                    }
                    v[4 * q4] = fmaf(f4.x, __uint_as_float(w.x << 16), v[4 * q4]);
                    v[4 * q4 + 1] = fmaf(f4.y, __uint_as_float(w.x & 0xFFFF0000u), v[4 * q4 + 1]);
                    v[4 * q4 + 2] = fmaf(f4.z, __uint_as_float(w.y << 16), v[4 * q4 + 2]);
                    v[4 * q4 + 3] = fmaf(f4.w, __uint_as_float(w.y & 0xFFFF0000u), v[4 * q4 + 3]);
                }
            }
        }
        if (a.nsplit == 1) {
            uint8_t* const obuf = j == 0 ? ob0 : ob1 + (j - 1) * (NH * 256);
            uint32_t* o32 = reinterpret_cast<uint32_t*>(obuf);
            const int De = D & ~1;  // the pair's even dim
            float rc = 1.f, rs = 0.f;
            if (De >= firstd) {
                rc = s_rc[De - firstd];
                rs = s_rc[De - firstd + 1];
            }
            // neighbouring lanes swap one value per pair of heads: the even lane then holds dims (De, De + 1) of
            // head 2p, the odd lane those of head 2p + 1; each rotates its pair by R_m^-1 and stores it packed
            float rr[G];
#pragma unroll
            for (int pp = 0; pp < G / 2; ++pp) {
                const float x0 = v[2 * pp] * inv[2 * pp], x1 = v[2 * pp + 1] * inv[2 * pp + 1];
                const float recv = __shfl_xor_sync(0xffffffffu, odd ? x0 : x1, 1);
                const float lo = odd ? recv : x0, hi = odd ? x1 : recv;
                rr[2 * pp] = lo * rc + hi * rs;
                rr[2 * pp + 1] = hi * rc - lo * rs;
            }
            if (!a.out8) {
#pragma unroll
                for (int pp = 0; pp < G / 2; ++pp)
                    o32[(h0 + 2 * pp + (odd ? 1 : 0)) * 64 + (d >> 1)] = bf16x2_rn(rr[2 * pp], rr[2 * pp + 1]);
            } else {
                // e4m3 ([P2] 融合点 2: the inverse rotation and the fp8 quantisation in one pass): each head's 128
                // dims of this tile share a scale amax / 448; the amax of a head is reduced over the lanes of its
                // parity, then over the quarter's four warps in shared memory (the statistics slots, free now)
                unsigned* s_amax = reinterpret_cast<unsigned*>(s_own);
                if (tid < NH) s_amax[tid] = 0u;
                __syncthreads();
#pragma unroll
                for (int pp = 0; pp < G / 2; ++pp) {
                    float am = fmaxf(fabsf(rr[2 * pp]), fabsf(rr[2 * pp + 1]));
#pragma unroll
                    for (int o = 2; o < 32; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
                    if (lane < 2) atomicMax(&s_amax[h0 + 2 * pp + lane], __float_as_uint(am));
                }
                __syncthreads();
                uint16_t* o16 = reinterpret_cast<uint16_t*>(obuf);  // [NH][128] e4m3 codes
#pragma unroll
                for (int pp = 0; pp < G / 2; ++pp) {
                    const int hh = h0 + 2 * pp + (odd ? 1 : 0);
                    const float am = __uint_as_float(s_amax[hh]);
                    const float sc = am > 0.f ? am / 448.f : 1.f;
                    o16[hh * 64 + (d >> 1)] =
                        (uint16_t)(float_to_e4m3(rr[2 * pp] / sc) | ((uint32_t)float_to_e4m3(rr[2 * pp + 1] / sc) << 8));
                }
                if (tid < NH) {
                    const float am = __uint_as_float(s_amax[tid]);
                    a.out_scale[((long long)row * a.heads + hg * NH + tid) * 4 + t] = am > 0.f ? am / 448.f : 1.f;
                }
            }
            if (tid == 0 && j == 0) DSA_STAMP(21);
            fence_proxy_async_smem();  // staged output -> async proxy (the TMA store)
            __syncthreads();
            if (tid == 0 && j == 0) DSA_STAMP(22);
            if (tid == 0) {  // NH rows of 128 dims -> out[row][hg * NH .. + NH][t * 128 .. + 128]
                tma_store_2d(omap, t * 128, row * a.heads + hg * NH, obuf);
                bulk_commit();
            }
        } else {
            const long long base0 = ((long long)row * a.nsplit + split) * a.heads + hg * NH + h0;
#pragma unroll
            for (int e = 0; e < G; ++e) a.ws_o[(base0 + e) * kD + D] = kOScale * v[e];
        }
    }
    if (crank == 0) {
        for (int h = tid; h < NH; h += kClThreads) {
            const float Ls = s_L[h], M = s_M[h], Es = s_E[h];
            if (a.nsplit == 1) {
                if (a.lse) a.lse[(long long)row * a.heads + hg * NH + h] = some(Es) ? (M + log2f(Es)) / kLog2e : -INFINITY;
            } else {
                const long long b = ((long long)row * a.nsplit + split) * a.heads + hg * NH + h;
                a.ws_ml[b * 4 + 0] = some(Ls) ? M : -INFINITY;
                a.ws_ml[b * 4 + 1] = Ls;
                a.ws_ml[b * 4 + 2] = Es;
                a.ws_ml[b * 4 + 3] = s_vote[0] ? 1.f : 0.f;  // a faulted split zeroes the row in the combine
            }
        }
    }
    if (tid == 0) DSA_STAMP(13);
    if (pusher || tid == 0) bulk_wait_all();  // this CTA's shared memory is no longer read by its copies / stores
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) {
        DSA_STAMP(14);
        DSA_STAMP_NS(30);
    }
    if (warp == 0) tmem_dealloc(tmem, L::kTmemCols);
}

// The kernel over DSA_FP4_BLOCK rows (attention_fp4.cu) for a plan of cl CTAs per cluster, heads per CTA hg.
dsa_status_t launch_attn_fp4(const AttnArgs& a, int hg, int cl, cudaStream_t st);
// Clusters of cl (1, 2 or 4) of its CTAs that the current device holds at once.
int fp4_clusters(int cl);
// Tensor maps of the query rows and of the output (attention.cu).
bool make_bf16_map(CUtensorMap* map, const void* base, uint64_t rows, int box_rows);
bool make_out_map(CUtensorMap* map, void* base, uint64_t rows, int box_rows, bool e4m3);
cudaError_t launch_attn_combine(const AttnArgs& a, cudaStream_t st);
constexpr int kFp4Keys = 48;  // keys per tile of that kernel

}  // namespace dsa
