// dsa_sparse_attn_* over DSA_FP4_BLOCK rows: MQA attention over gathered 4-bit rows plus the sliding window, K = V,
// with the inverse-RoPE epilogue fused into the store.
//
// [P1] "DeepSeek DSA、DeepSeek V4与vLLM Hybrid KV Cache详解" §4.2-4.3, §5.3; [P2] "DeepSeek V4 稀疏注意力完全解剖" 机制一,
// 机制四, 深潜 (Inverse RoPE), 第三层 (a quantised decode cache): out = R_m^-1 sum_j p_j k_j, p = softmax(<q, k_j> sm),
// k_j = s_j bs_{j, d/16} c_{j, d} with e2m1 codes c, e4m3 block scales bs and a power-of-two row scale s.
//
// A code times its block scale has at most 6 significant bits, so the rows are widened to bf16 exactly and both products
// run on bf16 tensor cores; the row scale multiplies the key's logit and its probability (a power of two: no rounding).
#include "attention.cuh"

namespace dsa {

// Work split as the bf16 kernel (attention.cu): a cluster of CL CTAs per (query row, group of NH <= 64 heads, key split),
// tile i of a CTA being the split's tile crank + CL i of 64 keys.  Inside a CTA, 16 warps:
//   warps 8-15  widen: each owns 8 keys of every tile.  Lanes 0-7 resolve the keys (top-k index -> block table -> row)
//               two tiles ahead, every lane loads 8 code bytes and one block scale of each row straight into registers
//               (two tiles in flight, nothing staged), and once the key stage is free (its P V is done) the codes become
//               bf16 and are stored 128B-swizzled as [64-dim chunk][64 keys][128 B];
//   warp 4      S = Q K^T (M = 64 heads, N = 64 keys);
//   warp 5      O^T += V^T P^T (four tiles of M = 128 dims, N = NH heads, K = 64 keys);
//   warps 0-3   softmax: 16 heads a warp, a head's 64 logits over the 4 lanes of a quad (the 16-lane TMEM load spreads a
//               row over a quad, so every lane works although M = 64 fills 16 of the 32 TMEM lanes).
// Two key stages, two S and two P buffers: S of tile i + 1 and the widening of tile i + 2 overlap the softmax and P V of i.
// A 64-key tile reads Q (64 KB) half as often per key as a 32-key one and issues N = 64 products, whose rate is the tensor
// pipe's and not the issuing warp's.
constexpr int kFp4Stage = kFp4Keys * kD * 2;
constexpr int kFp4Widen = 8;                           // widening warps
constexpr int kFp4PerWarp = kFp4Keys / kFp4Widen;      // keys of a tile per widening warp
constexpr int kFp4WidenThreads = 32 * kFp4Widen;
static_assert(kFp4PerWarp == 8, "lanes 0-7 resolve a warp's keys, its bits are one byte of the tile's mask");
// Widened values carry 2^-8: e2m1 bits placed in a bf16 are 2^-126 of the value, and the factor that undoes it times a
// block scale of up to 448 must stay below 2^128, so it is 2^118.
constexpr int kFp4Shift = 8;

template <int NH>
struct Fp4Smem {
    static constexpr int kQ = 64 * kD * 2;                          // [8][64 rows][128 B]
    static constexpr int kP = NH * 128;                             // [NH rows][64 keys] bf16
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kQ;                        // key stages; received tiles
    static constexpr int kOffP = kOffK + 2 * kFp4Stage;             // two P^T buffers; output staging at the end
    static constexpr int kOffKsc = kOffP + 2 * kP;                  // float [2][32][4]: see s_ksc
    static constexpr int kOffMask = kOffKsc + 2 * kFp4Keys * 8;     // uint64 [2]: valid keys of a stage
    static constexpr int kOffAlpha = kOffMask + 16;                 // float [2][NH]
    static constexpr int kOffVote = kOffAlpha + 2 * NH * 4;         // int [2][4]
    static constexpr int kOffOwn = kOffVote + 32;                   // float m[NH], l[NH], e[NH] of this CTA
    static constexpr int kOffStat = kOffOwn + 3 * NH * 4;           // float [4 ranks][NH][4]: (m, l, e, fault)
    static constexpr int kOffFac = kOffStat + 4 * NH * 16;          // float f[4 ranks][NH], 1/L, M, L, E [NH]
    static constexpr int kOffBt = kOffFac + 8 * NH * 4;             // int [kBtCache]: the request's main block table
    static constexpr int kOffSwb = kOffBt + kBtCache * 4;           // int [8]: window-pool blocks from that of wlo
    static constexpr int kOffFault = kOffSwb + 32;                  // int: a key of this CTA hit a device fault
    static constexpr int kOffRope = kOffFault + 16;                 // float [32][2]: cos, sin of each pair's angle at m
    static constexpr int kOffBar = kOffRope + 256;                  // 14 mbarriers, TMEM address
    static constexpr int kOffXfull = kOffBar + 11 * 8;              // the last three: received tile slots
    static constexpr int kOffTopk = kOffBar + 14 * 8 + 16;          // int [kFusedK]: the row's top-k (fused)
    static constexpr int kBytes = kOffTopk + kFusedK * 4;
    static constexpr int kAlloc = kBytes + 1024;                    // + alignment slack
    static constexpr int kOffOut1 = kOffK + kFp4Stage;              // second output staging buffer (the second stage)
    static_assert(kAlloc <= 227 * 1024, "shared memory per CTA");
    static_assert(kOffKsc % 16 == 0 && kOffMask % 16 == 0 && kOffAlpha % 16 == 0 && kOffVote % 16 == 0 &&
                      kOffOwn % 16 == 0 && kOffStat % 16 == 0 && kOffFac % 16 == 0 && kOffBt % 16 == 0 &&
                      kOffSwb % 16 == 0 && kOffFault % 16 == 0 && kOffRope % 16 == 0 && kOffBar % 16 == 0 &&
                      kOffTopk % 16 == 0,
                  "shared-memory regions 16-byte aligned");
    static constexpr int kTile = 128 * NH * 2;                      // one exchanged 128-dim O tile: [NH / 4][128] x 4 bf16
    static_assert(3 * kTile <= kQ, "the sent tiles fit in the query rows");
    static_assert(6 * kTile <= kQ + kFp4Stage, "the received tiles fit before the second output buffer");
    static_assert(NH * 128 * 2 <= 2 * kP, "an output tile must fit in the P^T buffers");
    static_assert(sizeof(TopkRowScratch<kClThreads, kFusedVpt, 4>) <= 2 * kFp4Stage, "the fused top-k's scratch");
    static constexpr int kTmemCols = 512;  // S: [2 buffers][64 keys]; O^T: [4 tiles][NH heads]
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// e4m3 byte -> bf16x2 of 2^118 times its value in both halves (exact, subnormal scales included): the byte's bits in a
// bf16 are 2^-120 of the value, and two multiplications by 2^127 and 2^111 restore the exponent.
__device__ __forceinline__ uint32_t block_scale_2p118(uint32_t byte) {
    return mul_bf16x2(mul_bf16x2(byte * 0x00100010u, 0x7F007F00u), 0x77007700u);
}

// Eight e2m1 codes (element j in nibble j) times the scale -> four words of two bf16 in element order.  A code's bits
// s ee m placed at bits 15, 8..6 of a bf16 are 2^-126 of its value, zero and 0.5 included (a bf16 subnormal): nibbles k
// and k + 4 shifted together to bit 6 and copied to bit 12 by one multiplication, then masked.  No conversion
// instruction: measured, those cost twice as much per value.
__device__ __forceinline__ void widen8(uint32_t w, uint32_t scale, uint32_t (&o)[4]) {
    const uint32_t v = w >> 8;
    uint32_t g[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t x = ((k & 2 ? v : w) * (k & 1 ? 4u : 64u)) & 0x03C003C0u;
        g[k] = mul_bf16x2((x * 65u) & 0x81C081C0u, scale);
    }
    o[0] = __byte_perm(g[0], g[1], 0x5410);
    o[1] = __byte_perm(g[2], g[3], 0x5410);
    o[2] = __byte_perm(g[0], g[1], 0x7632);
    o[3] = __byte_perm(g[2], g[3], 0x7632);
}

// 8 code bytes / one block scale of a row, zero when the key is masked (row < 0).
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int row, uint64_t policy) {
    uint2 c;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ge.s32 p, %4, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\t"
        "@p ld.global.L1::no_allocate.L2::cache_hint.v2.u32 {%0, %1}, [%2], %3;\n\t}"
        : "=&r"(c.x), "=&r"(c.y)
        : "l"(p), "l"(policy), "r"(row)
        : "memory");
    return c;
}
__device__ __forceinline__ uint32_t load_block_scale(const uint8_t* p, int row, uint64_t policy) {
    uint32_t b;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ge.s32 p, %3, 0;\n\tmov.u32 %0, 0;\n\t"
        "@p ld.global.L1::no_allocate.L2::cache_hint.u8 %0, [%1], %2;\n\t}"
        : "=&r"(b)
        : "l"(p), "l"(policy), "r"(row)
        : "memory");
    return b;
}

// 64 columns of a 16-lane accumulator (M = 64): lane 4 r + c of the warp gets, for row r and r + 8, columns
// 8 i + 2 c, 8 i + 2 c + 1 in registers 4 i, 4 i + 1 and 4 i + 2, 4 i + 3.  Valid after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld_16x64_nowait(uint32_t taddr, float (&v)[32]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// Two fp32 values in one register pair (packed arithmetic halves the instructions of the softmax).
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float* lo, float* hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

template <int NH, bool FUSED>
__global__ void __launch_bounds__(kClThreads, 1)
    attn_fp4_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap omap, AttnArgs a) {
    using L = Fp4Smem<NH>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sQ = smem_u32(smem + L::kOffQ), sK = smem_u32(smem + L::kOffK), sP = smem_u32(smem + L::kOffP);
    // the row scales of keys 2 p and 2 p + 1 of a stage, then the same times sm_scale log2(e)
    float* s_ksc = reinterpret_cast<float*>(smem + L::kOffKsc);
    uint8_t* s_mask8 = smem + L::kOffMask;
    float* s_alpha = reinterpret_cast<float*>(smem + L::kOffAlpha);
    int* s_vote = reinterpret_cast<int*>(smem + L::kOffVote);
    float* s_own = reinterpret_cast<float*>(smem + L::kOffOwn);
    // tile i: key stage, S columns and P^T buffer i & 1
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);  // [2] stage widened (widening warps)
    uint64_t* sfull = full + 2;                                         // [2] S in TMEM
    uint64_t* pfull = sfull + 2;                                        // [2] P^T written (4 softmax warps)
    uint64_t* pvdone = pfull + 2;                                       // [2] O^T += V^T P^T done
    uint64_t* qfull = pvdone + 2;                                       // query rows loaded
    uint64_t* rdone = qfull + 1;                                        // O^T rescaled (4 softmax warps)
    uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + L::kOffXfull);  // [3] each received tile slot loaded
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(xfull + 3);
    volatile int* s_fault = reinterpret_cast<volatile int*>(smem + L::kOffFault);
    float* s_rc = reinterpret_cast<float*>(smem + L::kOffRope);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int crank = (int)cluster_ctarank(), csize = (int)cluster_nctarank();
    const int cid = blockIdx.x / csize;
    const int split = cid % a.nsplit;
    const int hg = (cid / a.nsplit) % a.hg_count;
    const int row = cid / (a.nsplit * a.hg_count);
    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(&full[b], kFp4Widen);
            mbar_init(&sfull[b], 1);
            mbar_init(&pfull[b], 4);
            mbar_init(&pvdone[b], 1);
        }
        mbar_init(qfull, 1);
        mbar_init(rdone, 4);
        for (int b = 0; b < 3; ++b) mbar_init(&xfull[b], 1);
        *s_fault = 0;
        fence_barrier_init();
    }
    if constexpr (NH < 64)  // the S product reads 64 query rows: rows NH.. are zero
        for (int i = tid; i < 8 * (64 - NH) * 8; i += kClThreads) {
            const int c = i / ((64 - NH) * 8), rr = NH + (i / 8) % (64 - NH), u = i % 8;
            *reinterpret_cast<uint4*>(smem + L::kOffQ + c * 8192 + rr * 128 + u * 16) = make_uint4(0, 0, 0, 0);
        }
    fence_proxy_async_smem();
    if (warp == 0) tmem_alloc(s_tmem, L::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const uint32_t tS = tmem, tO = tmem + 2 * kFp4Keys;
    if (csize > 1) cluster_arrive_relaxed();  // phase 0: this CTA has started (waited on before DSMEM use)

    // Position, request, block tables and query rows: inputs that no kernel of the layer step writes, read while the
    // preceding kernel finishes.  Top-k indices, cache rows and every output come after the wait.
    const int r = a.q_req ? a.q_req[row] : row;
    const int ww = warp - 8, gt = tid - 256;  // widening warp and thread
    const bool bt_cached = a.main_bt.max_blocks <= kBtCache;
    constexpr int kBtPer = kBtCache / kFp4WidenThreads;
    int btv[kBtPer];
    if (ww >= 0) {
        const bool r_in = bt_cached && r >= 0 && r < a.main_bt.batch;
#pragma unroll
        for (int u = 0; u < kBtPer; ++u) {
            const int b = gt + u * kFp4WidenThreads;
            btv[u] = r_in && b < a.main_bt.max_blocks ? __ldg(a.main_bt.table + (long long)r * a.main_bt.max_blocks + b) : -1;
        }
    }
    const int m = a.q_pos[row];
    const bool row_ok = r >= 0 && r < a.main_bt.batch && r < a.swa_bt.batch && m >= 0;
    if (!row_ok && tid == 0) *s_fault = 1;
    const int n_vis = row_ok ? entries_formed((long long)m + 1, a.kind_w, a.kind_s) : 0;
    const int n_comp = (FUSED || a.topk) ? a.k : n_vis;
    const int wlo = max(0, m - a.window + 1);
    const int n_keys = row_ok ? n_comp + (m - wlo + 1) : 0;
    const int n_tiles = (n_keys + kFp4Keys - 1) / kFp4Keys;
    const int g_lo = split * a.cps, g_hi = min(n_tiles, g_lo + a.cps);
    const int n_mine = g_hi > g_lo + crank ? (g_hi - g_lo - crank + csize - 1) / csize : 0;
    int* s_bt = reinterpret_cast<int*>(smem + L::kOffBt);
    int* s_swb = reinterpret_cast<int*>(smem + L::kOffSwb);
    if (warp == 0 && lane < a.rope.rope_dim / 2) {  // R_m^-1 of the output: cos and sin of each pair's angle at m
        float c = 1.f, sn = 0.f;
        if (row_ok) rope_cos_sin(m, a.rope, lane, &c, &sn);
        s_rc[2 * lane] = c;
        s_rc[2 * lane + 1] = sn;
    }
    if (warp == 4 && n_mine > 0) {  // the query rows, one 64-dim box per lane
        if (lane == 0) mbar_expect_tx(qfull, NH * kD * 2);
        __syncwarp();
        if (lane < kD / 64) tma_load_2d(smem + L::kOffQ + lane * 8192, &qmap, lane * 64, row * a.heads + hg * NH, qfull);
        __syncwarp();
        if (lane == 0) mbar_arrive(qfull);
    }
    int swbv = -1;
    if (ww >= 0 && gt < 8 && n_mine > 0) {
        const int lb = wlo / kBlockPositions + gt;
        if (row_ok && lb <= m / kBlockPositions && lb < a.swa_bt.max_blocks)
            swbv = __ldg(a.swa_bt.table + (long long)r * a.swa_bt.max_blocks + lb);
    }
    auto store_tables = [&]() {  // by the widening warps; a key then resolves with one global load at most
        if (bt_cached)
#pragma unroll
            for (int u = 0; u < kBtPer; ++u) {
                const int b = gt + u * kFp4WidenThreads;
                if (b < a.main_bt.max_blocks) s_bt[b] = btv[u];
            }
        if (gt < 8) s_swb[gt] = swbv;
        named_bar_sync(1, kFp4WidenThreads);
    };
    if constexpr (FUSED) {
        if (ww >= 0 && n_mine > 0) store_tables();
    }
    pdl_wait();  // global memory the preceding kernel writes, and every output, only below
    pdl_launch_dependents();
    if (!row_ok && tid == 0 && crank == 0) report(a.status, DSA_ERR_DEVICE_FAULT);
    int* s_topk = reinterpret_cast<int*>(smem + L::kOffTopk);
    if constexpr (FUSED) {
        // the row's top-k of the indexer scores on this cluster (one cluster of four CTAs per row), every selected
        // entry written into each CTA's s_topk (and topk_out); its scratch is the key stages, idle until then.  Its
        // first cluster barrier completes phase 0.
        cg::cluster_group cluster = cg::this_cluster();
        cluster_wait();
        auto& ts = *reinterpret_cast<TopkRowScratch<kClThreads, kFusedVpt, 4>*>(smem + L::kOffK);
        int32_t* tout = a.topk_out + (long long)row * a.k;
        auto emit = [&](int pos, int idx) {
#pragma unroll
            for (int c = 0; c < 4; ++c) *cluster.map_shared_rank(s_topk + pos, c) = idx;
            tout[pos] = idx;
        };
        const int nv_row = a.n_valid[row];  // the same in every CTA of the cluster
        if (nv_row < 0 || nv_row > a.score_ld) {
            if (tid == 0 && crank == 0) report(a.status, DSA_ERR_DEVICE_FAULT);
            for (int i = crank * kClThreads + tid; i < a.k; i += 4 * kClThreads) emit(i, -1);
        } else {
            topk_row_cluster<kClThreads, kFusedVpt, 4>(cluster, ts, a.scores + (long long)row * a.score_ld, nv_row,
                                                       a.k, emit, a.status, 23);
        }
        cluster.sync();  // every CTA's s_topk complete; the scratch (key stages) no longer read by a peer
    }
    bool ok = true;

    if (ww >= 0) {
        // ---- widening warps ----------------------------------------------------------------------------
        // decode rows (one query row per request): a gathered row serves this query row only and leaves L2 first
        const uint64_t policy = a.q_req ? l2_evict_normal() : l2_evict_first();
        // lane u < 8: key u of the warp's 8 in tile i.  Step 1: its top-k index (no dependent load).
        auto key_id = [&](int i, int* id) -> int {  // the key's index in the row, -1 if there is none
            *id = -1;
            if (lane >= kFp4PerWarp || i >= n_mine) return -1;
            const int j = (g_lo + crank + csize * i) * kFp4Keys + ww * kFp4PerWarp + lane;
            if (j < n_comp) *id = FUSED ? s_topk[j] : (a.topk ? __ldg(a.topk + (long long)row * a.k + j) : j);
            return j < n_keys ? j : -1;
        };
        // Step 2: index -> pool row (-1: none), and whether the pool is the window's.
        auto key_row = [&](int j, int id, bool* window) -> int {
            *window = j >= n_comp;
            if (j < 0) return -1;
            int pb, nb, at, epb;  // physical block, blocks of the pool, row within the block, rows of a block
            if (j < n_comp) {
                if (id < 0) return -1;
                epb = a.main.rows_per_block, nb = a.main.num_blocks;
                const int lb = id / epb;
                const bool in = id < n_vis && lb < a.main_bt.max_blocks && (!bt_cached || DSA_IDX_OK(lb, kBtCache, a.status));
                pb = !in ? -1 : bt_cached ? s_bt[lb] : __ldg(a.main_bt.table + (long long)r * a.main_bt.max_blocks + lb);
                at = id - lb * epb;
            } else {
                const int pos = wlo + (j - n_comp), lb = pos / kBlockPositions;
                const int sb = lb - wlo / kBlockPositions;  // the window (<= 1024 positions) spans <= 5 blocks
                epb = kBlockPositions, nb = a.swa.num_blocks;
                pb = DSA_IDX_OK(sb, 8, a.status) ? s_swb[sb] : -1;
                at = pos - lb * kBlockPositions;
            }
            if (pb < 0 || pb >= nb) {
                report(a.status, DSA_ERR_DEVICE_FAULT);
                *s_fault = 1;
                return -1;
            }
            return pb * epb + at;
        };
        const uint8_t* const main_lane = static_cast<const uint8_t*>(a.main.data) + lane * 8;
        const uint8_t* const swa_lane = static_cast<const uint8_t*>(a.swa.data) + lane * 8;
        uint2 code[2][kFp4PerWarp];
        uint32_t bsc[2][kFp4PerWarp];
        float ksc[2];         // lanes 0-7: the row scales
        uint32_t valid[2];    // the warp's 8 mask bits
        auto issue = [&](int b, int j, int id) {
            bool window;
            const int kr = key_row(j, id, &window);
            valid[b] = __ballot_sync(0xffffffffu, kr >= 0) & 0xffu;
            const uint32_t wm = __ballot_sync(0xffffffffu, window);
            ksc[b] = 0.f;
            if (kr >= 0) ksc[b] = (window ? a.swa.scale : a.main.scale)[kr];
#pragma unroll
            for (int u = 0; u < kFp4PerWarp; ++u) {
                const int v = __shfl_sync(0xffffffffu, kr, u);
                const uint8_t* p = ((wm >> u) & 1 ? swa_lane : main_lane) + (long long)max(v, 0) * kFp4BlockRow;
                code[b][u] = load_codes(p, v, policy);
                bsc[b][u] = load_block_scale(p + (kD / 2 - 7 * lane), v, policy);
            }
        };
        // Lane l holds block l (16 dims): 16-byte pieces 2 (l & 3), 2 (l & 3) + 1 of 64-dim chunk l >> 2.  Lanes of odd
        // chunks store their second piece first, so that eight neighbouring lanes cover all banks.
        const int hf = (lane >> 2) & 1, p0 = 2 * (lane & 3) + hf;
        const uint32_t dst0 = sK + (lane >> 2) * (kFp4Keys * 128) + ww * 1024;  // the warp's 8-row group
        auto widen = [&](int b, int i) {
            const int st = i & 1;
            if (i >= 2) ok = ok && mbar_wait_bounded(&pvdone[st], ((i >> 1) - 1) & 1, kWaitLimitNs);  // stage free
            if (gt == 0) DSA_TRACE(i, 0);
            if (ok) {
                if (lane < kFp4PerWarp) {
                    float* k = s_ksc + st * 2 * kFp4Keys + (ww * kFp4PerWarp + lane) / 2 * 4 + (lane & 1);
                    k[0] = ksc[b];
                    k[2] = ksc[b] * a.scale_log2;
                }
                if (lane == 0) s_mask8[st * 8 + ww] = (uint8_t)valid[b];
#pragma unroll
                for (int u = 0; u < kFp4PerWarp; ++u) {
                    const uint32_t s2 = block_scale_2p118(bsc[b][u]);
                    const uint32_t base = dst0 + st * kFp4Stage + u * 128;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t o[4];
                        widen8((h ^ hf) ? code[b][u].y : code[b][u].x, s2, o);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(base + (((p0 ^ h) ^ u) << 4)),
                                     "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                                     : "memory");
                    }
                }
            }
            fence_proxy_async_smem();  // the bf16 rows -> visible to the tensor core (async proxy)
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
            if (gt == 0) DSA_TRACE(i, 1);
        };
        if (n_mine > 0) {
            int id0, id1, id2;
            const int j0 = key_id(0, &id0), j1 = key_id(1, &id1);
            if constexpr (!FUSED) store_tables();
            issue(0, j0, id0);
            issue(1, j1, id1);
            int j2 = key_id(2, &id2);
            // two tiles a turn (register buffers 0 and 1); tiles past the end resolve to nothing and are not widened
#pragma unroll 1
            for (int i = 0; i < n_mine; i += 2) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (i + b < n_mine) {
                        widen(b, i + b);
                        issue(b, j2, id2);  // tile i + b + 2
                        j2 = key_id(i + b + 3, &id2);
                    }
                }
            }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) report(a.status, DSA_ERR_TIMEOUT);
    } else if (warp == 5) {
        // ---- O^T += V^T P^T, issued by one elected lane ------------------------------------------------------
        const uint32_t idesc_o = idesc_bf16(NH, 1, 128);
        uint32_t rescales = 0;
        for (int i = 0; i < n_mine; ++i) {
            const int b = i & 1;
            ok = mbar_wait_bounded(&pfull[b], (i >> 1) & 1, kWaitLimitNs);  // P^T written (so S done, the stage full)
            if (ok && (s_vote[b * 4] | s_vote[b * 4 + 1] | s_vote[b * 4 + 2] | s_vote[b * 4 + 3]))
                ok = mbar_wait_bounded(rdone, rescales++ & 1, kWaitLimitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            if (tid == 160) DSA_TRACE(i, 6);
            const uint64_t dv = sw128_desc(sK + b * kFp4Stage, kFp4Keys * 128, 1024);
            const uint64_t dp = sw128_desc(sP + b * L::kP, 16, 1024);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int ks = 0; ks < kFp4Keys / 16; ++ks)
                    mma_bf16_ss_elect(tO + mt * NH,
                                      dv + (uint64_t)(((2 * mt) * (kFp4Keys * 128) + (2 * ks) * 1024) >> 4),
                                      dp + (uint64_t)((ks * 32) >> 4), idesc_o, (i > 0 || ks > 0) ? 1u : 0u);
            mma_commit_elect(&pvdone[b]);
            if (tid == 160) DSA_TRACE(i, 7);
        }
        if (!ok && lane == 0) report(a.status, DSA_ERR_TIMEOUT);
    } else if (warp == 4) {
        // ---- S = Q K^T, issued by one elected lane -----------------------------------------------------------
        const uint32_t idesc_s = idesc_bf16(kFp4Keys, 0, 64);
        const uint64_t dq = sw128_desc(sQ, 16, 1024);
        if (n_mine > 0) ok = mbar_wait_bounded(qfull, 0, kWaitLimitNs);
        for (int i = 0; i < n_mine; ++i) {
            const int b = i & 1;
            if (i >= 2) ok = ok && mbar_wait_bounded(&pfull[b], ((i >> 1) - 1) & 1, kWaitLimitNs);  // S buffer read
            ok = ok && mbar_wait_bounded(&full[b], (i >> 1) & 1, kWaitLimitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            if (tid == 128) DSA_TRACE(i, 2);
            const uint64_t dk = sw128_desc(sK + b * kFp4Stage, 16, 1024);
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
                const uint64_t off = (uint64_t)((((ks >> 2) * (64 * 128)) + (ks & 3) * 32) >> 4);  // 64-row chunks, both
                mma_bf16_ss_elect(tS + b * kFp4Keys, dq + off, dk + off, idesc_s, ks > 0 ? 1u : 0u);
            }
            mma_commit_elect(&sfull[b]);
            if (tid == 128) DSA_TRACE(i, 3);
        }
        if (!ok && lane == 0) report(a.status, DSA_ERR_TIMEOUT);
    } else if (warp < 4) {
        // ---- softmax warps: heads 16 warp + lane / 4 and + 8, keys 8 i + 2 (lane % 4), + 1 ------------------
        const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
        const int hr = lane >> 2, c = lane & 3;
        // m_run: the head's running maximum, lazy: it moves only when exceeded by more than 2^8, so O^T is rarely
        // rescaled and exp2(s - m) <= 2^8.  l_run: the lane's share of the sum of the fp32 probabilities, two halves
        float m_run[2] = {-INFINITY, -INFINITY};
        uint64_t l_run[2] = {0ull, 0ull};
        // O^T times alpha per head, when a head's maximum moved in tile i: after the other warps' votes for the tile are
        // in (their P^T is written) and the product of tile i - 1 is done; the product of tile i waits for it
        auto rescale = [&](int i) {
            const int b = i & 1;
            ok = ok && mbar_wait_bounded(&pfull[b], (i >> 1) & 1, kWaitLimitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || !(s_vote[b * 4] | s_vote[b * 4 + 1] | s_vote[b * 4 + 2] | s_vote[b * 4 + 3])) return;
            ok = mbar_wait_bounded(&pvdone[b ^ 1], ((i - 1) >> 1) & 1, kWaitLimitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
                tc_fence_after();
#pragma unroll 1
                for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
                    for (int c0 = 0; c0 < NH; c0 += 16) {
                        float v[16];
                        tmem_ld16(tO + mt * NH + lane_off + c0, v);
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] *= s_alpha[b * NH + c0 + e];
                        tmem_st16(tO + mt * NH + lane_off + c0, v);
                    }
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(rdone);
        };
        for (int i = 0; i < n_mine; ++i) {
            const int b = i & 1;
            if (i > 0) rescale(i - 1);
            ok = ok && mbar_wait_bounded(&full[b], (i >> 1) & 1, kWaitLimitNs);  // the stage's scales and mask
            ok = ok && mbar_wait_bounded(&sfull[b], (i >> 1) & 1, kWaitLimitNs);
            if (i >= 2) ok = ok && mbar_wait_bounded(&pvdone[b], ((i >> 1) - 1) & 1, kWaitLimitNs);  // P^T buffer free
            ok = __all_sync(0xffffffffu, ok);
            if (tid == 0) DSA_TRACE(i, 4);
            float alpha[2] = {1.f, 1.f};
            bool resc = false;
            if (ok) {
                tc_fence_after();
                float sv[32];  // logits of head h in 4 e + 2 h, 4 e + 2 h + 1: keys 8 e + 2 c, + 1
                tmem_ld_16x64_nowait(tS + b * kFp4Keys + lane_off, sv);
                const float4* k4 = reinterpret_cast<const float4*>(s_ksc + b * 2 * kFp4Keys) + c;
                const uint64_t vm = *reinterpret_cast<const uint64_t*>(s_mask8 + b * 8);
                float m0[2];  // the logits are taken relative to m0: the running maximum, 0 before the first key
                uint64_t neg[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    m0[h] = m_run[h] == -INFINITY ? 0.f : m_run[h];
                    neg[h] = pack_f32x2(-m0[h], -m0[h]);
                }
                tmem_wait_ld();
                tmem_regs_after_wait<32>(sv);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 k = k4[4 * e];
                    const uint64_t kl = pack_f32x2(k.z, k.w);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        unpack_f32x2(fma_f32x2(pack_f32x2(sv[4 * e + 2 * h], sv[4 * e + 2 * h + 1]), kl, neg[h]),
                                     &sv[4 * e + 2 * h], &sv[4 * e + 2 * h + 1]);
                }
                if (vm != ~0ull) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t bits = (uint32_t)(vm >> (8 * e)) >> (2 * c);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!(bits & 1)) sv[4 * e + 2 * h] = -INFINITY;
                            if (!(bits & 2)) sv[4 * e + 2 * h + 1] = -INFINITY;
                        }
                    }
                }
                float mx[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mx[h] = fmaxf(sv[2 * h], sv[2 * h + 1]);
#pragma unroll
                    for (int e = 1; e < 8; ++e) mx[h] = fmaxf(mx[h], fmaxf(sv[4 * e + 2 * h], sv[4 * e + 2 * h + 1]));
                    mx[h] = quad_max(mx[h]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (mx[h] > (m_run[h] == -INFINITY ? -INFINITY : kLazyLog2)) {  // also the first finite maximum
                        const float m_new = m0[h] + mx[h];
                        alpha[h] = exp2f(m_run[h] - m_new);
                        resc = i > 0;
                        m_run[h] = m_new;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            sv[4 * e + 2 * h] -= mx[h];
                            sv[4 * e + 2 * h + 1] -= mx[h];
                        }
                    }
                }
                uint64_t sum[2] = {0ull, 0ull};
                const int head0 = warp * 16 + hr;
                const uint32_t prow = sP + b * L::kP + head0 * 128 + 4 * c;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 k = k4[4 * e];
                    const uint64_t ks = pack_f32x2(k.x, k.y);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint64_t p = pack_f32x2(ex2_sfu(sv[4 * e + 2 * h]), ex2_sfu(sv[4 * e + 2 * h + 1]));
                        sum[h] = add_f32x2(sum[h], p);
                        float p0, p1;  // the probability that multiplies the codes carries the row scale
                        unpack_f32x2(mul_f32x2(p, ks), &p0, &p1);
                        if (NH == 64 || head0 + 8 * h < NH)
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(prow + h * 1024 + ((e ^ (hr & 7)) << 4)),
                                         "r"(bf16x2_rn(p0, p1))
                                         : "memory");
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) l_run[h] = fma_f32x2(l_run[h], pack_f32x2(alpha[h], alpha[h]), sum[h]);
            }
            if (c == 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (NH == 64 || warp * 16 + hr + 8 * h < NH) s_alpha[b * NH + warp * 16 + hr + 8 * h] = alpha[h];
            }
            const bool any = __any_sync(0xffffffffu, resc);
            if (lane == 0) s_vote[b * 4 + warp] = any ? 1 : 0;
            fence_proxy_async_smem();  // P^T stores -> async proxy
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pfull[b]);
            if (tid == 0) DSA_TRACE(i, 5);
        }
        if (n_mine > 0) {  // the last product must be complete before O^T is read
            rescale(n_mine - 1);
            ok = ok && mbar_wait_bounded(&pvdone[(n_mine - 1) & 1], ((n_mine - 1) >> 1) & 1, kWaitLimitNs);
            tc_fence_after();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int head = warp * 16 + hr + 8 * h;
            float l0, l1;
            unpack_f32x2(l_run[h], &l0, &l1);
            const float l = quad_sum(l0 + l1);
            if (c == 0 && head < NH) {
                // a NaN among masked or absent maxima only: give the partial a weight, so that the NaN reaches the row
                s_own[head] = m_run[h] == -INFINITY && l != l ? 0.f : m_run[h];
                s_own[NH + head] = l;
                s_own[2 * NH + head] = l;
            }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) report(a.status, DSA_ERR_TIMEOUT);
    }

    attn_finish<NH, L, FUSED, kFp4Shift, true>(a, &omap, smem, tmem, tO, row, split, hg, crank, csize, n_mine, ok);
}

template <int NH, bool FUSED>
static dsa_status_t launch(AttnArgs a, int cl, cudaStream_t st) {
    using L = Fp4Smem<NH>;
    a.scale_log2 *= (float)(1 << kFp4Shift);
    CUtensorMap qmap, omap;
    if (!make_bf16_map(&qmap, a.q, (uint64_t)a.rows * a.heads, NH)) return DSA_ERR_CUDA;
    if (!make_out_map(&omap, a.out8 ? static_cast<void*>(a.out8) : static_cast<void*>(a.out), (uint64_t)a.rows * a.heads,
                      NH, a.out8 != nullptr))
        return DSA_ERR_CUDA;
    if (cudaFuncSetAttribute(attn_fp4_kernel<NH, FUSED>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc) !=
        cudaSuccess)
        return DSA_ERR_CUDA;
    const long long grid = (long long)a.rows * a.hg_count * a.nsplit * cl;
    if (grid > 0x7fffffffll) return DSA_ERR_UNSUPPORTED;
    cudaError_t e = launch_pdl_cluster(attn_fp4_kernel<NH, FUSED>, dim3((unsigned)grid), dim3(kClThreads), L::kAlloc, st,
                                       cl, qmap, omap, a);
    if (e == cudaSuccess && a.nsplit > 1) e = launch_attn_combine(a, st);
    if (e != cudaSuccess) return DSA_ERR_CUDA;
    return launch_status();
}

dsa_status_t launch_attn_fp4(const AttnArgs& a, int hg, int cl, bool fused, cudaStream_t st) {
    if (fused) return launch<64, true>(a, cl, st);
    switch (hg) {
        case 16: return launch<16, false>(a, cl, st);
        case 32: return launch<32, false>(a, cl, st);
        default: return launch<64, false>(a, cl, st);
    }
}

}  // namespace dsa

DSA_TIMELINE_SETTER(dsa_timeline_attention_fp4)
