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
// tile i of a CTA being the split's tile crank + CL i of 48 keys.  Inside a CTA, 16 warps:
//   warps 8-15  widen: each owns 6 keys of every tile.  Lanes 0-5 resolve the keys (top-k index -> block table -> row)
//               ahead; the rows' bytes are copied into shared memory with cp.async, each quarter of the warp's share
//               again as soon as it is converted, so a tile's copies have a whole tile's time; the codes become bf16
//               and are stored 128B-swizzled as [64-dim chunk][48 keys][128 B], the first 256 dims, then the others;
//   warps 4, 6  S = Q K^T (M = 64 heads, N = 48 keys) of even and odd tiles;
//   warp 5      O^T += V^T P^T (four tiles of M = 128 dims, N = NH heads, K = 48 keys);
//   warps 0-3   softmax: 16 heads a warp, a head's 48 logits over the 4 lanes of a quad (the 16-lane TMEM load spreads a
//               row over a quad, so every lane works although M = 64 fills 16 of the 32 TMEM lanes).
// The widened keys are a ring of five half-tiles (48 keys x 256 dims): S starts on the first half, P V frees it first.  Two
// S and two P buffers.  A tile passes through four hands (widen, S, softmax, P V), each hand-over costing 250 to 400
// cycles: with two stages of 64 keys that chain, and not any unit, set the pace.  The rows go through shared memory and
// not straight into registers: 227 KB of shared memory leave the L1 cache about 220 lines, which the rows of one tile fill,
// and further loads wait for lines when they are issued.
constexpr int kFp4Ring = 5;                            // half-tiles
constexpr int kFp4Half = kFp4Keys * (kD / 2) * 2;
constexpr int kFp4Chunk = kFp4Keys * 128;              // bytes of a 64-dim chunk
constexpr int kFp4Tiles = 3;                           // tiles whose scales and masks are kept
constexpr int kFp4Widen = 8;                           // widening warps, two on each of the SM's four schedulers
constexpr int kFp4PerWarp = kFp4Keys / kFp4Widen;      // keys of a tile per widening warp
constexpr int kFp4Pairs = kFp4PerWarp / 2;             // a warp converts two rows at a time
constexpr int kFp4Groups = kFp4Keys / 8;               // groups of 8 keys (the softmax's columns)
constexpr uint64_t kFp4AllValid = 0x3F3F3F3F3F3F3F3Full;  // a mask byte per widening warp, a bit per key
static_assert(kFp4PerWarp == 6, "six mask bits a warp");
// Widened values carry 2^-8: e2m1 bits placed in a bf16 are 2^-126 of the value, and the factor that undoes it times a
// block scale of up to 448 must stay below 2^128, so it is 2^118.
constexpr int kFp4Shift = 8;

// Bounded wait (2 s of %globaltimer).  The try suspends the warp in hardware for up to kSuspendNs at a time: measured,
// spinning on the default, short suspension, the waiting warps took a quarter of all issue slots from the softmax and the
// widening.
constexpr uint32_t kSuspendNs = 100000;
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity) {
    const uint32_t addr = smem_u32(bar);
    auto attempt = [&]() {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(addr), "r"(parity), "r"(kSuspendNs)
            : "memory");
        return done != 0;
    };
    if (attempt()) return true;
    const uint64_t t0 = global_ns();
    while (!attempt())
        if (global_ns() - t0 > kWaitLimitNs) return false;
    return true;
}

template <int NH>
struct Fp4Smem {
    static constexpr int kQ = 64 * kD * 2;                          // [8][64 rows][128 B]
    static constexpr int kP = NH * 128;                             // [NH rows][64 keys] bf16, keys 0 .. 47 used
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kQ;                        // ring of widened half-tiles; received tiles
    static constexpr int kOffP = kOffK + kFp4Ring * kFp4Half;       // two P^T buffers; output staging at the end
    static constexpr int kOffRaw = kOffP + 2 * kP;                  // [48 keys][288 B]: a tile's rows as stored
    static constexpr int kOffKsc = kOffRaw + kFp4Keys * kFp4BlockRow;  // float [3][24][4]: see s_ksc
    static constexpr int kOffMask = kOffKsc + kFp4Tiles * kFp4Keys * 8;  // uint8 [3][8]: valid keys of each widening warp
    static constexpr int kOffAlpha = kOffMask + 32;                 // float [2][NH]
    static constexpr int kOffVote = kOffAlpha + 2 * NH * 4;         // int [2][4]
    static constexpr int kOffFault = kOffVote + 32;                 // int: a key of this CTA hit a device fault
    static constexpr int kOffRope = kOffFault + 16;                 // float [32][2]: cos, sin of each pair's angle at m
    static constexpr int kBars = 2 * kFp4Ring + 10;
    static constexpr int kOffBar = kOffRope + 256;                  // kBars mbarriers, TMEM address
    static constexpr int kOffXfull = kOffBar + (kBars - 3) * 8;     // the last three: received tile slots
    static constexpr int kBytes = kOffBar + kBars * 8 + 16;
    static constexpr int kAlloc = kBytes;                           // the base is declared 1024-byte aligned
    static_assert(kAlloc <= 227 * 1024, "shared memory per CTA");
    static constexpr int kTile = 128 * NH * 2;                      // one exchanged 128-dim O tile: [NH / 4][128] x 4 bf16
    // after the last product: the other output staging buffers, m, l, e and the weights, in the idle ring
    static constexpr int kOffOut1 = kOffK + 49152;
    static constexpr int kOffOwn = kOffOut1 + 3 * NH * 256;         // float m[NH], l[NH], e[NH] of this CTA
    static constexpr int kOffFac = kOffOwn + 3 * NH * 4;            // float f[4 ranks][NH], 1/L, M, L, E [NH]
    static_assert(kOffFac + 8 * NH * 4 <= kOffP, "within the ring");
    static_assert(3 * kTile <= kQ, "the sent tiles fit in the query rows");
    static_assert(6 * kTile <= kQ + 49152, "the received tiles end before the second output buffer");
    static_assert(NH * 128 * 2 <= 2 * kP, "an output tile must fit in the P^T buffers");
    // (m, l, e, fault) of rank c's head h, written by that rank while this CTA may still be multiplying: the two 16-byte
    // pieces of a P^T row behind its 48 keys, which no product reads, in each of the two buffers
    static __host__ __device__ constexpr int stat(int c, int h) {
        return kOffP + (c >> 1) * kP + h * 128 + (((6 + (c & 1)) ^ (h & 7)) << 4);
    }
    static_assert(kOffKsc % 16 == 0 && kOffMask % 16 == 0 && kOffAlpha % 16 == 0 && kOffVote % 16 == 0 &&
                      kOffOwn % 16 == 0 && kOffFac % 16 == 0 && kOffFault % 16 == 0 && kOffRope % 16 == 0 &&
                      kOffBar % 16 == 0 && kOffOut1 % 1024 == 0,
                  "shared-memory regions 16-byte aligned");
    static constexpr int kTmemCols = 512;  // S: [2 buffers][64 columns, 48 used]; O^T: [4 tiles][NH heads]
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

// *p if `in`, else -1, in the register that will be used: a branch or a copy around the load would wait for it here, and an
// ordinary load the compiler moves down to its first use, a tile later.
__device__ __forceinline__ int load_int_if(const int32_t* p, bool in) {
    int v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, -1;\n\t@p ld.global.b32 %0, [%1];\n\t}"
        : "=&r"(v)
        : "l"(p), "r"((uint32_t)in)
        : "memory");
    return v;
}

__device__ __forceinline__ float load_float_if(const float* p, bool in) {  // 0 if not
    float v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t@p ld.global.f32 %0, [%1];\n\t}"
        : "=&f"(v)
        : "l"(p), "r"((uint32_t)in)
        : "memory");
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// 48 columns of a 16-lane accumulator (M = 64): lane 4 r + c of the warp gets, for row r and r + 8, columns
// 8 i + 2 c, 8 i + 2 c + 1 in registers 4 i, 4 i + 1 and 4 i + 2, 4 i + 3.  Valid after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld_16x48_nowait(uint32_t taddr, float (&v)[24]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23])
                 : "r"(taddr + 32)
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

template <int NH>
__global__ void __launch_bounds__(kClThreads, 1)
    attn_fp4_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap omap, AttnArgs a) {
    using L = Fp4Smem<NH>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sQ = smem_u32(smem + L::kOffQ), sK = smem_u32(smem + L::kOffK), sP = smem_u32(smem + L::kOffP);
    // the row scales of keys 2 p and 2 p + 1 of a stage, then the same times sm_scale log2(e)
    float* s_ksc = reinterpret_cast<float*>(smem + L::kOffKsc);
    uint8_t* s_mask8 = smem + L::kOffMask;
    float* s_alpha = reinterpret_cast<float*>(smem + L::kOffAlpha);
    int* s_vote = reinterpret_cast<int*>(smem + L::kOffVote);
    // half h of tile i: ring slot (2 i + h) % 5; scales and mask i % 3; S columns and P^T buffer i & 1
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);  // [5] widened (widening warps)
    uint64_t* pvdone = full + kFp4Ring;                                 // [5] multiplied into O^T
    uint64_t* sfull = pvdone + kFp4Ring;                                // [2] S in TMEM
    uint64_t* pfull = sfull + 2;                                        // [2] P^T written (4 softmax warps)
    uint64_t* qfull = pfull + 2;                                        // query rows loaded
    uint64_t* rdone = qfull + 1;                                        // O^T rescaled (4 softmax warps)
    uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + L::kOffXfull);  // [3] each received tile slot loaded
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(xfull + 3);
    volatile int* s_fault = reinterpret_cast<volatile int*>(smem + L::kOffFault);
    float* s_rc = reinterpret_cast<float*>(smem + L::kOffRope);
    float* s_own = reinterpret_cast<float*>(smem + L::kOffOwn);  // written after the last product

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int crank = (int)cluster_ctarank(), csize = (int)cluster_nctarank();
    const int cid = blockIdx.x / csize;
    const int split = cid % a.nsplit;
    const int hg = (cid / a.nsplit) % a.hg_count;
    const int row = cid / (a.nsplit * a.hg_count);
    if (tid == 0) {
        DSA_STAMP(0);
        for (int b = 0; b < kFp4Ring; ++b) {
            mbar_init(&full[b], kFp4Widen);
            mbar_init(&pvdone[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sfull[b], 1);
            mbar_init(&pfull[b], 4);
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
    if (tid == 0) DSA_STAMP(1);
    const uint32_t tS = tmem, tO = tmem + 128;
    if (csize > 1) cluster_arrive_relaxed();  // phase 0: this CTA has started (waited on before DSMEM use)

    // Position, request, block tables and query rows: inputs that no kernel of the layer step writes, read while the
    // preceding kernel finishes.  Top-k indices, cache rows and every output come after the wait.
    const int r = a.q_req ? a.q_req[row] : row;
    const int m = a.q_pos[row];
    const bool row_ok = r >= 0 && r < a.main_bt.batch && r < a.swa_bt.batch && m >= 0;
    if (!row_ok && tid == 0) *s_fault = 1;
    const int n_vis = row_ok ? entries_formed((long long)m + 1, a.kind_w, a.kind_s) : 0;
    const int n_comp = a.topk ? a.k : n_vis;
    const int wlo = max(0, m - a.window + 1);
    const int n_keys = row_ok ? n_comp + (m - wlo + 1) : 0;
    const int n_tiles = (n_keys + kFp4Keys - 1) / kFp4Keys;
    const int g_lo = split * a.cps, g_hi = min(n_tiles, g_lo + a.cps);
    const int n_mine = g_hi > g_lo + crank ? (g_hi - g_lo - crank + csize - 1) / csize : 0;
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
    pdl_wait();  // global memory the preceding kernel writes, and every output, only below
    pdl_launch_dependents();
    if (tid == 0) DSA_STAMP(2);
    if (!row_ok && tid == 0 && crank == 0) report(a.status, DSA_ERR_DEVICE_FAULT);
    bool ok = true;

    if (warp >= 8) {
        // ---- widening warps ----------------------------------------------------------------------------
        const int ww = warp - 8;
        // A key is resolved in three steps, a tile apart, so that no load waits for another: lanes 0-5, key `lane` of the
        // warp's 6 in tile i, j its index in the row (-1: none).  Step 1: its entry (top-k index; -1: none) or position.
        const int main_shift = __ffs(a.main.rows_per_block) - 1;  // 64 or 2 rows a block; the window's 256
        const int32_t* const row_topk = a.topk + (long long)row * a.k;
        auto key_index = [&](int i) -> int {
            const int j = (g_lo + crank + csize * i) * kFp4Keys + ww * kFp4PerWarp + lane;
            return lane < kFp4PerWarp && i < n_mine && j < n_keys ? j : -1;
        };
        auto key_entry = [&](int j) -> int { return load_int_if(row_topk + max(j, 0), a.topk && j >= 0 && j < n_comp); };
        auto key_id = [&](int j, int entry) -> int { return j >= n_comp ? wlo + (j - n_comp) : (a.topk ? entry : j); };
        // Step 2: the physical block, from the block table (-1: unmapped, beyond the table or not visible).
        auto key_block = [&](int j, int id) -> int {
            const bool window = j >= n_comp;
            const dsa_block_table_t& bt = window ? a.swa_bt : a.main_bt;
            const int lb = max(id, 0) >> (window ? 8 : main_shift);
            return load_int_if(bt.table + (long long)r * bt.max_blocks + lb,
                               j >= 0 && id >= 0 && (window || id < n_vis) && lb < bt.max_blocks);
        };
        // Step 3: the pool row (-1: none).
        auto key_row = [&](int j, int id, int block) -> int {
            if (j < 0 || id < 0) return -1;
            const bool window = j >= n_comp;
            if (block < 0 || block >= (window ? a.swa.num_blocks : a.main.num_blocks)) {
                report(a.status, DSA_ERR_DEVICE_FAULT);
                *s_fault = 1;
                return -1;
            }
            const int shift = window ? 8 : main_shift;
            return (block << shift) + (id & ((1 << shift) - 1));
        };
        // Converting, lane l = 16 q + t: of each pair of the warp's rows row q, and of each half of the dims block t (16 dims:
        // 16-byte pieces 2 (t & 3), 2 (t & 3) + 1 of 64-dim chunk t >> 2 of the half).  Lanes of odd chunks store their
        // second piece first, so that eight neighbouring lanes cover all banks.
        const int q = lane >> 4, t = lane & 15;
        const uint32_t raw = smem_u32(smem + L::kOffRaw) + ww * (kFp4PerWarp * kFp4BlockRow);
        const uint32_t raw_codes = raw + q * kFp4BlockRow + t * 8, raw_scale = raw + q * kFp4BlockRow + kD / 2 + t;
        const int hf = (t >> 2) & 1, p0 = 2 * (t & 3) + hf;
        uint32_t dst[kFp4Pairs][2];  // where the lane's pieces of its row of each pair go, within a ring slot
#pragma unroll
        for (int u = 0; u < kFp4Pairs; ++u)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int kk = ww * kFp4PerWarp + 2 * u + q;
                dst[u][g] = sK + (t >> 2) * kFp4Chunk + (kk >> 3) * 1024 + (kk & 7) * 128 + (((p0 ^ g) ^ (kk & 7)) << 4);
            }
        // Copying, lanes 0-17: of a pair's row lane / 9, 16-byte piece lane % 9 of a half (8 of codes, one of 16 scales).
        const int cr = lane >= 9 ? 1 : 0, cp = lane - 9 * cr;
        const uint32_t cp_off = cp < 8 ? cp * 16 : kD / 2, cp_step = cp < 8 ? kD / 4 : 16;  // half 0, and to half 1
        uint64_t src[kFp4Pairs];     // global address of the lane's piece (half 0) of the row of each pair
        uint32_t src_bytes[kFp4Pairs];  // 16, or 0 to fill with zeros (a masked key)
        // the rows of a tile, by the lanes that own them (kr: pool row or -1): their addresses to the copying lanes
        auto aim = [&](int kr, bool window) {
            const uint8_t* data = static_cast<const uint8_t*>(window ? a.swa.data : a.main.data);
            const uint64_t at = reinterpret_cast<uint64_t>(data) + (uint64_t)max(kr, 0) * kFp4BlockRow;
            const uint32_t valid = __ballot_sync(0xffffffffu, kr >= 0);
#pragma unroll
            for (int u = 0; u < kFp4Pairs; ++u) {
                src[u] = __shfl_sync(0xffffffffu, at, 2 * u + cr) + cp_off;
                src_bytes[u] = (valid >> (2 * u + cr)) & 1 ? 16u : 0u;
            }
            return valid;
        };
        auto copy = [&](int h, int u) {  // one group
            if (lane < 18)
                cp_async16_nc(raw + (2 * u + cr) * kFp4BlockRow + cp_off + h * cp_step,
                              reinterpret_cast<const void*>(src[u] + h * cp_step), src_bytes[u]);
            cp_async_commit();
        };
        if (n_mine > 0) {
            const int j0 = key_index(0), e0 = key_entry(j0), e1 = key_entry(key_index(1));
            int entry = key_entry(key_index(2));                       // of tile i + 2, loop-carried
            const int id0 = key_id(j0, e0), b0 = key_block(j0, id0);
            int id = key_id(key_index(1), e1), block = key_block(key_index(1), id);  // of tile i + 1
            int kr = key_row(j0, id0, b0);
            bool window = j0 >= n_comp;
            uint32_t valid = aim(kr, window);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int u = 0; u < kFp4Pairs; ++u) copy(h, u);
            float ksc = load_float_if((window ? a.swa.scale : a.main.scale) + max(kr, 0), kr >= 0);
            int slot = 0, kt = 0;
            uint32_t lap = 0;  // of the ring
#pragma unroll 1
            for (int i = 0; i < n_mine; ++i) {
                // tile i + 1's rows, whose copies follow each part of tile i that has been converted
                const int j1 = key_index(i + 1), j2 = key_index(i + 2);
                kr = key_row(j1, id, block);
                window = j1 >= n_comp;
                id = key_id(j2, entry);
                block = key_block(j2, id);
                entry = key_entry(key_index(i + 3));
                const uint32_t mask = valid;
                const float scale = ksc;
                valid = aim(kr, window);
                ksc = load_float_if((window ? a.swa.scale : a.main.scale) + max(kr, 0), kr >= 0);
                if (ww == 0 && lane == 0) DSA_TRACE(i, 0);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (lap > 0) ok = ok && wait_bar(&pvdone[slot], (lap - 1) & 1);
                    if (h == 0 && ok) {
                        if (lane < kFp4PerWarp) {
                            float* k = s_ksc + kt * 2 * kFp4Keys + (ww * kFp4PerWarp + lane) / 2 * 4 + (lane & 1);
                            k[0] = scale;
                            k[2] = scale * a.scale_log2;
                        }
                        if (lane == 0) s_mask8[kt * 8 + ww] = (uint8_t)mask;
                    }
#pragma unroll
                    for (int u = 0; u < kFp4Pairs; ++u) {
                        cp_async_wait_group<2 * kFp4Pairs - 1>();  // this part of tile i, six groups ago
                        __syncwarp();
                        const uint2 code = lds64(raw_codes + 2 * u * kFp4BlockRow + h * (kD / 4));
                        const uint32_t s2 = block_scale_2p118(lds8(raw_scale + 2 * u * kFp4BlockRow + h * 16));
                        __syncwarp();
                        copy(h, u);  // the same part of tile i + 1
                        if (ok) {
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                uint32_t o[4];
                                widen8((g ^ hf) ? code.y : code.x, s2, o);
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst[u][g] + slot * kFp4Half),
                                             "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                                             : "memory");
                            }
                        }
                    }
                    fence_proxy_async_smem();  // the bf16 rows -> visible to the tensor core (async proxy)
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[slot]);
                    if (++slot == kFp4Ring) slot = 0, ++lap;
                }
                if (++kt == kFp4Tiles) kt = 0;
                if (ww == 0 && lane == 0) DSA_TRACE(i, 1);
            }
            cp_async_wait_all();
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) report(a.status, DSA_ERR_TIMEOUT);
    } else if (warp == 5) {
        // ---- O^T += V^T P^T, issued by one elected lane ------------------------------------------------------
        const uint32_t idesc_o = idesc_bf16(NH, 1, 128);
        uint32_t rescales = 0;
        int slot = 0;
        for (int i = 0; i < n_mine; ++i) {
            const int b = i & 1;
            ok = wait_bar(&pfull[b], (i >> 1) & 1);  // P^T written (so S done, the stage full)
            if (ok && (s_vote[b * 4] | s_vote[b * 4 + 1] | s_vote[b * 4 + 2] | s_vote[b * 4 + 3]))
                ok = wait_bar(rdone, rescales++ & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) DSA_TRACE(i, 6);
            const uint64_t dp = sw128_desc(sP + b * L::kP, 16, 1024);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint64_t dv = sw128_desc(sK + slot * kFp4Half, kFp4Chunk, 1024);
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int ks = 0; ks < kFp4Keys / 16; ++ks)
                        mma_bf16_ss_elect(tO + (2 * h + mt) * NH,
                                          dv + (uint64_t)(((2 * mt) * kFp4Chunk + (2 * ks) * 1024) >> 4),
                                          dp + (uint64_t)((ks * 32) >> 4), idesc_o, (i > 0 || ks > 0) ? 1u : 0u);
                mma_commit_elect(&pvdone[slot]);
                if (++slot == kFp4Ring) slot = 0;
            }
            if (lane == 0) DSA_TRACE(i, 7);
        }
        if (!ok && lane == 0) report(a.status, DSA_ERR_TIMEOUT);
    } else if (warp == 4 || warp == 6) {
        // ---- S = Q K^T of every other tile, issued by one elected lane (one warp alone issues slower than the tensor
        // cores multiply) ------------------------------------------------------------------------------------
        const int b = warp == 6;
        const uint32_t idesc_s = idesc_bf16(kFp4Keys, 0, 64);
        const uint64_t dq = sw128_desc(sQ, 16, 1024);
        if (n_mine > b) ok = wait_bar(qfull, 0);
        for (int i = b; i < n_mine; i += 2) {
            if (i >= 2) ok = ok && wait_bar(&pfull[b], ((i >> 1) - 1) & 1);  // S buffer read
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = 2 * i + h, slot = n % kFp4Ring;
                ok = ok && wait_bar(&full[slot], (n / kFp4Ring) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (lane == 0 && h == 0) DSA_TRACE(i, 2);
                const uint64_t dk = sw128_desc(sK + slot * kFp4Half, 16, 1024);
#pragma unroll
                for (int ks = 0; ks < kD / 32; ++ks)
                    mma_bf16_ss_elect(tS + b * 64, dq + (uint64_t)(((((ks >> 2) + 4 * h) * 8192) + (ks & 3) * 32) >> 4),
                                      dk + (uint64_t)((((ks >> 2) * kFp4Chunk) + (ks & 3) * 32) >> 4), idesc_s,
                                      h + ks > 0 ? 1u : 0u);
            }
            if (!ok) break;
            mma_commit_elect(&sfull[b]);
            if (lane == 0) DSA_TRACE(i, 3);
        }
        if (!ok && lane == 0) report(a.status, DSA_ERR_TIMEOUT);
    } else if (warp < 4) {
        // ---- softmax warps: heads 16 warp + lane / 4 and + 8, keys 8 e + 2 (lane % 4), + 1 ------------------
        const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
        const int hr = lane >> 2, c = lane & 3;
        // m_run: the head's running maximum, lazy: it moves only when exceeded by more than 2^8, so O^T is rarely
        // rescaled and exp2(s - m) <= 2^8.  l_run: the lane's share of the sum of the fp32 probabilities, two halves
        float m_run[2] = {-INFINITY, -INFINITY};
        uint64_t l_run[2] = {0ull, 0ull};
        // O^T times alpha per head, when a head's maximum moved in tile i: after the other warps' votes for the tile are
        // in (their P^T is written) and the product of tile i - 1 is done; the product of tile i waits for it
        auto wait_pv = [&](int i) { return wait_bar(&pvdone[(2 * i + 1) % kFp4Ring], ((2 * i + 1) / kFp4Ring) & 1); };
        auto rescale = [&](int i) {
            const int b = i & 1;
            ok = ok && wait_bar(&pfull[b], (i >> 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || !(s_vote[b * 4] | s_vote[b * 4 + 1] | s_vote[b * 4 + 2] | s_vote[b * 4 + 3])) return;
            ok = wait_pv(i - 1);
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
            const int b = i & 1, kt = i % kFp4Tiles;
            if (i > 0) rescale(i - 1);
            ok = ok && wait_bar(&full[2 * i % kFp4Ring], (2 * i / kFp4Ring) & 1);  // the tile's scales and mask
            ok = ok && wait_bar(&sfull[b], (i >> 1) & 1);
            if (i >= 2) ok = ok && wait_pv(i - 2);  // P^T buffer free
            ok = __all_sync(0xffffffffu, ok);
            if (tid == 0) DSA_TRACE(i, 4);
            float alpha[2] = {1.f, 1.f};
            bool resc = false;
            if (ok) {
                tc_fence_after();
                float sv[24];  // logits of head h in 4 e + 2 h, 4 e + 2 h + 1: keys 8 e + 2 c, + 1
                tmem_ld_16x48_nowait(tS + b * 64 + lane_off, sv);
                const float4* k4 = reinterpret_cast<const float4*>(s_ksc + kt * 2 * kFp4Keys) + c;
                const uint64_t vm = *reinterpret_cast<const uint64_t*>(s_mask8 + kt * 8);
                float m0[2];  // the logits are taken relative to m0: the running maximum, 0 before the first key
                uint64_t neg[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    m0[h] = m_run[h] == -INFINITY ? 0.f : m_run[h];
                    neg[h] = pack_f32x2(-m0[h], -m0[h]);
                }
                tmem_wait_ld();
                tmem_regs_after_wait<24>(sv);
#pragma unroll
                for (int e = 0; e < kFp4Groups; ++e) {
                    const float4 k = k4[4 * e];
                    const uint64_t kl = pack_f32x2(k.z, k.w);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        unpack_f32x2(fma_f32x2(pack_f32x2(sv[4 * e + 2 * h], sv[4 * e + 2 * h + 1]), kl, neg[h]),
                                     &sv[4 * e + 2 * h], &sv[4 * e + 2 * h + 1]);
                }
                if (vm != kFp4AllValid) {
#pragma unroll
                    for (int e = 0; e < kFp4Groups; ++e) {
                        const int kk = 8 * e + 2 * c;  // and kk + 1: the same warp's, six keys being three pairs
                        const uint32_t bits = (uint32_t)(vm >> (kk / kFp4PerWarp * 8 + kk % kFp4PerWarp));
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
                    for (int e = 1; e < kFp4Groups; ++e) mx[h] = fmaxf(mx[h], fmaxf(sv[4 * e + 2 * h], sv[4 * e + 2 * h + 1]));
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
                        for (int e = 0; e < kFp4Groups; ++e) {
                            sv[4 * e + 2 * h] -= mx[h];
                            sv[4 * e + 2 * h + 1] -= mx[h];
                        }
                    }
                }
                uint64_t sum[2] = {0ull, 0ull};
                const int head0 = warp * 16 + hr;
                const uint32_t prow = sP + b * L::kP + head0 * 128 + 4 * c;
#pragma unroll
                for (int e = 0; e < kFp4Groups; ++e) {
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
            ok = ok && wait_pv(n_mine - 1);
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

    attn_finish<NH, L, false, kFp4Shift, true>(a, &omap, smem, tmem, tO, row, split, hg, crank, csize, n_mine, ok);
}

template <int NH>
static dsa_status_t launch(AttnArgs a, int cl, cudaStream_t st) {
    using L = Fp4Smem<NH>;
    a.scale_log2 *= (float)(1 << kFp4Shift);
    CUtensorMap qmap, omap;
    if (!make_bf16_map(&qmap, a.q, (uint64_t)a.rows * a.heads, NH)) return DSA_ERR_CUDA;
    if (!make_out_map(&omap, a.out8 ? static_cast<void*>(a.out8) : static_cast<void*>(a.out), (uint64_t)a.rows * a.heads,
                      NH, a.out8 != nullptr))
        return DSA_ERR_CUDA;
    if (cudaFuncSetAttribute(attn_fp4_kernel<NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc) !=
        cudaSuccess)
        return DSA_ERR_CUDA;
    const long long grid = (long long)a.rows * a.hg_count * a.nsplit * cl;
    if (grid > 0x7fffffffll) return DSA_ERR_UNSUPPORTED;
    cudaError_t e = launch_pdl_cluster(attn_fp4_kernel<NH>, dim3((unsigned)grid), dim3(kClThreads), L::kAlloc, st,
                                       cl, qmap, omap, a);
    if (e == cudaSuccess && a.nsplit > 1) e = launch_attn_combine(a, st);
    if (e != cudaSuccess) return DSA_ERR_CUDA;
    return launch_status();
}

dsa_status_t launch_attn_fp4(const AttnArgs& a, int hg, int cl, cudaStream_t st) {
    switch (hg) {
        case 16: return launch<16>(a, cl, st);
        case 32: return launch<32>(a, cl, st);
        default: return launch<64>(a, cl, st);
    }
}

}  // namespace dsa

DSA_TIMELINE_SETTER(dsa_timeline_attention_fp4)
