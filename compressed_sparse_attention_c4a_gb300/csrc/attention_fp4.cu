// dsa_sparse_attn_* over DSA_FP4_BLOCK rows: MQA attention over gathered 4-bit rows plus the sliding window, K = V,
// with the inverse-RoPE epilogue fused into the store.
//
// [P1] "DeepSeek DSA、DeepSeek V4与vLLM Hybrid KV Cache详解" §4.2-4.3, §5.3; [P2] "DeepSeek V4 稀疏注意力完全解剖" 机制一,
// 机制四, 深潜 (Inverse RoPE), 第三层 (a quantised decode cache): out = R_m^-1 sum_j p_j k_j, p = softmax(<q, k_j> sm),
// k_j = s_j bs_{j, d/16} c_{j, d} with e2m1 codes c, e4m3 block scales bs and a power-of-two row scale s.
//
// A code times its block scale has at most 6 significant bits, so the rows are widened to bf16 exactly and both products
// run on bf16 tensor cores; the row scale multiplies the key's logit and its probability (a power of two: no rounding).
// Rounded to fewer than 32 bits: a probability for P V (bf16, as the tensor core takes it; the normaliser sums the rounded
// ones, so a row's weights add up to one), a CTA's partial output when a cluster merges (attn_finish), and the output.
#include <algorithm>

#include "attention.cuh"

namespace dsa {

// Two kernels over the same warp roles.
//
// Few rows (attn_fp4_kernel<NH, false>): as the bf16 kernel (attention.cu), a cluster of CL CTAs per (query row, group of
// NH <= 64 heads, key split), tile i of a CTA being the split's tile crank + CL i of 48 keys, merged by attn_finish.
// Many rows (attn_fp4_kernel<NH, true>: a row in one CTA, no split): one CTA per SM takes units (row, head group) one after
// another, and everything runs on from one to the next: the next row's keys are resolved, copied and widened and its first
// logits computed before the last row's O^T has been stored.  (One CTA a row spent 22K of its 62K cycles, 640 keys, before
// the first tile and after the last.)
//
// The tiles of a CTA form one stream, described by a ring of six entries: the keys' addresses, scales and mask, and whether
// the tile is the first or last of its row or the last of all.
//   warp 7      resolves: two tiles at a time, three keys a lane (top-k index -> block table -> row address, row scale).  The
//               -1 that a top-k row ends in are cut off (many rows), and a tile without a key is left out: 1153 prefill
//               rows with lists of 333, mostly padding, 16 heads, 130 us with all tiles, 91 without empty ones, 66 so;
//   warps 8-15  widen: each owns 6 keys of every tile.  The rows' bytes are copied into shared memory with cp.async, the next
//               tile's as soon as this one's have been read into registers; the codes become bf16 and are stored
//               128B-swizzled as [64-dim chunk][48 keys][128 B], the first 256 dims, then the others.  Many rows: between
//               two tiles, when a row's last product is done, these warps read its O^T from TMEM, rotate and store it;
//   warps 4, 6  S = Q K^T (M = 64 heads, N = 48 keys) of even and odd tiles;
//   warp 5      O^T += V^T P^T (four tiles of M = 128 dims, N = NH heads, K = 48 keys);
//   warps 0-3   softmax: 16 heads a warp, a head's 48 logits over the 4 lanes of a quad (the 16-lane TMEM load spreads a
//               row over a quad, so every lane works although M = 64 fills 16 of the 32 TMEM lanes).
// The widened keys are a ring of five half-tiles (48 keys x 256 dims): S starts on the first half, P V frees it first.  Two
// S and two P buffers.
//
// What bounds it (2048 rows of 640 keys, 64 heads: 327 us, a tile in about 2,800 cycles): shared memory is busy for 2,120
// of them by its bytes alone (reads of S 896 and of P V 576, widened stores 384, P^T 48, the rows' copies and loads 216),
// and a row's O^T is read out while its successor's products wait, about 5,000 cycles a row.  What else was measured on the
// way, in us, each against the kernel of its time: one CTA a row 463 against 394; rows loaded straight into registers 446
// (227 KB of shared memory leave the L1 cache about 220 lines, which the rows of one tile fill, and further loads wait for
// lines when they are issued); loops unrolled and waits inline with 64-bit times 578 (the roles share the instruction
// caches); matrix instructions with descriptors computed in ordinary registers 390 against 361 (77 cycles to issue one, 35
// with uniform ones); the rows fetched by a warp of its own, with bulk copies 509 (100 cycles a row), with cp.async 397;
// tiles of 32 keys 416; a finished row stored as soon as its product is done, at any half-tile, 375 against 361; the copies
// in halves, each when its half has been converted, 334 against 325; twelve widening warps of 4 keys 325 against 317.
// A decode row's 31,000 cycles (32 rows of 640 keys, clusters of 4: 16.3 us): 7,000 until the first tile is widened (position,
// block table, rows, one load after the other), 13,000 for four tiles (widening, S, softmax, P V, one after the other), 11,000
// for the merge across the cluster.  The same rows in bf16, which need no widening, take 14.0 us, one row of 16 heads 11.0
// against 11.8; 16 rows of 8,320 keys 52.7 against 51.4, the prefill above 405 against 328.
constexpr int kFp4Ring = 5;                            // widened half-tiles
constexpr int kFp4Half = kFp4Keys * (kD / 2) * 2;
constexpr int kFp4Chunk = kFp4Keys * 128;              // bytes of a 64-dim chunk
constexpr int kFp4Entries = 6;                         // described tiles
constexpr int kFp4Widen = 8;                           // widening warps, two on each of the SM's four schedulers
constexpr int kFp4PerWarp = kFp4Keys / kFp4Widen;      // keys of a tile per widening warp
constexpr int kFp4Pairs = kFp4PerWarp / 2;             // a warp converts two rows at a time
static_assert(kFp4Widen * kFp4PerWarp == kFp4Keys && kFp4Pairs * 2 == kFp4PerWarp && 256 + 32 * kFp4Widen == kClThreads, "roles");
constexpr int kFp4Groups = kFp4Keys / 8;               // groups of 8 keys (the softmax's columns)
constexpr uint64_t kFp4AllValid = (1ull << kFp4Keys) - 1;
constexpr uint64_t kFp4Fault = 1ull << 63;             // mask bit: a key of the tile hit a device fault
// what an entry says of its tile
constexpr int kFirst = 1, kLast = 2, kFinal = 4;  // of its row; of the stream
constexpr int kOdd = 8, kOdd2 = 16;               // the two lowest bits of the row's ordinal
// Widened values carry 2^-8: e2m1 bits placed in a bf16 are 2^-126 of the value, and the factor that undoes it times a
// block scale of up to 448 must stay below 2^128, so it is 2^118.
constexpr int kFp4Shift = 8;

// Bounded wait (2 s of %globaltimer, its low word).  Inline, but a few instructions: the kernel's roles run side by side and
// share the instruction caches (with 64-bit times, every tile loop unrolled and the rare paths inline the schedulers mostly
// waited for instructions, 3.9 cycles of it per issued instruction).  A call out of line here makes every value that is
// live across a wait take a register that calls preserve: 357 us for the prefill below against 334.
__device__ __forceinline__ uint32_t global_ns_lo() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint32_t t0 = global_ns_lo();
#pragma unroll 1
    do {
        if (mbar_try_wait(bar, parity)) return true;
    } while (global_ns_lo() - t0 <= (uint32_t)kWaitLimitNs);
    return false;
}
static_assert(kWaitLimitNs < 0x80000000ull, "within the low word");

template <int NH>
struct Fp4Smem {
    static constexpr int kQ = 64 * kD * 2;                          // [8][64 rows][128 B]
    static constexpr int kP = NH * 128;                             // [NH rows][64 keys] bf16, keys 0 .. 47 used
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kQ;                        // ring of widened half-tiles; received tiles
    static constexpr int kOffP = kOffK + kFp4Ring * kFp4Half;       // two P^T buffers; output staging at the end
    static constexpr int kOffRaw = kOffP + 2 * kP;                  // [48 keys][288 B]: a tile's rows as stored
    static constexpr int kOffAddr = kOffRaw + kFp4Keys * kFp4BlockRow;  // uint64 [6][48]: address of a key's row, 0 masked
    static constexpr int kOffKsc = kOffAddr + kFp4Entries * kFp4Keys * 8;  // float [6][24][4]: see s_ksc
    static constexpr int kOffMask = kOffKsc + kFp4Entries * kFp4Keys * 8;  // uint64 [6]: valid keys, kFp4Fault
    static constexpr int kOffInfo = kOffMask + kFp4Entries * 8;     // int [6][4]: flags, unit, position
    static constexpr int kOffAlpha = kOffInfo + kFp4Entries * 16;   // float [2][NH]
    static constexpr int kOffVote = kOffAlpha + 2 * NH * 4;         // int [2][4]: a softmax warp's vote for a rescale
    static constexpr int kOffPinfo = kOffVote + 32;                 // int [2]: flags of the tile in a P^T buffer
    static constexpr int kOffInv = kOffPinfo + 16;                  // float [2][NH]: output factor of a finished row
    static constexpr int kOffRow = kOffInv + 2 * NH * 4;            // int [2][4]: its unit, -, position, fault
    // int: a key of this CTA hit a device fault; many rows: the fewest rows that a widening warp whose waits ran out has stored
    static constexpr int kOffFault = kOffRow + 32;
    static constexpr int kOffRope = kOffFault + 16;                 // float [32][2]: cos, sin of each pair's angle at m
    static constexpr int kBars = 2 * kFp4Ring + 3 * kFp4Entries + 13;
    static constexpr int kOffBar = kOffRope + 256;                  // kBars mbarriers, TMEM address
    static constexpr int kOffXfull = kOffBar + (kBars - 4) * 8;     // three of the last four: received tile slots
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
    static_assert(kOffRaw % 16 == 0 && kOffAddr % 16 == 0 && kOffKsc % 16 == 0 && kOffMask % 16 == 0 &&
                      kOffInfo % 16 == 0 && kOffAlpha % 16 == 0 && kOffVote % 16 == 0 && kOffInv % 16 == 0 &&
                      kOffRow % 16 == 0 && kOffOwn % 16 == 0 && kOffFac % 16 == 0 && kOffFault % 16 == 0 &&
                      kOffRope % 16 == 0 && kOffBar % 16 == 0 && kOffOut1 % 1024 == 0,
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

// A descriptor like d with this low word (address, leading offset): the sum of a descriptor and an offset within shared
// memory carries nothing into the high word.
__device__ __forceinline__ uint64_t desc_lo(uint64_t d, uint32_t lo) { return (d & 0xffffffff00000000ull) | lo; }

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

// The two bf16 values of a word added to two fp32 sums, without widening them first (widened by shifts 328 us for the prefill
// below, 327 so; by a warp-level product with a matrix of ones 341).
__device__ __forceinline__ void add_bf16x2(uint32_t w, float (&s)[2]) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
        : "+f"(s[0]), "+f"(s[1])
        : "r"(w));
}

// O^T of the calling warp's quadrant times alpha per head (a rare step, kept out of the loops).
template <int NH>
__device__ __noinline__ void rescale_quadrant(uint32_t taddr, const float* alpha) {
#pragma unroll 1
    for (int c0 = 0; c0 < 4 * NH; c0 += 16) {
        float v[16];
        tmem_ld16(taddr + c0, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] *= alpha[c0 % NH + e];
        tmem_st16(taddr + c0, v);
    }
    tmem_wait_st();
}

// A finished row's output, by the widening warps (ww): O^T from TMEM, times the row's factor per head, rotated
// by R_m^-1, to global memory.  Warp quadrant = 32 dims of each 128-dim tile, lane = dim, half of the heads; a store of a
// warp is 64 bytes of one head's row.  (Neighbouring lanes exchanging values to store words of two dims: 361 us for the
// prefill below, 355 so.)
template <int NH>
__device__ __noinline__ void store_row(const RopeTable& rope, uint16_t* out_row, uint32_t taddr, const float* inv, int ww,
                                       int m, bool fault, uint64_t* ofree) {
    constexpr int kHeads = NH / 2, kStep = kHeads < 16 ? kHeads : 16, kSteps = kHeads / kStep;
    const int lane = threadIdx.x & 31, quad = ww & 3, hbase = (ww >> 2) * kHeads;
    const int first_rot = kD - rope.rope_dim;
    taddr += ((uint32_t)(quad * 32) << 16) + hbase;
    inv += hbase;
    float v[kStep];
    tmem_ld_nowait<kStep>(taddr, v);
#pragma unroll 1
    for (int n = 0; n < 4 * kSteps; ++n) {  // 128-dim tile n / kSteps, kStep heads
        const int tt = n / kSteps, h0 = n % kSteps * kStep;
        const int dim = tt * 128 + quad * 32 + (lane & ~1);  // the pair's even dim
        float x[kStep];
        tmem_wait_ld();
        tmem_regs_after_wait<kStep>(v);
#pragma unroll
        for (int e = 0; e < kStep; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(inv + h0 + e);
            x[e] = v[e] * f.x, x[e + 1] = v[e + 1] * f.y, x[e + 2] = v[e + 2] * f.z, x[e + 3] = v[e + 3] * f.w;
        }
        if (n + 1 < 4 * kSteps) {
            tmem_ld_nowait<kStep>(taddr + (n + 1) / kSteps * NH + (n + 1) % kSteps * kStep, v);
        } else {  // all read: the next row's products may begin
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ofree);
        }
        if (fault) {
#pragma unroll
            for (int e = 0; e < kStep; ++e) x[e] = 0.f;
        }
        uint16_t* const to = out_row + (hbase + h0) * kD + tt * 128 + quad * 32 + lane;
        if (!__any_sync(0xffffffffu, dim >= first_rot)) {
#pragma unroll
            for (int e = 0; e < kStep; e += 2) {
                const uint32_t w = bf16x2_rn(x[e], x[e + 1]);
                to[e * kD] = (uint16_t)w;
                to[(e + 1) * kD] = (uint16_t)(w >> 16);
            }
        } else {
            float cs = 1.f, sn = 0.f;
            if (dim >= first_rot && !fault) rope_cos_sin(m, rope, (dim - first_rot) >> 1, &cs, &sn);
            if (lane & 1) sn = -sn;
#pragma unroll
            for (int e = 0; e < kStep; e += 2) {
                const float y0 = __shfl_xor_sync(0xffffffffu, x[e], 1), y1 = __shfl_xor_sync(0xffffffffu, x[e + 1], 1);
                const uint32_t w = bf16x2_rn(x[e] * cs + y0 * sn, x[e + 1] * cs + y1 * sn);
                to[e * kD] = (uint16_t)w;
                to[(e + 1) * kD] = (uint16_t)(w >> 16);
            }
        }
    }
}

// Zeros for the rows of a CTA from its row number `done` on, lse -inf (a wait ran out).
template <int NH>
__device__ __noinline__ void zero_rows(const AttnArgs& a, int unit0, int unit_step, int units, int done) {
    for (long long unit = unit0 + (long long)done * unit_step; unit < units; unit += unit_step) {
        const long long first = unit * NH;  // a row's head groups follow one another
        for (int i = threadIdx.x; i < NH * kD / 8; i += kClThreads)
            reinterpret_cast<uint4*>(a.out + first * kD)[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int h = threadIdx.x; h < NH; h += kClThreads) a.lse[first + h] = -INFINITY;
    }
}

// The unit (query row, head group) that a CTA works on and its share of the row's tiles.
struct Unit {
    int row, hg, r, m;
    int n_vis, n_comp, wlo, n_keys;
    int first, step, end, tiles;  // the CTA's tile i is the row's tile first + step i < end; tiles >= 1 (if there is none,
                                  // one of masked keys)
    bool ok;
};

template <int NH, bool ROWS>
__global__ void __launch_bounds__(kClThreads, 1)
    attn_fp4_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap omap,
                    const __grid_constant__ AttnArgs a) {
    using L = Fp4Smem<NH>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sQ = smem_u32(smem + L::kOffQ), sK = smem_u32(smem + L::kOffK), sP = smem_u32(smem + L::kOffP);
    uint64_t* s_addr = reinterpret_cast<uint64_t*>(smem + L::kOffAddr);
    // the row scales of keys 2 p and 2 p + 1 of a tile, then the same times sm_scale log2(e)
    float* s_ksc = reinterpret_cast<float*>(smem + L::kOffKsc);
    uint64_t* s_mask = reinterpret_cast<uint64_t*>(smem + L::kOffMask);
    int* s_info = reinterpret_cast<int*>(smem + L::kOffInfo);
    float* s_alpha = reinterpret_cast<float*>(smem + L::kOffAlpha);
    int* s_vote = reinterpret_cast<int*>(smem + L::kOffVote);
    int* s_pinfo = reinterpret_cast<int*>(smem + L::kOffPinfo);
    float* s_inv = reinterpret_cast<float*>(smem + L::kOffInv);
    int* s_orow = reinterpret_cast<int*>(smem + L::kOffRow);
    // tile g: entry g % 6; half h in ring slot (2 g + h) % 5; S columns and P^T buffer g & 1
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);  // [5] half-tile widened (widening warps)
    uint64_t* pvdone = full + kFp4Ring;                                 // [5] multiplied into O^T
    uint64_t* rfull = pvdone + kFp4Ring;                                // [6] entry: addresses, mask, flags
    uint64_t* kfull = rfull + kFp4Entries;                              // [6] entry: scales
    uint64_t* kfree = kfull + kFp4Entries;                              // [6] entry read (softmax warps, next S warp)
    uint64_t* sfull = kfree + kFp4Entries;                              // [2] S in TMEM
    uint64_t* pfull = sfull + 2;                                        // [2] P^T written (4 softmax warps)
    // [2] query rows loaded, by the parity of the row's ordinal: an S warp sees every second tile only, and with one barrier
    // it could wait for row r + 1 by parity before row r's load is complete
    uint64_t* qfull = pfull + 2;
    uint64_t* rdone = qfull + 2;                                        // O^T rescaled (4 softmax warps)
    uint64_t* ostat = rdone + 1;                                        // a row's factors written (4 softmax warps)
    uint64_t* ofree = ostat + 1;                                        // its O^T read (widening warps)
    uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + L::kOffXfull);  // [3] each received tile slot loaded
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(xfull + 4);
    volatile int* s_fault = reinterpret_cast<volatile int*>(smem + L::kOffFault);
    float* s_rc = reinterpret_cast<float*>(smem + L::kOffRope);
    float* s_own = reinterpret_cast<float*>(smem + L::kOffOwn);  // written after the last product

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in all lanes
    const int crank = ROWS ? 0 : (int)cluster_ctarank(), csize = ROWS ? 1 : (int)cluster_nctarank();
    const int cid = blockIdx.x / csize;
    const int split = ROWS ? 0 : cid % a.nsplit;
    // units: ROWS: blockIdx.x, + gridDim.x, ... of rows * head groups; else the one of this cluster
    const int unit0 = ROWS ? (int)blockIdx.x : cid / a.nsplit, units = a.rows * a.hg_count;
    const int unit_step = ROWS ? (int)gridDim.x : units;
    if (tid == 0) {
        DSA_STAMP(0);
        for (int b = 0; b < kFp4Ring; ++b) {
            mbar_init(&full[b], kFp4Widen);
            mbar_init(&pvdone[b], 1);
        }
        for (int b = 0; b < kFp4Entries; ++b) {
            mbar_init(&rfull[b], 1);
            mbar_init(&kfull[b], 1);
            mbar_init(&kfree[b], 5);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sfull[b], 1);
            mbar_init(&pfull[b], 4);
        }
        mbar_init(&qfull[0], 1);
        mbar_init(&qfull[1], 1);
        mbar_init(rdone, 4);
        mbar_init(ostat, 4);
        mbar_init(ofree, kFp4Widen);
        for (int b = 0; b < 3; ++b) mbar_init(&xfull[b], 1);
        *s_fault = ROWS ? 0x7fffffff : 0;
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
    // all 512 columns are this CTA's, so its base is column 0
    constexpr uint32_t tmem = 0, tS = 0, tO = 128;
    if constexpr (!ROWS)
        if (csize > 1) cluster_arrive_relaxed();  // phase 0: this CTA has started (waited on before DSMEM use)

    // Position, request, block tables and query rows: inputs that no kernel of the layer step writes, read while the
    // preceding kernel finishes.  Top-k indices, cache rows and every output come after the wait.
    auto row_of = [&](int unit) { return unit >> (a.hg_count - 1); };  // one head group a row, or two
    auto make_unit = [&](int unit, int r, int m, int listed) {  // listed: top-k entries to look at
        Unit u;
        u.row = row_of(unit);
        u.hg = unit - u.row * a.hg_count;
        u.r = r;
        u.m = m;
        u.ok = r >= 0 && r < a.main_bt.batch && r < a.swa_bt.batch && m >= 0;
        const uint32_t tokens = (uint32_t)m + 1u;  // entries_formed() by a shift: the stride is a power of two
        u.n_vis = u.ok && tokens >= (uint32_t)a.kind_w ? (int)((tokens - a.kind_w) >> (__ffs(a.kind_s) - 1)) + 1 : 0;
        u.n_comp = a.topk ? listed : u.n_vis;
        u.wlo = max(0, m - a.window + 1);
        u.n_keys = u.ok ? u.n_comp + (m - u.wlo + 1) : 0;
        const int n_tiles = (u.n_keys + kFp4Keys - 1) / kFp4Keys;
        u.first = split * a.cps + crank;
        u.step = csize;
        // never more tiles than planned: without a top-k list the position alone sets n_keys, and one beyond the block table
        // (2^31 - 1: 11 million tiles) has its first unmapped key, a device fault, among the planned tiles
        u.end = min(n_tiles, (split + 1) * a.cps);
        u.tiles = u.end > u.first ? (u.end - u.first + csize - 1) >> (__ffs(csize) - 1) : 1;
        return u;
    };
    auto load_q = [&](int unit, int odd) {  // by one warp: one 64-dim box per lane
        const int row = row_of(unit);
        const int never = row == a.stall_row && crank == csize - 1 ? 16 : 0;  // test hook: bytes that no copy brings
        if (lane == 0) mbar_expect_tx(&qfull[odd], NH * kD * 2 + never);
        __syncwarp();
        if (lane < kD / 64)
            tma_load_2d(smem + L::kOffQ + lane * 8192, &qmap, lane * 64, row * a.heads + (unit - row * a.hg_count) * NH,
                        &qfull[odd]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&qfull[odd]);
    };
    if (warp == 4) load_q(unit0, 0);
    int r0 = 0, m0 = 0;
    if (warp == 7 || warp == 3) {
        r0 = a.q_req ? a.q_req[row_of(unit0)] : row_of(unit0);
        m0 = a.q_pos[row_of(unit0)];
    }
    if constexpr (!ROWS)
        if (warp == 3 && lane < a.rope.rope_dim / 2) {  // R_m^-1 of the output: cos and sin of each pair's angle at m
            float c = 1.f, sn = 0.f;
            if (m0 >= 0) rope_cos_sin(m0, a.rope, lane, &c, &sn);
            s_rc[2 * lane] = c;
            s_rc[2 * lane + 1] = sn;
        }
    pdl_wait();  // global memory the preceding kernel writes, and every output, only below
    pdl_launch_dependents();
    if (tid == 0) DSA_STAMP(2);
    bool ok = true;
    auto entry_wait = [&](uint64_t* bars, int g) { return wait_bar(&bars[g % kFp4Entries], (g / kFp4Entries) & 1); };

    if (warp == 7) {
        // ---- resolve: every unit's tiles, two at a time: key kk = lane + 32 e of the two tiles' 96 ---------------
        const int main_shift = __ffs(a.main.rows_per_block) - 1;  // 64 or 2 rows a block; the window's 256
        int g = 0;
        int tail = ROWS ? load_int_if(a.topk + (long long)row_of(unit0) * a.k + a.k - 1, a.topk != nullptr) : 0;
        for (int unit = unit0, ord = 0; unit < units && ok; unit += unit_step, ++ord) {
            const int32_t* const row_topk = a.topk + (long long)row_of(unit) * a.k;
            int entry[3];  // top-k indices of the next two tiles' keys (-1: none); the first ones before the position is here
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                const int kk = lane + 32 * e, t = (ROWS ? 0 : split * a.cps) + crank + (kk < kFp4Keys ? 0 : csize);
                const int j = t * kFp4Keys + kk % kFp4Keys;
                entry[e] = load_int_if(row_topk + j, a.topk && j < a.k && DSA_IDX_OK(j, a.k, a.status));
            }
            int listed = a.k;
            if (ROWS && a.topk && tail < 0) {  // the list without the -1 it ends in, looked through from its end
                for (listed = a.k - 1; listed > 0;) {
                    int v[8], top = -1;
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const int j = listed - 1 - (32 * n + lane);
                        v[n] = load_int_if(row_topk + max(j, 0), j >= 0);
                    }
#pragma unroll
                    for (int n = 0; n < 8; ++n) top = max(top, v[n] >= 0 ? listed - 1 - (32 * n + lane) : -1);
                    top = __reduce_max_sync(0xffffffffu, top);
                    listed = top >= 0 ? top + 1 : max(listed - 256, 0);
                    if (top >= 0) break;
                }
            }
            const Unit u = make_unit(unit, r0, m0, listed);
            if (unit + unit_step < units) {  // the next unit's, in flight meanwhile
                const int next = row_of(unit + unit_step);
                r0 = a.q_req ? load_int_if(a.q_req + next, true) : next;
                m0 = load_int_if(a.q_pos + next, true);
                tail = ROWS ? load_int_if(a.topk + (long long)next * a.k + a.k - 1, a.topk != nullptr) : 0;
            }
            if (!u.ok && lane == 0 && crank == 0) report(a.status, DSA_ERR_DEVICE_FAULT);
            auto key_index = [&](int i, int e) -> int {  // of the row, -1: none
                const int kk = lane + 32 * e, t = i + kk / kFp4Keys;
                const int tile = u.first + u.step * t, j = tile * kFp4Keys + kk % kFp4Keys;
                return tile < u.end && j < u.n_keys ? j : -1;
            };
            bool first = true;
            for (int i = 0; i < u.tiles && ok; i += 2) {
                const bool two = i + 1 < u.tiles;
                if (g >= kFp4Entries) ok = entry_wait(kfree, g - kFp4Entries);
                if (two && g + 1 >= kFp4Entries) ok = ok && entry_wait(kfree, g + 1 - kFp4Entries);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                int j[3], id[3], block[3], row[3];
                uint64_t addr[3];
                uint32_t valid[3], bad = !u.ok;
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    j[e] = key_index(i, e);
                    const bool window = j[e] >= u.n_comp;
                    id[e] = j[e] < 0 ? -1 : window ? u.wlo + (j[e] - u.n_comp) : (a.topk ? entry[e] : j[e]);
                    const dsa_block_table_t& bt = window ? a.swa_bt : a.main_bt;
                    const int lb = max(id[e], 0) >> (window ? 8 : main_shift);
                    block[e] = load_int_if(bt.table + (long long)u.r * bt.max_blocks + lb,
                                           id[e] >= 0 && (window || id[e] < u.n_vis) && lb < bt.max_blocks &&
                                               DSA_IDX_OK((long long)u.r * bt.max_blocks + lb,
                                                          (long long)bt.batch * bt.max_blocks, a.status));
                }
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    const int jn = key_index(i + 2, e);
                    entry[e] = load_int_if(row_topk + max(jn, 0), a.topk && jn >= 0 && jn < u.n_comp && DSA_IDX_OK(jn, a.k, a.status));
                }
                float scale[3];
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    const bool window = j[e] >= u.n_comp;
                    const dsa_pool_t& pool = window ? a.swa : a.main;
                    row[e] = -1;
                    if (id[e] >= 0) {
                        if (block[e] < 0 || block[e] >= pool.num_blocks) bad |= 2u;
                        else row[e] = (block[e] << (window ? 8 : main_shift)) + (id[e] & (window ? 255 : (1 << main_shift) - 1));
                        if (row[e] >= 0 && !DSA_IDX_OK(row[e], (long long)pool.num_blocks * pool.rows_per_block, a.status))
                            row[e] = -1;
                    }
                    scale[e] = load_float_if(pool.scale + max(row[e], 0), row[e] >= 0);
                    valid[e] = __ballot_sync(0xffffffffu, row[e] >= 0);
                    addr[e] = row[e] < 0 ? 0ull : reinterpret_cast<uint64_t>(pool.data) + (uint64_t)row[e] * kFp4BlockRow;
                }
                bad = __any_sync(0xffffffffu, bad != 0);
                if (bad && u.ok && lane == 0) report(a.status, DSA_ERR_DEVICE_FAULT);
                // a tile without a key is left out (the padding of a short top-k row), unless it is the last
                const uint64_t mask0 = (uint64_t)valid[0] | (uint64_t)(valid[1] & 0xffffu) << 32;
                const uint64_t mask1 = (uint64_t)(valid[1] >> 16) | (uint64_t)valid[2] << 16;
                const bool put0 = mask0 || bad || i + 1 == u.tiles, put1 = two && (mask1 || bad || i + 2 == u.tiles);
                const int at0 = g % kFp4Entries, at1 = (g + (put0 ? 1 : 0)) % kFp4Entries;
                const bool mine = lane == 0 ? put0 : lane == 1 && put1;  // lanes 0 and 1 write a tile's entry
                const int my_at = lane == 0 ? at0 : at1;
                if (mine && DSA_IDX_OK(my_at, kFp4Entries, a.status)) {
                    s_mask[my_at] = (lane == 0 ? mask0 : mask1) | (bad ? kFp4Fault : 0ull);
                    const bool last = i + lane + 1 == u.tiles;
                    s_info[4 * my_at] = (first && (lane == 0 || !put0) ? kFirst : 0) | (last ? kLast : 0) | (ord & 3) * kOdd |
                                        (last && unit + unit_step >= units ? kFinal : 0);
                    s_info[4 * my_at + 1] = unit;
                    s_info[4 * my_at + 2] = u.m;
                }
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    const int kk = lane + 32 * e, slot = (kk < kFp4Keys ? at0 : at1) * kFp4Keys + kk % kFp4Keys;
                    if ((kk < kFp4Keys ? put0 : put1) && DSA_IDX_OK(slot, kFp4Entries * kFp4Keys, a.status)) s_addr[slot] = addr[e];
                }
                __syncwarp();
                if (mine) mbar_arrive(&rfull[my_at]);
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    const int kk = lane + 32 * e, key = kk % kFp4Keys;
                    const int slot = (kk < kFp4Keys ? at0 : at1) * 2 * kFp4Keys + key / 2 * 4 + (key & 1);
                    if ((kk < kFp4Keys ? put0 : put1) && DSA_IDX_OK(slot + 2, kFp4Entries * 2 * kFp4Keys, a.status)) {
                        float* k = s_ksc + slot;
                        k[0] = scale[e];
                        k[2] = scale[e] * a.scale_log2;
                    }
                }
                __syncwarp();
                if (mine) mbar_arrive(&kfull[my_at]);
                g += (put0 ? 1 : 0) + (put1 ? 1 : 0);
                first = first && !put0 && !put1;
            }
        }
        if (!ok && lane == 0) report(a.status, DSA_ERR_TIMEOUT);
    } else if (warp >= 8) {
        // ---- widen -------------------------------------------------------------------------------------------
        const int ww = warp - 8;
        // Converting, lane l = 16 q + t: of each pair of the warp's rows row q, and of each half of the dims block t (16 dims:
        // 16-byte pieces 2 (t & 3), 2 (t & 3) + 1 of 64-dim chunk t >> 2 of the half).  Lanes of odd chunks store their
        // second piece first, so that eight neighbouring lanes cover all banks.
        const int q = lane >> 4, t = lane & 15;
        const uint32_t raw = smem_u32(smem + L::kOffRaw) + ww * (kFp4PerWarp * kFp4BlockRow);
        const uint32_t raw_codes = raw + q * kFp4BlockRow + t * 8, raw_scale = raw + q * kFp4BlockRow + kD / 2 + t;
        const int hf = (t >> 2) & 1, p0 = 2 * (t & 3) + hf;
        const uint32_t dst0 = sK + (t >> 2) * kFp4Chunk;
        // Copying: the warp's rows are kFp4PerWarp * 18 pieces of 16 bytes, contiguous in shared memory; a lane's are lane + 32 n.
        constexpr int kPieces = kFp4PerWarp * 18, kCopies = (kPieces + 31) / 32;
        uint64_t src[kCopies];        // global addresses of the lane's pieces
        uint32_t src_bytes[kCopies];  // 16, or 0 to fill with zeros (a masked key)
        auto aim = [&](int g) {       // at tile g's rows
#pragma unroll
            for (int n = 0; n < kCopies; ++n) {
                const int p = lane + 32 * n, r = p / 18;
                const int key = g % kFp4Entries * kFp4Keys + ww * kFp4PerWarp + min(r, kFp4PerWarp - 1);
                const uint64_t at = DSA_IDX_OK(key, kFp4Entries * kFp4Keys, a.status) ? s_addr[key] : 0ull;
                src[n] = (at ? at : reinterpret_cast<uint64_t>(a.main.data)) + (p - 18 * r) * 16;
                src_bytes[n] = at ? 16u : 0u;
            }
        };
        auto copy = [&]() {
#pragma unroll
            for (int n = 0; n < kCopies; ++n)
                if (lane + 32 * n < kPieces && DSA_IDX_OK(ww * kPieces + lane + 32 * n, kFp4Keys * 18, a.status))
                    cp_async16_nc(raw + (lane + 32 * n) * 16, reinterpret_cast<const void*>(src[n]), src_bytes[n]);
            cp_async_commit();
        };
        ok = __all_sync(0xffffffffu, entry_wait(rfull, 0));
        if (ok) {
            aim(0);
            copy();
        }
        int done = 0;  // rows stored
        auto output = [&]() {  // the next finished row, whose last product is known to be complete
            const int par = done & 1;
            ok = __all_sync(0xffffffffu, wait_bar(ostat, par));
            if (!ok) return;
            const int unit = s_orow[par * 4], row = row_of(unit);
            tc_fence_after();
            store_row<NH>(a.rope, a.out + ((long long)row * a.heads + (unit - row * a.hg_count) * NH) * kD, tO, s_inv + par * NH,
                          ww, s_orow[par * 4 + 2], s_orow[par * 4 + 3], ofree);
            ++done;
        };
        int ends[3] = {0, 0, 0}, n_ends = 0;  // half-tiles after which the next rows' products are complete
        int slot = 0;
        uint32_t lap = 0;  // of the ring
#pragma unroll 1
        for (int g = 0; ok; ++g) {
            const int info = s_info[4 * (g % kFp4Entries)];
            const bool final = info & kFinal, last = info & kLast;
            if (final) {
#pragma unroll
                for (int n = 0; n < kCopies; ++n) src_bytes[n] = 0u;
            } else {  // tile g + 1's rows, whose copies follow each part of tile g that has been converted
                ok = __all_sync(0xffffffffu, entry_wait(rfull, g + 1));
                if (!ok) break;
                aim(g + 1);
            }
            if (ww == 0 && lane == 0) DSA_TRACE(g, 0);
            uint2 code[2][kFp4Pairs];
            uint32_t byte[2][kFp4Pairs];
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if (lap > 0) ok = ok && wait_bar(&pvdone[slot], (lap - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if constexpr (ROWS)
                    if (ok && n_ends > 0 && ends[0] + kFp4Ring == 2 * g + h) {  // that was a row's last product
                        output();
                        ends[0] = ends[1], ends[1] = ends[2], --n_ends;
                    }
                if (!ok) break;
                if (h == 0) {
                    cp_async_wait_all();
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < kFp4Pairs; ++u)
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            code[n][u] = lds64(raw_codes + 2 * u * kFp4BlockRow + n * (kD / 4));
                            byte[n][u] = lds8(raw_scale + 2 * u * kFp4BlockRow + n * 16);
                        }
                    __syncwarp();
                    copy();  // tile g + 1's rows take their place
                } else {
#pragma unroll
                    for (int u = 0; u < kFp4Pairs; ++u) code[0][u] = code[1][u], byte[0][u] = byte[1][u];
                }
                const uint32_t to = dst0 + slot * kFp4Half;
#pragma unroll
                for (int u = 0; u < kFp4Pairs; ++u) {
                    const int kk = ww * kFp4PerWarp + 2 * u + q;
                    const uint32_t at = to + (kk >> 3) * 1024 + (kk & 7) * 128, s2 = block_scale_2p118(byte[0][u]);
                    const uint32_t piece = (p0 ^ (kk & 7)) << 4;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t o[4];
                        widen8((e != 0) != (hf != 0) ? code[0][u].y : code[0][u].x, s2, o);
                        if (DSA_IDX_OK(at + (piece ^ (16u * e)) - sK, kFp4Ring * kFp4Half - 15, a.status))
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + (piece ^ (16u * e))), "r"(o[0]),
                                         "r"(o[1]), "r"(o[2]), "r"(o[3])
                                         : "memory");
                    }
                }
                fence_proxy_async_smem();  // the bf16 rows -> visible to the tensor core (async proxy)
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[slot]);
                if (++slot == kFp4Ring) slot = 0, ++lap;
            }
            if (ww == 0 && lane == 0) DSA_TRACE(g, 1);
            if constexpr (ROWS)
                if (last) {
                    const int end = 2 * g + 1;
                    if (n_ends == 0) ends[0] = end;
                    else if (n_ends == 1) ends[1] = end;
                    else ends[2] = end;
                    ++n_ends;
                }
            if (final) break;
        }
        if constexpr (ROWS)
            while (ok && n_ends > 0) {
                ok = __all_sync(0xffffffffu, wait_bar(&pvdone[ends[0] % kFp4Ring], (ends[0] / kFp4Ring) & 1));
                if (ok) output();
                ends[0] = ends[1], ends[1] = ends[2], --n_ends;
            }
        cp_async_wait_all();
        if (!ok && lane == 0) {
            report(a.status, DSA_ERR_TIMEOUT);
            if constexpr (ROWS) atomicMin(reinterpret_cast<int*>(smem + L::kOffFault), done);
        }
    } else if (warp == 5) {
        // ---- O^T += V^T P^T, issued by one elected lane ------------------------------------------------------
        const uint32_t idesc_o = idesc_bf16(NH, 1, 128);
        const uint64_t dp = sw128_desc(sP, 16, 1024), dv = sw128_desc(sK, kFp4Chunk, 1024);
        uint32_t rescales = 0, rows = 0;
        int slot = 0;
        for (int g = 0; ok; ++g) {
            const int b = g & 1;
            ok = wait_bar(&pfull[b], (g >> 1) & 1);  // P^T written (so S done, the half-tiles full)
            const int info = s_pinfo[b];
            if (ok && (s_vote[b * 4] | s_vote[b * 4 + 1] | s_vote[b * 4 + 2] | s_vote[b * 4 + 3]))
                ok = wait_bar(rdone, rescales++ & 1);
            if constexpr (ROWS)
                if (info & kFirst) {  // the previous row's O^T has been read
                    if (rows > 0) ok = ok && wait_bar(ofree, (rows - 1) & 1);
                    ++rows;
                }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) DSA_TRACE(g, 6);
            const uint32_t p_lo = __shfl_sync(0xffffffffu, (uint32_t)sw128_desc(sP + b * L::kP, 16, 1024), 0);
            const uint32_t more = info & kFirst ? 0u : 1u;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const uint32_t v_lo = __shfl_sync(0xffffffffu, (uint32_t)sw128_desc(sK + slot * kFp4Half, kFp4Chunk, 1024), 0);
                const uint32_t d = __shfl_sync(0xffffffffu, tO + 2 * h * NH, 0);
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int ks = 0; ks < kFp4Keys / 16; ++ks)
                        mma_bf16_ss_elect(d + mt * NH, desc_lo(dv, v_lo + (((2 * mt) * kFp4Chunk + (2 * ks) * 1024) >> 4)),
                                          desc_lo(dp, p_lo + ((ks * 32) >> 4)), idesc_o, ks > 0 ? 1u : more);
                mma_commit_elect(&pvdone[slot]);
                if (++slot == kFp4Ring) slot = 0;
            }
            if (lane == 0) DSA_TRACE(g, 7);
            if (info & kFinal) break;
        }
        if (!ok && lane == 0) report(a.status, DSA_ERR_TIMEOUT);
    } else if (warp == 4 || warp == 6) {
        // ---- S = Q K^T of every other tile, issued by one elected lane (one warp alone issues slower than the tensor
        // cores multiply) ------------------------------------------------------------------------------------
        const int b = warp == 6;
        const uint32_t idesc_s = idesc_bf16(kFp4Keys, 0, 64);
        const uint64_t dq = sw128_desc(sQ, 16, 1024);
        for (int g = b;; g += 2) {
            if (g > 0) {  // is there a tile g?
                ok = ok && entry_wait(rfull, g - 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const bool end = s_info[4 * ((g - 1) % kFp4Entries)] & kFinal;
                __syncwarp();
                if (lane == 0) mbar_arrive(&kfree[(g - 1) % kFp4Entries]);
                if (end) break;
            }
            if (g >= 2) ok = ok && wait_bar(&pfull[b], ((g >> 1) - 1) & 1);  // S buffer read
            int info = 0;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int n = 2 * g + h, slot = n % kFp4Ring;
                ok = ok && wait_bar(&full[slot], (n / kFp4Ring) & 1);
                if (h == 0) {
                    info = s_info[4 * (g % kFp4Entries)];
                    ok = ok && wait_bar(&qfull[info & kOdd ? 1 : 0], info & kOdd2 ? 1 : 0);  // the row's queries
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (lane == 0 && h == 0) DSA_TRACE(g, 2);
                // 64-dim chunks: 64 query rows / 48 key rows apart
                const uint32_t q_lo = __shfl_sync(0xffffffffu, (uint32_t)dq + ((4 * h * 8192) >> 4), 0);
                const uint32_t k_lo = __shfl_sync(0xffffffffu, (uint32_t)sw128_desc(sK + slot * kFp4Half, 16, 1024), 0);
                const uint32_t d = __shfl_sync(0xffffffffu, tS + b * 64, 0);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    mma_bf16_ss_elect(d, desc_lo(dq, q_lo + (((i >> 2) * 8192 + (i & 3) * 32) >> 4)),
                                      desc_lo(dq, k_lo + (((i >> 2) * kFp4Chunk + (i & 3) * 32) >> 4)), idesc_s,
                                      i > 0 ? 1u : (uint32_t)h);
            }
            if (!ok) break;
            const int unit = s_info[4 * (g % kFp4Entries) + 1];
            mma_commit_elect(&sfull[b]);
            if (lane == 0) DSA_TRACE(g, 3);
            if (info & kFinal) break;
            if constexpr (ROWS) {
                if ((info & kFirst) && unit + unit_step < units && lane == 0) {  // the next unit's queries, towards L2
                    const int row = row_of(unit + unit_step);
                    const long long qrow = (long long)row * a.heads + (unit + unit_step - row * a.hg_count) * NH;
                    prefetch_l2(a.q + qrow * kD, NH * kD * 2);
                }
                if (info & kLast) {  // the row's last product: the next queries take their place
                    ok = wait_bar(&sfull[b], (g >> 1) & 1);
                    if (g > 0) ok = ok && wait_bar(&sfull[b ^ 1], ((g - 1) >> 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    load_q(unit + unit_step, info & kOdd ? 0 : 1);
                }
            }
        }
        if (!ok && lane == 0) report(a.status, DSA_ERR_TIMEOUT);
    } else if (warp < 4) {
        // ---- softmax: heads 16 warp + lane / 4 and + 8, keys 8 e + 2 (lane % 4), + 1 -----------------------------
        const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
        const int hr = lane >> 2, c = lane & 3, head0 = warp * 16 + hr;
        // m_run: the head's running maximum, lazy: it moves only when exceeded by more than 2^8, so O^T is rarely
        // rescaled and exp2(s - m) <= 2^8.  l_run: the lane's share of the sum of the probabilities as rounded for P V (the
        // output's normaliser: values that all keys share come out exactly), two halves; e_run: of the fp32 probabilities
        // (the log-sum-exp).  The prefill below takes 327 us so, 318 with one sum of fp32 probabilities
        float m_run[2] = {-INFINITY, -INFINITY};
        uint64_t l_run[2] = {0ull, 0ull}, e_run[2] = {0ull, 0ull};
        bool seen = false;  // a fault bit in one of the row's masks
        int rows = 0;
        auto wait_pv = [&](int g) { return wait_bar(&pvdone[(2 * g + 1) % kFp4Ring], ((2 * g + 1) / kFp4Ring) & 1); };
        // O^T times alpha per head, when a head's maximum moved in tile g: after the other warps' votes for the tile are
        // in (their P^T is written) and the product of tile g - 1 is done; the product of tile g waits for it
        auto rescale = [&](int g) {
            const int b = g & 1;
            ok = ok && wait_bar(&pfull[b], (g >> 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || !(s_vote[b * 4] | s_vote[b * 4 + 1] | s_vote[b * 4 + 2] | s_vote[b * 4 + 3])) return;
            ok = __all_sync(0xffffffffu, wait_pv(g - 1));
            if (ok) {
                tc_fence_after();
                rescale_quadrant<NH>(tO + lane_off, s_alpha + b * NH);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(rdone);
        };
        for (int g = 0;; ++g) {
            const int b = g & 1, at = g % kFp4Entries;
            if (g > 0) rescale(g - 1);
            ok = ok && entry_wait(kfull, g);  // the tile's scales, mask and flags
            ok = ok && wait_bar(&sfull[b], (g >> 1) & 1);
            if (g >= 2) ok = ok && wait_pv(g - 2);  // P^T buffer free
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (tid == 0) DSA_TRACE(g, 4);
            const int info = s_info[4 * at];
            if (info & kFirst) {
                m_run[0] = m_run[1] = -INFINITY;
                l_run[0] = l_run[1] = e_run[0] = e_run[1] = 0ull;
                seen = false;
            }
            float alpha[2] = {1.f, 1.f};
            bool resc = false;
            tc_fence_after();
            float sv[24];  // logits of head h in 4 e + 2 h, 4 e + 2 h + 1: keys 8 e + 2 c, + 1
            tmem_ld_16x48_nowait(tS + b * 64 + lane_off, sv);
            const float2* k2 = reinterpret_cast<const float2*>(s_ksc + at * 2 * kFp4Keys) + 2 * c;
            const uint64_t vm = s_mask[at];
            seen = seen || (vm & kFp4Fault);
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
                const float2 k = k2[8 * e + 1];
                const uint64_t kl = pack_f32x2(k.x, k.y);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    unpack_f32x2(fma_f32x2(pack_f32x2(sv[4 * e + 2 * h], sv[4 * e + 2 * h + 1]), kl, neg[h]),
                                 &sv[4 * e + 2 * h], &sv[4 * e + 2 * h + 1]);
            }
            if ((vm & kFp4AllValid) != kFp4AllValid) {
#pragma unroll
                for (int e = 0; e < kFp4Groups; ++e) {
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
                for (int e = 1; e < kFp4Groups; ++e) mx[h] = fmaxf(mx[h], fmaxf(sv[4 * e + 2 * h], sv[4 * e + 2 * h + 1]));
                mx[h] = quad_max(mx[h]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (mx[h] > (m_run[h] == -INFINITY ? -INFINITY : kLazyLog2)) {  // also the first finite maximum
                    const float m_new = m0[h] + mx[h];
                    alpha[h] = exp2f(m_run[h] - m_new);
                    resc = !(info & kFirst);
                    m_run[h] = m_new;
#pragma unroll
                    for (int e = 0; e < kFp4Groups; ++e) {
                        sv[4 * e + 2 * h] -= mx[h];
                        sv[4 * e + 2 * h + 1] -= mx[h];
                    }
                }
            }
            float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
            uint64_t esum[2] = {0ull, 0ull};
            const uint32_t prow = sP + b * L::kP + head0 * 128 + 4 * c;
#pragma unroll
            for (int e = 0; e < kFp4Groups; ++e) {
                const float2 k = k2[8 * e];
                const uint64_t ks = pack_f32x2(k.x, k.y);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint64_t p = pack_f32x2(ex2_sfu(sv[4 * e + 2 * h]), ex2_sfu(sv[4 * e + 2 * h + 1]));
                    esum[h] = add_f32x2(esum[h], p);
                    float p0, p1;
                    unpack_f32x2(p, &p0, &p1);
                    add_bf16x2(bf16x2_rn(p0, p1), sum[h]);
                    // the probability that multiplies the codes carries the row scale: a power of two, so it rounds alike
                    unpack_f32x2(mul_f32x2(p, ks), &p0, &p1);
                    if ((NH == 64 || head0 + 8 * h < NH) &&
                        DSA_IDX_OK(prow + h * 1024 + ((e ^ (hr & 7)) << 4) - sP, 2 * L::kP - 3, a.status))
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(prow + h * 1024 + ((e ^ (hr & 7)) << 4)),
                                     "r"(bf16x2_rn(p0, p1))
                                     : "memory");
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l_run[h] = fma_f32x2(l_run[h], pack_f32x2(alpha[h], alpha[h]), pack_f32x2(sum[h][0], sum[h][1]));
                e_run[h] = fma_f32x2(e_run[h], pack_f32x2(alpha[h], alpha[h]), esum[h]);
            }
            if (c == 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (NH == 64 || head0 + 8 * h < NH) s_alpha[b * NH + head0 + 8 * h] = alpha[h];
            }
            const bool any = __any_sync(0xffffffffu, resc);
            if (lane == 0) {
                s_vote[b * 4 + warp] = any ? 1 : 0;
                if (warp == 0) s_pinfo[b] = info;
            }
            if constexpr (ROWS)  // the row before this one has been stored (P V of this row waits for that, too): no output
                             // still reads the factors whose place this row's take
                if ((info & kLast) && rows > 0) ok = __all_sync(0xffffffffu, wait_bar(ofree, (rows - 1) & 1));
            fence_proxy_async_smem();  // P^T stores -> async proxy
            tc_fence_before();
            __syncwarp();
            const int unit = s_info[4 * at + 1], pos = s_info[4 * at + 2];
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&pfull[b]);
                mbar_arrive(&kfree[at]);
            }
            if (tid == 0) DSA_TRACE(g, 5);
            if (info & kLast) {
                const bool fault = seen;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int head = head0 + 8 * h;
                    float l0, l1, e0, e1;
                    unpack_f32x2(l_run[h], &l0, &l1);
                    unpack_f32x2(e_run[h], &e0, &e1);
                    const float l = quad_sum(l0 + l1), e = quad_sum(e0 + e1);
                    if (c != 0 || (NH < 64 && head >= NH)) continue;
                    if constexpr (ROWS) {  // the output's factor, and the log-sum-exp
                        const bool some = !(l <= 0.f) && !fault;
                        s_inv[(rows & 1) * NH + head] = some ? (float)(1 << kFp4Shift) / l : 0.f;
                        const int row = row_of(unit);
                        if (a.lse)
                            a.lse[(long long)row * a.heads + (unit - row * a.hg_count) * NH + head] =
                                some ? (m_run[h] + log2f(e)) / kLog2e : -INFINITY;
                    } else {  // read after the last product (their place is in the ring)
                        l_run[h] = pack_f32x2(l, e);
                    }
                }
                if constexpr (ROWS) {
                    if (tid == 0) {
                        s_orow[(rows & 1) * 4] = unit;
                        s_orow[(rows & 1) * 4 + 2] = pos;
                        s_orow[(rows & 1) * 4 + 3] = fault;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ostat);
                    ++rows;
                }
            }
            if (info & kFinal) {
                rescale(g);
                if constexpr (!ROWS) {  // the last product must be complete before O^T is read
                    ok = __all_sync(0xffffffffu, ok && wait_pv(g));
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int head = head0 + 8 * h;
                        float l, e;
                        unpack_f32x2(l_run[h], &l, &e);
                        if (c == 0 && (NH == 64 || head < NH)) {
                            // a NaN among masked or absent maxima only: give the partial a weight, so that the NaN
                            // reaches the row
                            s_own[head] = m_run[h] == -INFINITY && l != l ? 0.f : m_run[h];
                            s_own[NH + head] = l;
                            s_own[2 * NH + head] = e;
                        }
                    }
                    if (tid == 0 && seen) *s_fault = 1;
                }
                break;
            }
        }
        if (!ok && lane == 0) report(a.status, DSA_ERR_TIMEOUT);
    }

    if constexpr (ROWS) {
        tc_fence_before();
        const bool all_ok = __syncthreads_and(ok);
        tc_fence_after();
        if (warp == 0) tmem_dealloc(tmem, L::kTmemCols);
        if (!all_ok) zero_rows<NH>(a, unit0, unit_step, units, *s_fault);
    } else {
        const int row = row_of(unit0);
        attn_finish<NH, L, false, kFp4Shift, true>(a, &omap, smem, tmem, tO, row, split, unit0 - row * a.hg_count, crank,
                                                   csize, 1, ok);
    }
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
    const long long units = (long long)a.rows * a.hg_count, grid = units * a.nsplit * cl;
    if (grid > 0x7fffffffll) return DSA_ERR_UNSUPPORTED;
    // whole rows in a CTA, written as bf16: the kernel that runs on from row to row (the e4m3 output needs each 128-dim
    // block's largest value first)
    const bool rows = cl == 1 && a.nsplit == 1 && !a.out8;
    auto kernel = rows ? attn_fp4_kernel<NH, true> : attn_fp4_kernel<NH, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc) != cudaSuccess)
        return DSA_ERR_CUDA;
    cudaError_t e;
    if (rows)
        e = launch_pdl(kernel, dim3((unsigned)std::min<long long>(units, sm_count())), dim3(kClThreads), L::kAlloc, st,
                       qmap, omap, a);
    else
        e = launch_pdl_cluster(kernel, dim3((unsigned)grid), dim3(kClThreads), L::kAlloc, st, cl, qmap, omap, a);
    if (e == cudaSuccess && a.nsplit > 1) e = launch_attn_combine(a, st);
    if (e != cudaSuccess) return DSA_ERR_CUDA;
    return launch_status();
}

int fp4_clusters(int cl) {
    int dev = 0;
    if (cl == 1 || cudaGetDevice(&dev) != cudaSuccess) return sm_count() / cl;
    static std::atomic<int> known[16][2];  // by device and cluster size; 0: not asked yet
    std::atomic<int>* const seen = dev < 16 ? &known[dev][cl == 4] : nullptr;
    if (seen && seen->load(std::memory_order_relaxed) > 0) return seen->load(std::memory_order_relaxed);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(sm_count() / cl * cl));
    cfg.blockDim = dim3(kClThreads);
    cfg.dynamicSmemBytes = Fp4Smem<64>::kAlloc;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool clean = cudaPeekAtLastError() == cudaSuccess;
    if (cudaFuncSetAttribute(attn_fp4_kernel<64, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Fp4Smem<64>::kAlloc) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, attn_fp4_kernel<64, false>, &cfg) != cudaSuccess || n < 1) {
        if (clean) cudaGetLastError();  // this question's own error, not one that the caller has not seen yet
        return sm_count() / cl;
    }
    if (seen) seen->store(n, std::memory_order_relaxed);
    return n;
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
