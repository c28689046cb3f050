// Verify attention over an 8-bit history on tensor cores (bf16 queries and tails, head
// dimension 64 or 128, any group size), written for sm_103a.
//
// Both products are formed transposed, with the keys (and then the head dimension) as the
// M = 128 operand and the query rows of the KV-head group as N:
//   S^T[key, row] = K Q^T            A = K (tensor memory), B = Q (shared memory)
//   O^T[dim, row] += V^T P^T         A = V^T (tensor memory), B = P (shared memory, MN-major)
// A verify step has few rows (4 to 128 for a KV head), so rows in M would leave most of every
// tensor instruction idle (44 of 128 rows for an 11-node chain); in N they cost what they
// are, in steps of 16.  It also gives every softmax thread one key: the key's page scale is
// one number of the thread, and the running maximum needs no reduction at all until some
// score passes its reference by more than 2^8 (the group of warps votes; the reference of the
// row then moves, O is rescaled, and the tile is taken again).
//
// The 8-bit codes become fp16 exactly, so K and V lose nothing.  Q is held as fp16 times one power
// of two for the CTA (its largest magnitude becomes 2^14..2^15, so elements down to 2^-30 of that
// keep all 8 bits of a bf16).  Where some 16 bytes of Q hold nothing above 2^-20 of its largest (a
// padded batch's rows may hold anything), or its largest is below 2^-86, Q stays bf16 and K becomes
// bf16 over the pages too, both exact: no row depends on what another holds.
//
// P is fp16 of 2^(s - ref), 2^7 at the reference and below 2^15, so it keeps 11 bits down to 2^-21
// of the row's largest and fades out below 2^-31.
//
// V takes its page's scale relative to a unit, the power of two at or below the largest scale of
// the CTA's pages, which multiplies O at the end: exact for powers of two down to 2^-15, where
// e4m3's smallest code is fp16's.  Other scales and their products are rounded to fp16, 2^-11 each,
// as long as the products are normal numbers, down to 2^-5.  Where the V scales of a CTA's pages
// lie further apart (an all-zero block, whose scale is 1, beside values below 2^-7 is enough), or
// the unit is so far from 1 that the tail rows' P, which are divided by it, could leave fp32's
// range, V and P are bf16 over its pages too, with V at its true size: bf16 has fp32's exponents,
// so a page counts by its probability and its values whatever lies beside it, and P (and V with a
// scale that is no power of two) keeps 8 bits.  Tail rows and speculative rows are bf16 as they
// are: those tiles, the last of a sequence, run the same way in bf16.
//
// Both operands that come from the cache are converted in registers on their way from the raw
// stages to tensor memory, K by rows and V through transposing 8-bit ldmatrix loads, so a
// code byte crosses shared memory twice (copy in, read out).  With V as a shared-memory
// operand in fp16 it would be written and read there once more at twice the width, and
// shared-memory bandwidth (128 B a clock), not HBM, bounded that version (72 us where this
// one takes 66 with the same roles).
//
// CTA = (sequence and split, block of at most 128 group rows; KV head).  Tiles are 128 keys:
// two pages, or 128 tail rows.  Warps:
//   softmax     groups of 4; warp w owns the keys, later the output dimensions, of
//               tensor-memory lane quadrant w % 4.  Up to 48 rows two groups take the tiles in
//               turn, each with its own references and O^T, joined at the end; above, four
//               groups take every tile and a quarter of its rows (launch_rows).  The chain of a
//               tile (load S, compare, vote, exponentials, store P) takes a group 2200 to 2700
//               cycles, nearly whatever its columns: warps' latencies, not a unit's rate
//   converters  4 for K and 4 for V
//   chooser     1: from the softmax warps' maxima of Q and of V's scales, the powers of two that the
//               fp16 forms are relative to, or that the split is wide (bf16)
//   producer    1: copies pages (K and V of a page and head are 128 d contiguous bytes)
//               into a ring of raw stages by TMA
//   issuer      1: the MMAs, in the order in which their inputs become ready
// Every wait is bounded in wall-clock time; after a failed wait the kernel records an error
// code, stops issuing, drains and returns.
//
// Measured with the merge (us, floor by bytes at 6778 GB/s): 11 queries of 32 heads over 8 KV
// heads, d = 128: 120K 46.5 (37.2), 32K 21.7 (10.0); one query over 4K 8.7 (1.3); 64 heads
// over 8, 128K 76 (39.7); d = 64, 120K 39 (18.6); a tree of 32 nodes, 28 heads over 4, four
// histories of 32K to 96K 187 (40; 62 by tensor rate).  Of a call about 9 us are the start (the
// lengths, page ids and first pages one after the other, cold code, the first references) and the
// end (join, merge).  In between, 44 rows take 1400 cycles a tile, what HBM delivers; more
// rows, and d = 64, whose tiles are half the bytes, are bound by the softmax warps' chain: with
// the polls of waiting warps cut by a third, or with naps between them, the times stay, and so
// they do with the vote on a barrier phase of its own that overlaps the exponentials (8 % more).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <cstddef>

#include "attn_q8.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace rapid {

namespace {

constexpr int kMaxRawStages = 6;
constexpr int kFlagged = 64;           // elements of V remembered for not being finite
constexpr uint32_t kTmemCols = 512;

constexpr float kRefShift = 7.f;       // P is 2^7 at the reference ...
constexpr float kNoKey = 3e38f;        // -(reference) of a row that has seen no key: any finite
                                       // score passes it
constexpr float kMaxLog2P = 15.f;      // ... and the reference moves before P passes 2^15
                                       // (fp16 ends at 65504)
constexpr float kLeastRel = 1.f / 32768;   // least V scale, relative to the unit, that fp16 holds ...
constexpr float kOddScale = 1.f / 1024;    // ... of powers of two; others count that much smaller
constexpr int kMostQ = 20;                 // log2 of the range of Q's pieces that fp16 takes ...
constexpr int kLeastQ = -86;               // ... and of its largest
constexpr float kMostUnit = 4294967296.f;  // 2^32: a unit past it or below its reciprocal is not used

// COLS: rows of one softmax group (a multiple of 8).  ALT: two groups take tiles in turn (all
// rows each); else four take every tile, a quarter of the rows each.
template <int D, int COLS, bool ALT>
struct Plan {
    static constexpr int kGroups = ALT ? 2 : 4;
    static constexpr int kN = ALT ? COLS : 4 * COLS;        // N of the products
    static constexpr int kConvWarp = 4 * kGroups;
    static constexpr int kSoftmaxThreads = 128 * kGroups;
    static constexpr int kProducerWarp = kConvWarp + 8;              // 4 for K, 4 for V
    static constexpr int kChooserWarp = kProducerWarp + 1;
    static constexpr int kMmaWarp = kProducerWarp + 3;
    static constexpr int kThreads = 32 * (kProducerWarp + 4);
    // A block starts with kLaunchRegs registers a thread; its warpgroups share them out anew.
    static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
    static constexpr int kSoftmaxRegs = ALT ? (COLS <= 32 ? 112 : 136) : 88;
    static constexpr int kConvRegs = ALT ? (COLS <= 32 ? 96 : 80) : 56;
    static constexpr int kLastRegs = ALT ? (COLS <= 32 ? 56 : 48) : 40;
    static_assert(kGroups * kSoftmaxRegs + 2 * kConvRegs + kLastRegs <= kLaunchRegs * (kThreads / 128),
                  "registers of a block");
    // Tensor-memory columns: K and V tiles (64 each), O^T (of each group), two S^T buffers.
    static constexpr int kKBufs = kN <= 64 ? 2 : 1;
    static constexpr int kVBufs = kN <= 96 ? 2 : 1;
    static constexpr uint32_t kNCols = kN < 32 ? 32 : kN;
    static constexpr uint32_t kTmemK = 0;
    static constexpr uint32_t kTmemV = 64 * kKBufs;
    static constexpr uint32_t kTmemO = kTmemV + 64 * kVBufs;
    static constexpr uint32_t kTmemS = kTmemO + (ALT ? 2 : 1) * kNCols;
    static_assert(kTmemS + 2 * kNCols <= kTmemCols, "tensor memory");
    static constexpr int kPageBytes = 2 * kPageTokens * D;  // K and V of one page and head
    static constexpr int kRawBytes = 2 * kPageBytes;        // one stage: two pages
    static constexpr int kPBuf = (kN + 63) / 64 * (kQ8Tile * 128);
    static constexpr int kPBytes = (ALT ? 2 : 1) * kPBuf;   // one for each group in ALT
    static constexpr int kQBlock = kN * 128;                // 64 dimensions of Q
    static constexpr int kOffP = 0;
    static constexpr int kOffQ = kOffP + kPBytes;
    static constexpr int kOffRaw = kOffQ + (D / 64) * kQBlock;
    static constexpr int kScalarBytes = 4096;
    static constexpr int kFit = (232448 - 1024 - kScalarBytes - kOffRaw) / kRawBytes;
    static constexpr int kStages = kFit < kMaxRawStages ? kFit : kMaxRawStages;
    static constexpr int kOffScalar = kOffRaw + kStages * kRawBytes;
    static constexpr int kSmemBytes = kOffScalar + kScalarBytes + 1024;
    static_assert(D == 64 || D == 128, "head dimension 64 or 128");
    static constexpr int kPart = ALT ? 64 : 32;             // numbers of a warp in Scalars::part
    static_assert(COLS % 8 == 0 && COLS <= kPart, "rows of a group");
    static_assert(kOffRaw % 1024 == 0 && kStages >= 3, "raw stages");
};

struct Scalars {
    uint64_t raw_full[kMaxRawStages];
    uint64_t raw_free[kMaxRawStages];
    uint64_t q_full;         // Q in shared memory
    uint64_t k_full[2];      // K in tensor memory
    uint64_t s_full[2];      // S^T done (and K's buffer free)
    uint64_t s_free[2];      // S^T loaded by the softmax warps
    uint64_t v_full[2];      // V^T in tensor memory
    uint64_t pv_done[2];     // O^T += V^T P^T of a tile done (V's buffer and P free)
    uint64_t p_full[2];      // P of a tile in shared memory (of each group in ALT)
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    Q8Split split;
    Q8Keys keys;
    alignas(16) float neg_ref[128];   // -(reference) of every row (64 g + row in ALT): P = 2^(s + neg_ref)
    alignas(16) float corr[128];
    float part[512];         // per softmax warp: a number for each of its rows
    float wunit[16], wlow[16];
    uint16_t wmax[16], wleast[16];
    int fail[4];             // a softmax group's failed wait
    int q_wide;              // Q as it is, K of the pages in bf16
    float q_mul;             // else the power of two of Q's fp16 form
    float unit;              // power of two below the largest V scale of the split: O = unit * O^T; or -1
                             // where they are wide (V and P of the pages in bf16, O = O^T)
    int flagged;             // elements of the tail rows' V that are not finite
    int64_t flagged_at[kFlagged];      // row * d + dimension
};
static_assert(sizeof(Scalars) <= 4096, "scalar block too small");
static_assert(offsetof(Scalars, neg_ref) % 16 == 0 && offsetof(Scalars, corr) % 16 == 0,
              "rows' references are read four at a time");

enum : unsigned int {
    kRoleProducer = 0x11u << 24, kRoleMma = 0x12u << 24, kRoleSoftmax = 0x13u << 24,
    kRoleConvert = 0x14u << 24,
    kBarRawFull = 1u << 16, kBarRawFree = 2u << 16, kBarS = 3u << 16, kBarPv = 4u << 16,
    kBarK = 5u << 16, kBarDrain = 6u << 16, kBarQ = 7u << 16, kBarP = 8u << 16, kBarV = 9u << 16
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// This warpgroup's registers a thread from NOW to N.  An increase waits for registers that the
// others release; a decrease to more than there are is an illegal instruction.
template <int NOW, int N> __device__ __forceinline__ void set_regs() {
    static_assert(N >= 24 && N <= 256 && N % 8 == 0 && NOW % 8 == 0, "registers in steps of 8");
    if constexpr (N > NOW) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    if constexpr (N < NOW) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float warp_max_redux(float x) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
}
// Four e4m3 codes to four fp16 values (exact).
__device__ __forceinline__ uint2 e4m3x4_to_f16x4(uint32_t w) {
    uint2 r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(w));
    return r;
}

// Barrier `id` of N threads with an OR over them: the same answer in each.
template <int N>
__device__ __forceinline__ bool barrier_any(int id, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(id), "n"(N)
        : "memory");
    return r != 0;
}
// ... of one softmax group.
__device__ __forceinline__ bool group_any(int gr, bool x) { return barrier_any<128>(1 + gr, x); }
__device__ __forceinline__ void group_sync(int gr) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + gr) : "memory");
}

// Instruction descriptor: fp32 sums, A and B fp16 or bf16, A K-major, B K- or MN-major, M = 128.
constexpr uint32_t idesc(bool bf16, bool b_mn, int n) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ uint32_t timer_low() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
// Shared addresses of the loops, as numbers that the compiler does not see through: it would
// otherwise work an address out again from the CTA's window at every use (four instructions
// and a special register: 14 such reads for a tile and softmax warp).
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
    asm volatile("mov.b32 %0, %0;" : "+r"(x));
    return x;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds_u4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts_u4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
// Test of a phase that the hardware suspends for a while (a system-dependent time, after which
// it is false): a waiting warp takes few issue slots from the others.
__device__ __forceinline__ bool try_suspended(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits, bounded in time by the low word of the nanosecond clock (2^30 of them, about a second;
// legitimate waits last microseconds).  A role keeps the code of the wait that gave up and
// records it once, at its end: a wait has to be a few instructions, because the roles' loops
// share a small instruction cache and a launch fetches them anew.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, unsigned code, unsigned& failed) {
    if (try_suspended(bar, parity)) return true;
    const uint32_t t0 = timer_low();
    do {
        if (try_suspended(bar, parity)) return true;
    } while (timer_low() - t0 < 1u << 30);
    failed = code;
    return false;
}
__device__ __forceinline__ void record(unsigned int* err, unsigned failed) {
    if (failed && err) {
        atomicOr(err, kErrWaitTimeout);
        atomicCAS(err + 1, 0u, failed | 0x80000000u);
    }
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A V scale as the choice between fp16 and bf16 counts it.
__device__ __forceinline__ float counted(float scale) {
    return (__float_as_uint(scale) & 0x7fffffu) ? scale * kOddScale : scale;
}
// Scale of V of a page (an id outside the pool, which the producer flags, reads as page 0).
__device__ __forceinline__ float v_scale(const AttnQ8Params& p, int page, int g) {
    const int id = (unsigned)page < (unsigned)p.n_pages ? page : 0;
    return __ldg(p.scales + ((int64_t)id * p.Hkv + g) * 2 + 1);
}
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// STEPS products of 16 in a row, issued by the lane with `leader` set: A in tensor memory, 8
// columns a step; B's descriptor low word grows by B_STEP a step, by B_JUMP more after four
// steps.  The first one starts the sum where `accumulate` is 0.
template <int STEPS, int B_STEP, int B_JUMP>
__device__ __forceinline__ void mma_chain_if(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                             uint32_t idesc, uint32_t accumulate) {
#pragma unroll
    for (int k = 0; k < STEPS; k += 4) {
        asm volatile(
            "{\n\t.reg .pred p, q, t;\n\t"
            ".reg .b64 b1, b2, b3;\n\t"
            ".reg .b32 a1, a2, a3;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "setp.eq.b32 t, 0, 0;\n\t"
            "add.u32 a1, %1, 8;\n\t"
            "add.u32 a2, %1, 16;\n\t"
            "add.u32 a3, %1, 24;\n\t"
            "add.u64 b1, %2, %6;\n\t"
            "add.u64 b2, %2, %7;\n\t"
            "add.u64 b3, %2, %8;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d_tmem),
            "r"(a_tmem + (uint32_t)(8 * k)), "l"(b + (uint64_t)(k * B_STEP + (k >> 2) * B_JUMP)), "r"(idesc),
            "r"(k > 0 ? 1u : accumulate), "r"(leader), "n"(B_STEP), "n"(2 * B_STEP), "n"(3 * B_STEP)
            : "memory");
    }
}
__device__ __forceinline__ void mma_commit_if(uint32_t leader, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}

// Two transposed 16 x 16 byte matrices; lanes 0..15 and 16..31 give the addresses of their rows.
__device__ __forceinline__ void ldmatrix_t_b8_x2(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Sums of v[0..7] over the warp; lane l returns the one of column l / 4 (halving the columns
// a lane carries at each of the first three exchanges: 9 shuffles instead of 40).
__device__ __forceinline__ float warp_sum8(float (&v)[8], int lane) {
    float a[4], c[2];
    const bool h4 = lane & 16, h2 = lane & 8, h1 = lane & 4;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        a[e] = (h4 ? v[4 + e] : v[e]) + __shfl_xor_sync(0xffffffffu, h4 ? v[e] : v[4 + e], 16);
#pragma unroll
    for (int e = 0; e < 2; ++e)
        c[e] = (h2 ? a[2 + e] : a[e]) + __shfl_xor_sync(0xffffffffu, h2 ? a[e] : a[2 + e], 8);
    float s = (h1 ? c[1] : c[0]) + __shfl_xor_sync(0xffffffffu, h1 ? c[0] : c[1], 4);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    return s + __shfl_xor_sync(0xffffffffu, s, 1);
}

// The pages of a wide split, K or V, as bf16 into tensor memory: K where the pieces of Q are too far
// apart, V at its true size where the V scales are too far apart or too far from 1.  The converters'
// loop over again, apart from theirs because the same code inside it costs the splits that never
// reach it 1 to 5 us.  Every code takes two conversions more than to fp16: a 120K chain whose V is
// wide 83 us, whose Q is 65 (46.5 otherwise), 64 heads over 8 at 128K 98 and 93 (76), the tree 223
// and 205 (187).  Returns the code of a wait that gave up, or 0.
template <int D, int COLS, bool ALT>
static __device__ __noinline__ unsigned wide_tiles(const AttnQ8Params& p, const int32_t* ids, int pages, int g,
                                                   int tiles, bool do_k, uint32_t sb, uint32_t src,
                                                   uint32_t piece0, uint32_t lanes) {
    using L = Plan<D, COLS, ALT>;
    const int lane = threadIdx.x & 31;
    const uint32_t swizzle = (uint32_t)(D == 128 ? lane : lane >> 1) & 7u;   // of V's lines
    unsigned failed = 0;
    int st = 0;
    uint32_t lap = 0;
    auto bar = [&](size_t offset, int i) -> uint32_t { return sb + (uint32_t)offset + 8u * (uint32_t)i; };
    auto scale_of = [&](int page) -> float {            // K's scale is the softmax warps' business
        return do_k ? 1.f : page < pages ? v_scale(p, __ldg(ids + page), g) : 0.f;
    };
    float next0 = scale_of(0), next1 = scale_of(1);
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
        const float s0 = next0, s1 = next1;
        next0 = scale_of(2 * i + 2);
        next1 = scale_of(2 * i + 3);
        const unsigned code = kRoleConvert | (unsigned)(i & 0xffff);
        const int bufs = do_k ? L::kKBufs : L::kVBufs, j = i - bufs;
        bool ok = wait_for(bar(offsetof(Scalars, raw_full), st), lap, code | kBarRawFull, failed);
        if (ok && j >= 0)                               // the product that read this buffer last
            ok = wait_for(bar(do_k ? offsetof(Scalars, s_full) : offsetof(Scalars, pv_done), j & 1),
                          (uint32_t)((j >> 1) & 1), code | (do_k ? kBarS : kBarPv), failed);
        if (!__all_sync(0xffffffffu, ok)) return failed ? failed : code;
        tc_fence_after();
        const uint32_t from = src + (uint32_t)(st * L::kRawBytes);
        const uint32_t dst = lanes + (do_k ? L::kTmemK : L::kTmemV) + (uint32_t)(64 * (i % bufs));
        const bool two = 2 * i + 1 < pages;
#pragma unroll 1
        for (int h = 0; h < D / 64; ++h) {
            // K: 16 codes of the thread's key, 8 columns.  V: 32 keys x 16 dimensions, 16 columns of
            // 16 lanes; a page that is not there reads as zeros.
            uint32_t r[4][4] = {};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (do_k) {
                    const uint4 v = lds_u4(from ^ (uint32_t)((4 * h + m) << 4));
                    r[m][0] = v.x; r[m][1] = v.y; r[m][2] = v.z; r[m][3] = v.w;
                } else if (m < 2 || two) {
                    ldmatrix_t_b8_x2(from + (uint32_t)((m >> 1) * L::kPageBytes + (m & 1) * 32 * D) +
                                         (((piece0 + (uint32_t)h) ^ swizzle) << 4), r[m]);
                }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float s = m < 2 ? s0 : s1;
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint2 y = e4m3x4_to_f16x4(r[m][e]);
                    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&y.x));
                    const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&y.y));
                    w[2 * e] = bf16x2(a.x * s, a.y * s);
                    w[2 * e + 1] = bf16x2(c.x * s, c.y * s);
                }
                if (do_k) tmem_st8(dst + (uint32_t)(8 * (4 * h + m)), w);
                else tmem_st_16x256b_x2(dst + ((uint32_t)(16 * h) << 16) + (uint32_t)(16 * m), w);
            }
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(bar(do_k ? offsetof(Scalars, k_full) : offsetof(Scalars, v_full), i % bufs));
        __syncwarp();
        if (lane == 0) arrive(bar(offsetof(Scalars, raw_free), st));
        if (++st == L::kStages) { st = 0; lap ^= 1u; }
    }
    return 0;
}

template <int D, int COLS, bool ALT>
__global__ void __launch_bounds__(Plan<D, COLS, ALT>::kThreads, 1)
attn_q8_tc_kernel(const __grid_constant__ CUtensorMap pool, const AttnQ8Params p, const int n_rb,
                  const int rows_per_block) {
    using L = Plan<D, COLS, ALT>;
    constexpr int kStages = L::kStages, kN = L::kN, KB = L::kKBufs, VB = L::kVBufs;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Scalars* sc = reinterpret_cast<Scalars*>(smem + L::kOffScalar);

    // the warp index through a shuffle: known to be the same in all lanes, so that the roles'
    // branches, addresses and descriptors stay on the uniform path
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int slot_idx = blockIdx.x / n_rb, rb = blockIdx.x - slot_idx * n_rb;
    const int g = blockIdx.y;
    const int r0 = rb * rows_per_block;                 // first group row of this CTA
    const int Rb = min(rows_per_block, p.R - r0);       // its rows

    if (tid == 32) {
#pragma unroll 1
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sc->raw_full[i], 1);
            mbar_init(&sc->raw_free[i], 8);
        }
        mbar_init(&sc->q_full, L::kSoftmaxThreads);
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
            mbar_init(&sc->k_full[u], 128);
            mbar_init(&sc->s_full[u], 1);
            mbar_init(&sc->s_free[u], ALT ? 4 : 4 * L::kGroups);
            mbar_init(&sc->p_full[u], ALT ? 128 : L::kSoftmaxThreads);
            mbar_init(&sc->v_full[u], 128);
            mbar_init(&sc->pv_done[u], 1);
        }
        mbar_init(&sc->drain, 1);
        sc->abort = 0;
        sc->flagged = 0;
        for (int i = 0; i < 4; ++i) sc->fail[i] = 0;
        fence_mbar_init();
    }
    if (tid >= 64 && tid < 192) sc->neg_ref[tid - 64] = kNoKey;
    if (warp == L::kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sc->tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    griddep_wait();
    if (warp == 0) {
        Q8Keys k;
        const Q8Split sp0 = q8_split_of<kQ8Tile>(p, slot_idx, &k);
        if (lane == 0) {
            sc->split = sp0;
            sc->keys = k;
            if (sp0.b >= 0 && sp0.t_begin == 0 && rb == 0) {
                p.part_first[sp0.b * p.Hkv + g] = sp0.first;
                p.part_count[sp0.b * p.Hkv + g] = sp0.count;
            }
        }
    }
    tc_fence_before();   // the allocation, before its address is read
    __syncthreads();
    tc_fence_after();

    const Q8Split sp = sc->split;
    const bool has_work = sp.b >= 0;
    const int b = has_work ? sp.b : 0;
    const int64_t bg = (int64_t)b * p.Hkv + g;
    const Q8Keys keys = sc->keys;
    const int t_begin = sp.t_begin, t_end = sp.t_end;
    const int n = has_work ? t_end - t_begin : 0;
    const int n_page = min(max(keys.page_tiles - t_begin, 0), n);   // the first n_page tiles are pages
    const int64_t tail_keys = keys.tail + p.n_q;
    const uint4* Qg = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(p.Q) +
        (((int64_t)b * p.Hq + (int64_t)g * p.G) * p.n_q + r0) * D);
    const uint32_t tmem = sc->tmem_base;
    // Q in shared memory: K-major, 128-byte swizzle, blocks of 64 dimensions; piece i is 8
    // elements of row i / (D / 8).  Rows past the CTA's are zero.
    auto q_address = [&](int i) -> uint4* {
        const int r = i / (D / 8), j = i - r * (D / 8);
        return reinterpret_cast<uint4*>(smem + L::kOffQ + (j >> 3) * L::kQBlock + r * 128 +
                                        (((j & 7) ^ (r & 7)) << 4));
    };

    const uint32_t sb = opaque(smem_u32(sc));
    auto at = [&](size_t offset, int i = 0) -> uint32_t { return sb + (uint32_t)offset + 8u * (uint32_t)i; };

    if (n <= 0) {
        // nothing to do
    } else if (warp >= L::kProducerWarp) {
        set_regs<L::kLaunchRegs, L::kLastRegs>();
        unsigned failed = 0;                            // code of a wait that gave up
        if (warp == L::kProducerWarp) {
            // ------------------------------ producer --------------------------
            // lane i holds the id of page 32 k + i of the split
            const uint64_t policy = l2_policy_evict_first();
            const bool once = n_rb == 1;                // else the other row blocks read it again
            const int first_page = 2 * t_begin, last_page = keys.pages;
            int id = 0, issued = 0, st = 0;
            uint32_t lap = 0;                           // parity of the ring's current lap
            bool ok = true;
#pragma unroll 1
            for (int i = 0; i < n_page && ok; ++i) {
                if ((i & 15) == 0) {
                    const int j = first_page + 2 * i + lane;
                    id = j < last_page ? q8_page(p, b, j) : 0;
                }
                const int id0 = __shfl_sync(0xffffffffu, id, (2 * i) & 31);
                const int id1 = __shfl_sync(0xffffffffu, id, (2 * i + 1) & 31);
                if (lane == 0) {
                    if (i >= kStages)
                        ok = wait_for(at(offsetof(Scalars, raw_free), st), lap ^ 1u,
                                                kRoleProducer | kBarRawFree | (unsigned)(i & 0xffff), failed);
                    if (*((volatile int*)&sc->abort)) ok = false;
                    if (ok) {
                        uint8_t* dst = smem + L::kOffRaw + st * L::kRawBytes;
                        const bool two = first_page + 2 * i + 1 < last_page;
                        mbar_arrive_expect_tx(&sc->raw_full[st], two ? L::kRawBytes : L::kPageBytes);
                        const int y0 = (id0 * p.Hkv + g) * D, y1 = (id1 * p.Hkv + g) * D;
                        if (once) {
                            tma_load_2d_hint(dst, &pool, 0, y0, &sc->raw_full[st], policy);
                            if (two) tma_load_2d_hint(dst + L::kPageBytes, &pool, 0, y1, &sc->raw_full[st], policy);
                        } else {
                            tma_load_2d(dst, &pool, 0, y0, &sc->raw_full[st]);
                            if (two) tma_load_2d(dst + L::kPageBytes, &pool, 0, y1, &sc->raw_full[st]);
                        }
                        ++issued;
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
                if (++st == kStages) { st = 0; lap ^= 1u; }
            }
            if (!ok && lane == 0) {
                sc->abort = 1;
#pragma unroll 1
                // let the copies still in flight land before the CTA exits
                for (int i = max(0, issued - kStages); i < issued; ++i)
                    mbar_wait(&sc->raw_full[i % kStages], (i / kStages) & 1, p.err,
                              kRoleProducer | kBarRawFull | (unsigned)(i & 0xffff));
            }
        } else if (warp == L::kMmaWarp) {
            // ------------------------------ issuer ----------------------------
            // The whole warp runs the loop, so that addresses and descriptors stay in uniform
            // registers, and one elected lane issues.  The order is fixed, S of tile i + 2
            // (its buffer is free once S of tile i is loaded) before the product of tile i:
            // that is the order in which the inputs come.
            constexpr uint32_t kS16 = idesc(false, false, kN), kSb = idesc(true, false, kN);
            constexpr uint32_t kO16 = idesc(false, true, kN), kOb = idesc(true, true, kN);
            const uint32_t base = smem_u32(smem);
            // warp reductions of values that are the same in every lane, into uniform registers
            const uint32_t tm = __reduce_or_sync(0xffffffffu, tmem);
            const int tiles = __reduce_max_sync(0xffffffffu, n), page_tiles = __reduce_max_sync(0xffffffffu, n_page);
            const uint64_t qd = sdesc(base + L::kOffQ, 16, 1024);
            const uint64_t pd = sdesc(base + L::kOffP, kQ8Tile * 128, 1024);
            const uint32_t leader = elect_one();
            int s16_tiles = 0;                          // tiles whose Q and K are fp16
            auto wait = [&](uint32_t bar, uint32_t par, unsigned code) {
                return __all_sync(0xffffffffu, wait_for(bar, par, kRoleMma | code, failed)) != 0;
            };
            auto scores = [&](int j) -> bool {
                if (!wait(at(offsetof(Scalars, k_full), j % KB), (uint32_t)((j / KB) & 1), kBarK | (unsigned)(j & 0xffff))) return false;
                if (j >= 2 && !wait(at(offsetof(Scalars, s_free), j & 1), (uint32_t)(((j >> 1) - 1) & 1), kBarS | (unsigned)(j & 0xffff)))
                    return false;
                tc_fence_after();
                const uint32_t dS = tm + L::kTmemS + (uint32_t)(j & 1) * L::kNCols;
                const uint32_t aK = tm + L::kTmemK + (uint32_t)(64 * (j % KB));
                const uint32_t id = j < s16_tiles ? kS16 : kSb;
                mma_chain_if<D / 16, 2, L::kQBlock / 16 - 8>(leader, dS, aK, qd, id, 0u);
                mma_commit_if(leader, at(offsetof(Scalars, s_full), j & 1));
                return true;
            };
            bool ok = wait(at(offsetof(Scalars, q_full)), 0, kBarQ);
            if (ok && !__reduce_or_sync(0xffffffffu, (uint32_t)sc->q_wide)) s16_tiles = page_tiles;
            // ... and whose P and V are
            const int o16_tiles = ok && __reduce_or_sync(0xffffffffu, sc->unit < 0.f ? 1u : 0u) ? 0 : page_tiles;
            ok = ok && scores(0);
            if (tiles > 1) ok = ok && scores(1);
#pragma unroll 1
            for (int i = 0; ok && i < tiles; ++i) {
                if (i + 2 < tiles) ok = scores(i + 2);
                // ALT: group i & 1 and its tile i >> 1
                const int pb = ALT ? i & 1 : 0;
                ok = ok && wait(at(offsetof(Scalars, p_full), pb), (uint32_t)((ALT ? i >> 1 : i) & 1), kBarP | (unsigned)(i & 0xffff));
                ok = ok && wait(at(offsetof(Scalars, v_full), i % VB), (uint32_t)((i / VB) & 1), kBarV | (unsigned)(i & 0xffff));
                if (!ok) break;
                tc_fence_after();
                const uint32_t dO = tm + L::kTmemO + (uint32_t)pb * L::kNCols;
                const uint32_t aV = tm + L::kTmemV + (uint32_t)(64 * (i % VB));
                const uint64_t bP = pd + (uint64_t)(pb * (L::kPBuf >> 4));
                const uint32_t id = i < o16_tiles ? kO16 : kOb;
                const uint32_t add = i < (ALT ? 2 : 1) ? 0u : 1u;   // the group's first product starts O^T
                mma_chain_if<kQ8Tile / 16, 128, 0>(leader, dO, aV, bP, id, add);
                mma_commit_if(leader, at(offsetof(Scalars, pv_done), i & 1));
            }
            if (!ok) sc->abort = 1;
            mma_commit_if(leader, at(offsetof(Scalars, drain)));
            wait_for(at(offsetof(Scalars, drain)), 0, kRoleMma | kBarDrain, failed);
        }
        else if (warp == L::kChooserWarp) {
            // ------------------------------ chooser ---------------------------
            // From the softmax warps' maxima and minima: the unit of O^T, the power of two of Q, and
            // whether fp16 holds them.  In a warp of its own, because the same lines at the start
            // of the softmax warps change their loop for the worse (120K chain 49 us).
            asm volatile("barrier.cta.sync 6, %0;" ::"n"(L::kSoftmaxThreads + 32) : "memory");
            const bool on = lane < 4 * L::kGroups;
            const uint32_t top = __reduce_max_sync(0xffffffffu, on ? sc->wmax[lane] : 0u);
            const uint32_t least = __reduce_min_sync(0xffffffffu, on ? sc->wleast[lane] : 0xffffu) + 1;
            const float low = -warp_max(on ? -sc->wlow[lane] : -INFINITY);
            float unit = warp_max(on ? sc->wunit[lane] : 0.f);
            unit = __uint_as_float(__float_as_uint(unit) & 0x7f800000u);
            if (n_page == 0) unit = 1.f;
            else if (low < unit * kLeastRel || !(unit * kMostUnit >= 1.f && unit <= kMostUnit)) unit = -1.f;
            // Q's largest magnitude, 1.f * 2^k, becomes 1.f * 2^14
            const int k = (int)(top >> 7) - 127, k_least = (int)(least >> 7) - 127;
            const bool apart = n_page > 0 && top && (k - k_least > kMostQ || k < kLeastQ);
            if (lane == 0) {
                sc->unit = unit;
                sc->q_wide = apart;
                sc->q_mul = __uint_as_float((uint32_t)(127 + (apart || !top ? 0 : 14 - k)) << 23);
            }
            asm volatile("barrier.cta.arrive 7, %0;" ::"n"(L::kSoftmaxThreads + 32) : "memory");
        }
        if (lane == 0) record(p.err, failed);
    } else if (warp >= L::kConvWarp) {
        // ------------------------------ converters ----------------------------
        set_regs<L::kLaunchRegs, L::kConvRegs>();
        const int t = tid & 127, q4 = t >> 5;
        const bool do_k = warp < L::kConvWarp + 4, do_v = !do_k;
        const uint32_t lanes = tmem + ((uint32_t)(q4 * 32) << 16);
        const __nv_bfloat16* Kh = static_cast<const __nv_bfloat16*>(p.K) + bg * p.cap * D;
        const __nv_bfloat16* Vh = static_cast<const __nv_bfloat16*>(p.V) + bg * p.cap * D;
        // K codes: thread t's key is row t % 64 of page t / 64.  A line of 128 bytes holds
        // 128 / d keys.
        const int k_line = D == 128 ? t & 63 : (t & 63) >> 1;
        const int k_piece = D == 128 ? 0 : 4 * (t & 1);
        const uint32_t k_src = opaque(smem_u32(smem + L::kOffRaw + (t >> 6) * L::kPageBytes + k_line * 128 +
                                               ((k_piece ^ (k_line & 7)) << 4)));
        // V codes: a transposing load takes 32 keys x 16 dimensions, lane l giving the address
        // of key l's 16 bytes; lane l then holds dimensions l / 4 and l / 4 + 8, keys
        // 4 (l % 4) .. + 3 of each half, which as fp16 pairs are the 16x256b tensor-memory layout
        const int v_line = D == 128 ? lane : lane >> 1;               // line of the load's key
        const int v_piece = D == 128 ? 0 : 4 * (lane & 1);
        const uint32_t v_src = opaque(smem_u32(smem + L::kOffRaw + kPageTokens * D + v_line * 128));
        // page ids of the split, and the scales of V of a tile's two pages as fp16 pairs relative
        // to the unit of O^T, 32 tiles at a time like the softmax warps'
        const int32_t* ids = p.page_table + (int64_t)b * p.max_pages + 2 * t_begin;
        const int my_pages = min(keys.pages - 2 * t_begin, 2 * n_page);   // ids[0, my_pages) exist
        float inv_unit = 1.f;
        auto page_ids = [&](int i) -> int2 {
            return make_int2(2 * i < my_pages ? __ldg(ids + 2 * i) : 0,
                             2 * i + 1 < my_pages ? __ldg(ids + 2 * i + 1) : 0);
        };
        auto v_units = [&](int i, int2 id) -> uint2 {                 // 0 where there is no page
            const float x = 2 * i < my_pages ? v_scale(p, id.x, g) * inv_unit : 0.f;
            const float y = 2 * i + 1 < my_pages ? v_scale(p, id.y, g) * inv_unit : 0.f;
            return make_uint2(f16x2(x, x), f16x2(y, y));
        };
        int2 id_next = make_int2(0, 0);
        uint2 unit_now = make_uint2(0, 0), unit_next = make_uint2(0, 0);
        bool ok = true, wide = false;
        unsigned failed = 0;
        if (do_k && n_page > 0) {
            ok = wait_for(at(offsetof(Scalars, q_full)), 0, kRoleConvert | kBarQ, failed);
            wide = ok && sc->q_wide;
        }
        if (do_v && n_page > 0) {
            const int2 id0 = page_ids(lane);
            id_next = page_ids(32 + lane);
            ok = wait_for(at(offsetof(Scalars, q_full)), 0, kRoleConvert | kBarQ, failed);   // the unit is there
            inv_unit = 1.f / sc->unit;
            wide = ok && inv_unit < 0.f;
            unit_now = v_units(lane, id0);
        }
        int st = 0, first = 0;
        uint32_t lap = 0;
        ok = __all_sync(0xffffffffu, ok) != 0;
        if (__builtin_expect(ok && wide, 0)) {
            failed = wide_tiles<D, COLS, ALT>(p, ids, my_pages, g, n_page, do_k, sb, do_k ? k_src : v_src,
                                              (uint32_t)(v_piece + (D == 128 ? 2 * q4 : q4)), lanes);
            ok = __all_sync(0xffffffffu, failed == 0) != 0;
            first = n_page;
            st = n_page % kStages;
            lap = (uint32_t)(n_page / kStages) & 1u;
        }
#pragma unroll 1
        for (int i = first; i < n && ok; ++i) {
            const bool paged = i < n_page;
            const unsigned code = kRoleConvert | (unsigned)(i & 0xffff);
            const int64_t k0 = (int64_t)(t_begin + i - keys.page_tiles) * kQ8Tile;   // tail tile's first row
            if (paged)
                ok = wait_for(at(offsetof(Scalars, raw_full), st), lap, code | kBarRawFull, failed);
            if (do_k) {
                // S of tile i - KB has read this K buffer
                if (ok && i >= KB)
                    ok = wait_for(at(offsetof(Scalars, s_full), (i - KB) & 1), (uint32_t)(((i - KB) >> 1) & 1), code | kBarS, failed);
                if (ok && !paged && i == n_page && i > 0) {
                    // first tail tile after pages: Q becomes bf16 once S of tile i - 1 has read it
                    ok = wait_for(at(offsetof(Scalars, s_full), (i - 1) & 1), (uint32_t)(((i - 1) >> 1) & 1), code | kBarS, failed);
                    if (ok) {
#pragma unroll 1
                        for (int x = t; x < kN * (D / 8); x += 128)
                            *q_address(x) = x < Rb * (D / 8) ? Qg[x] : make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t dst = lanes + L::kTmemK + (uint32_t)(64 * (i % KB));
                if (__builtin_expect(paged, 1)) {
                    const uint32_t line = k_src + (uint32_t)(st * L::kRawBytes);
#pragma unroll 1
                    for (int h = 0; h < D / 64; ++h) {
                        uint4 v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            v[j] = lds_u4(line ^ (uint32_t)((4 * h + j) << 4));
                        uint32_t w[32];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint2 y = e4m3x4_to_f16x4(x[e]);
                                w[8 * j + 2 * e] = y.x;
                                w[8 * j + 2 * e + 1] = y.y;
                            }
                        }
                        tmem_st32(dst + (uint32_t)(32 * h), w);
                    }
                } else {
                    const bool live = k0 + t < tail_keys;
                    const uint4* row = reinterpret_cast<const uint4*>(Kh + (k0 + t) * D);
#pragma unroll 1
                    for (int j = 0; j < D / 16; ++j) {                // 16 elements: 8 columns
                        const uint4 v0 = live ? row[2 * j] : make_uint4(0, 0, 0, 0);
                        const uint4 v1 = live ? row[2 * j + 1] : make_uint4(0, 0, 0, 0);
                        const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
                        tmem_st8(dst + (uint32_t)(8 * j), w);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                arrive(at(offsetof(Scalars, k_full), i % KB));
            }
            if (do_v) {
                const uint32_t unit0 = __shfl_sync(0xffffffffu, unit_now.x, i & 31);   // of the
                const uint32_t unit1 = __shfl_sync(0xffffffffu, unit_now.y, i & 31);   // tile's two pages
                if ((i & 31) == 8) unit_next = v_units(i - 8 + 32 + lane, id_next);
                if ((i & 31) == 31) {
                    unit_now = unit_next;
                    id_next = page_ids(i + 33 + lane);
                }
                // the product of tile i - VB has read this V buffer
                if (ok && i >= VB)
                    ok = wait_for(at(offsetof(Scalars, pv_done), (i - VB) & 1), (uint32_t)(((i - VB) >> 1) & 1), code | kBarPv, failed);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t dst = lanes + L::kTmemV + (uint32_t)(64 * (i % VB));
                if (__builtin_expect(paged, 1)) {
                    const bool two = 2 * i + 1 < my_pages;
                    const uint32_t src = v_src + (uint32_t)(st * L::kRawBytes);
#pragma unroll 1
                    for (int h = 0; h < D / 64; ++h) {
                        // 16 dimensions of the quadrant into 16 of its lanes
                        const uint32_t piece = (uint32_t)(((v_piece + (D == 128 ? 2 * q4 + h : q4)) ^ (v_line & 7)) << 4);
                        uint32_t w[32];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {                 // 32 keys, two loads to a page
                            uint32_t r[4] = {0, 0, 0, 0};             // a page that is not there reads as zeros
                            if (m < 2 || two)
                                ldmatrix_t_b8_x2(src + (uint32_t)((m >> 1) * L::kPageBytes + (m & 1) * 32 * D) + piece, r);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint2 y = e4m3x4_to_f16x4(r[e]);
                                w[8 * m + 2 * e] = mul_f16x2(y.x, m < 2 ? unit0 : unit1);
                                w[8 * m + 2 * e + 1] = mul_f16x2(y.y, m < 2 ? unit0 : unit1);
                            }
                        }
                        tmem_st_16x256b_x8(dst + ((uint32_t)(16 * h) << 16), w);
                    }
                } else {
                    // One dimension to a thread.  Elements that are not finite would turn hidden
                    // keys' zero probabilities into NaN: they are zero here and join the rows
                    // that see them at the end.
                    const int dim = D == 128 ? 32 * q4 + lane : 16 * q4 + lane;
                    const bool mine = D == 128 || lane < 16;
                    const uint16_t* col = reinterpret_cast<const uint16_t*>(Vh) + dim;
#pragma unroll 1
                    for (int j = 0; j < kQ8Tile / 16; ++j) {          // 16 keys: 8 columns
                        uint32_t x[16], w[8];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int64_t key = k0 + 16 * j + e;
                            x[e] = mine && key < tail_keys ? col[key * D] : 0u;
                        }
                        uint32_t odd = 0;
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if ((x[e] & 0x7f80u) == 0x7f80u) { x[e] = 0; odd |= 1u << e; }
#pragma unroll 1
                        for (; odd; odd &= odd - 1) {
                            const int at = atomicAdd(&sc->flagged, 1);
                            if (at < kFlagged) sc->flagged_at[at] = (k0 + 16 * j + __ffs(odd) - 1) * D + dim;
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = x[2 * e] | x[2 * e + 1] << 16;
                        __syncwarp();
                        tmem_st8(dst + (uint32_t)(8 * j), w);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                arrive(at(offsetof(Scalars, v_full), i % VB));
            }
            if (paged) {                                              // this group has read the raw stage
                __syncwarp();
                if (lane == 0) arrive(at(offsetof(Scalars, raw_free), st));
                if (++st == kStages) { st = 0; lap ^= 1u; }
            }
        }
        if (!ok) sc->abort = 1;
        record(p.err, failed);
    } else {
        // ------------------------------ softmax -------------------------------
        set_regs<L::kLaunchRegs, L::kSoftmaxRegs>();
        const int gr = warp >> 2, q4 = warp & 3;
        const int t = tid & 127;                        // this thread's key of every tile
        const int c0 = ALT ? 0 : gr * COLS;             // first row (column of S^T) of the group
        const int first_tile = ALT ? gr : 0;
        constexpr int kStep = ALT ? 2 : 1;              // tiles from one of the group's to its next
        const uint32_t lanes = tmem + ((uint32_t)(q4 * 32) << 16);
        const int64_t slot = ((int64_t)g * p.S + slot_idx) * p.R + r0;   // this CTA's partial rows
        float* my_part = sc->part + warp * L::kPart;
        const float* group_part = sc->part + 4 * gr * L::kPart;
        float* neg_ref = sc->neg_ref + (ALT ? 64 * gr : c0);
        float* corr = sc->corr + (ALT ? 64 * gr : c0);
        const uint32_t refs = opaque(smem_u32(neg_ref));
        // where the thread's key stores P: piece j (8 rows) of the group is 16 bytes, swizzled.
        // A group starts at piece c0 / 8, where COLS / 8 is a power of two that leaves j's bits.
        constexpr bool kPow2 = ALT || (COLS & (COLS - 1)) == 0;
        const uint32_t p_row = opaque(smem_u32(
            smem + L::kOffP + (ALT ? gr * L::kPBuf : 0) + t * 128 +
            (kPow2 ? (c0 >> 6) * (kQ8Tile * 128) + ((((c0 >> 3) & 7) ^ (t & 7)) << 4) : 0)));
        auto p_at = [&](int j) -> uint32_t {
            if (kPow2) return (p_row ^ (uint32_t)((j & 7) << 4)) + (uint32_t)((j >> 3) * (kQ8Tile * 128));
            const int jj = c0 / 8 + j;
            return p_row + (uint32_t)((jj >> 3) * (kQ8Tile * 128) + (((jj & 7) ^ (t & 7)) << 4));
        };
        const uint32_t o_base = lanes + L::kTmemO + (ALT ? (uint32_t)gr * L::kNCols : (uint32_t)c0);
        const int half = t >> 6;

        // Scales of K of this thread's keys, fetched a batch of the group's tiles ahead (the page
        // ids two; the producer flags an id outside the pool).  With four groups a batch is 32
        // tiles, lane l holding the scale of tile l, and a tile's comes by a shuffle: fewer
        // instructions to a tile (70B shape 79 -> 75.5 us, tree 198 -> 188, together with the same
        // for V).  Groups that take tiles in turn fetch one tile at a time (d = 64 at 120K: 41.6 us,
        // with batches of 32 44.3).
        constexpr int kBatch = ALT ? 1 : 32;
        const int32_t* ids = p.page_table + (int64_t)b * p.max_pages + 2 * t_begin;
        const int my_pages = min(keys.pages - 2 * t_begin, 2 * n_page);   // ids[0, my_pages) exist
        auto page_of = [&](int j) -> int { return j < my_pages ? __ldg(ids + j) : 0; };
        auto scale_of = [&](int page) -> float {
            const int id = (unsigned)page < (unsigned)p.n_pages ? page : 0;
            return __ldg(p.scales + ((int64_t)id * p.Hkv + g) * 2);
        };
        // One pass over Q (into shared memory as it is) and over the scales of V: what the CTA's
        // fp16 forms are relative to.  All loads that wait for nothing go out first.
        constexpr int T = L::kSoftmaxThreads;
        constexpr int kQPieces = (kN * (D / 8) + T - 1) / T;
        auto page_idx = [&](int turn) {
            return 2 * (first_tile + kStep * (turn + (kBatch > 1 ? lane : 0))) + half;
        };
        const int page_unit = page_of(tid), page_first = page_of(page_idx(0));
        int page_next = page_of(page_idx(kBatch));
        uint4 qv[kQPieces];
#pragma unroll
        for (int e = 0; e < kQPieces; ++e)
            qv[e] = tid + e * T < Rb * (D / 8) ? Qg[tid + e * T] : make_uint4(0, 0, 0, 0);
        float unit = tid < my_pages ? v_scale(p, page_unit, g) : 0.f;   // largest and smallest
        float scale_now = scale_of(page_first), scale_next = 0.f;
        // largest finite magnitude of Q's pieces (bits order as values), and the least of a piece
        // that is not all 0, less 1
        uint32_t q_bits = 0, q_least = 0xffffu;
#pragma unroll
        for (int e = 0; e < kQPieces; ++e) {
            const uint32_t w[4] = {qv[e].x, qv[e].y, qv[e].z, qv[e].w};
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = w[j] & 0x7fffu, y = w[j] >> 16 & 0x7fffu;
                m = max(m, max(x < 0x7f80u ? x : 0u, y < 0x7f80u ? y : 0u));
            }
            q_bits = max(q_bits, m);
            q_least = min(q_least, m - 1);
        }
        q_bits = __reduce_max_sync(0xffffffffu, q_bits);
        q_least = __reduce_min_sync(0xffffffffu, q_least);
        if (lane == 0) {
            sc->wmax[warp] = (uint16_t)q_bits;
            sc->wleast[warp] = (uint16_t)q_least;
        }
        float low = tid < my_pages ? counted(unit) : INFINITY;
#pragma unroll 1
        for (int j = tid + T; j < my_pages; j += T) {
            const float s = v_scale(p, __ldg(ids + j), g);
            unit = fmaxf(unit, s);
            low = fminf(low, counted(s));
        }
        unit = warp_max(unit);
        low = -warp_max(-low);
        if (lane == 0) {
            sc->wunit[warp] = unit;
            sc->wlow[warp] = low;
        }
        asm volatile("barrier.cta.arrive 6, %0;" ::"n"(T + 32) : "memory");   // to the chooser ...
        asm volatile("barrier.cta.sync 7, %0;" ::"n"(T + 32) : "memory");     // ... and its answer
        unit = sc->unit;
        const float q_mul = sc->q_mul;
        const bool q_wide = sc->q_wide;
#pragma unroll
        for (int e = 0; e < kQPieces; ++e) {
            if (n_page > 0 && !q_wide) {
                uint32_t* w = reinterpret_cast<uint32_t*>(&qv[e]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = f16x2(__uint_as_float(w[j] << 16) * q_mul, __uint_as_float(w[j] & 0xffff0000u) * q_mul);
            }
            if (tid + e * T < kN * (D / 8)) *q_address(tid + e * T) = qv[e];
        }
        fence_proxy_async_smem();
        arrive(at(offsetof(Scalars, q_full)));
        const float a_page = p.scale_log2 * (1.f / q_mul);

        float2 l2[COLS / 2];                            // this thread's part of the rows' sums
#pragma unroll
        for (int c = 0; c < COLS / 2; ++c) l2[c] = make_float2(0.f, 0.f);
        bool fail = false;
        unsigned failed = 0;
#pragma unroll 1
        for (int i = first_tile; i < n; i += kStep) {
            const int u = i & 1;
            const int prev = i - kStep;                 // the product that used this group's P and O^T last
            const bool paged = i < n_page;
            const unsigned code = kRoleSoftmax | (unsigned)(i & 0xffff);
            const int turn = ALT ? i >> 1 : i;          // of the group's tiles
            if (turn % kBatch == 0) {
                scale_next = scale_of(page_next);
                page_next = page_of(page_idx(turn + 2 * kBatch));
            }
            // which of the rows see this thread's key
            uint64_t seen;
            float a;                                    // s = a * S^T
            if (__builtin_expect(paged, 1)) {
                seen = 2 * i + half < my_pages ? ~0ull : 0ull;
                a = (kBatch > 1 ? __shfl_sync(0xffffffffu, scale_now, turn % kBatch) : scale_now) * a_page;
            } else {
                const int64_t key = (int64_t)(t_begin + i - keys.page_tiles) * kQ8Tile + t;
                const int64_t node = key - keys.tail;
                seen = key < tail_keys ? ~0ull : 0ull;
                if (node >= 0 && key < tail_keys) {
                    seen = 0;
                    const uint8_t* column = p.mask ? p.mask + (int64_t)b * p.n_q * p.n_q + node : nullptr;
                    int iq = (r0 + c0) % p.n_q;         // of the group row
#pragma unroll 8
                    for (int c = 0; c < COLS; ++c) {    // loads of several rows in flight
                        const bool vis = column ? __ldg(column + iq * p.n_q) != 0 : node <= iq;
                        seen |= (vis ? 1ull : 0ull) << c;
                        if (++iq == p.n_q) iq = 0;
                    }
                }
                a = p.scale_log2;
            }
            fail |= !wait_for(at(offsetof(Scalars, s_full), u), (uint32_t)((i >> 1) & 1), code | kBarS, failed);
            tc_fence_after();
            float2 x[COLS / 2];
            const uint32_t s_addr = lanes + L::kTmemS + (uint32_t)u * L::kNCols + (uint32_t)c0;
            bool quit = false;                          // a wait failed in the group
#pragma unroll 1
            for (int pass = 0;; ++pass) {
                uint32_t r[COLS];
#pragma unroll
                for (int ch = 0; ch < COLS; ch += 8) tmem_ld8(s_addr + ch, reinterpret_cast<uint32_t(&)[8]>(r[ch]));
                tmem_wait_ld();
                const float2 aa = make_float2(a, a);
#pragma unroll
                for (int c = 0; c < COLS; c += 4) {
                    const float4 nr = lds_f4(refs + 4 * c);
                    x[c / 2] = fma2(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), aa, make_float2(nr.x, nr.y));
                    x[c / 2 + 1] = fma2(make_float2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])), aa, make_float2(nr.z, nr.w));
                }
                if (__builtin_expect(seen != ~0ull, 0)) {
                    uint64_t bits = seen;
#pragma unroll
                    for (int c = 0; c < COLS / 2; ++c) {
                        if (!(bits & 1ull)) x[c].x = -INFINITY;
                        if (!(bits & 2ull)) x[c].y = -INFINITY;
                        bits >>= 2;
                    }
                }
                float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
                for (int c = 0; c < COLS / 2; c += 2) {
                    top0 = fmax3(top0, x[c].x, x[c].y);
                    top1 = fmax3(top1, x[c + 1].x, x[c + 1].y);
                }
                const bool over = fmaxf(top0, top1) > kMaxLog2P;   // some score passed its reference by too much
                if (fail) sc->fail[gr] = 1;
                if (__builtin_expect(!group_any(gr, over || fail), 1)) break;
                if (pass > 0) {
                    // scores past 2^26, whose own rounding is that coarse: hold them at the limit
#pragma unroll
                    for (int c = 0; c < COLS / 2; ++c) {
                        x[c].x = x[c].x > kMaxLog2P ? kMaxLog2P : x[c].x;
                        x[c].y = x[c].y > kMaxLog2P ? kMaxLog2P : x[c].y;
                    }
                    break;
                }
                // set before the barrier above, and again at the earliest after the ones below:
                // the whole group reads the same
                quit = *((volatile int*)&sc->fail[gr]) != 0;
                if (quit) break;
                // ---- the references of the rows that need it move; then S^T is taken again ----
                uint64_t bits = seen;
#pragma unroll 2
                for (int ch = 0; ch < COLS / 8; ++ch) {
                    uint32_t r[8];
                    tmem_ld8(s_addr + 8 * ch, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float m = warp_max_redux((bits & 1ull) ? __uint_as_float(r[c]) * a : -INFINITY);
                        if (lane == 0) my_part[8 * ch + c] = m;
                        bits >>= 1;
                    }
                }
                group_sync(gr);
                if (t < COLS) {
                    const float* m4 = group_part + t;
                    const float m = fmaxf(fmaxf(m4[0], m4[L::kPart]), fmaxf(m4[2 * L::kPart], m4[3 * L::kPart]));
                    const float old = neg_ref[t];
                    float f = 1.f;
                    if (m + old > kMaxLog2P) {
                        neg_ref[t] = kRefShift - m;
                        f = ex2(kRefShift - m - old);   // 0 for the first key of the row
                    }
                    corr[t] = f;
                }
                group_sync(gr);
                if (prev >= 0) {
                    fail |= !wait_for(at(offsetof(Scalars, pv_done), prev & 1), (uint32_t)((prev >> 1) & 1), code | kBarPv, failed);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int ch = 0; ch < COLS / 8; ++ch) {
                        uint32_t o[8];
                        const uint32_t o_addr = o_base + (uint32_t)(8 * ch);
                        tmem_ld8(o_addr, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            o[c] = __float_as_uint(__uint_as_float(o[c]) * corr[8 * ch + c]);
                        tmem_st8(o_addr, o);
                    }
                    tmem_wait_st();
#pragma unroll
                    for (int c = 0; c < COLS; c += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(corr + c);
                        l2[c / 2] = mul2(l2[c / 2], make_float2(f.x, f.y));
                        l2[c / 2 + 1] = mul2(l2[c / 2 + 1], make_float2(f.z, f.w));
                    }
                }
            }
            if (quit) {
                fail = true;
                break;
            }
            // S^T is in registers: the buffer is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(at(offsetof(Scalars, s_free), u));
            uint32_t pk[COLS / 2];
            if (__builtin_expect(paged && unit > 0.f, 1)) {
#pragma unroll
                for (int c = 0; c < COLS / 2; ++c) {
                    const float2 e = make_float2(ex2(x[c].x), ex2(x[c].y));
                    l2[c] = add2(l2[c], e);
                    pk[c] = f16x2(e.x, e.y);
                }
            } else {
                const float v1 = 1.f / fabsf(unit);     // V as it is: P takes the unit
                const float2 vm = make_float2(v1, v1);
#pragma unroll
                for (int c = 0; c < COLS / 2; ++c) {
                    const float2 e = make_float2(ex2(x[c].x), ex2(x[c].y));
                    l2[c] = add2(l2[c], e);
                    const float2 w = mul2(e, vm);
                    pk[c] = bf16x2(w.x, w.y);
                }
            }
            // P's buffer is free once the previous product has read it
            if (prev >= 0)
                fail |= !wait_for(at(offsetof(Scalars, pv_done), prev & 1), (uint32_t)((prev >> 1) & 1), code | kBarPv, failed);
            if (!fail) {
#pragma unroll
                for (int j = 0; j < COLS / 8; ++j)
                    sts_u4(p_at(j), make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]));
                fence_proxy_async_smem();
                tc_fence_before();
                arrive(at(offsetof(Scalars, p_full), ALT ? gr : 0));
            }
            __syncwarp();
            if (turn % kBatch == kBatch - 1) scale_now = scale_next;
        }
        if (tid == 0) griddep_launch_dependents();
        // the rows' sums over this warp's keys
#pragma unroll
        for (int c = 0; c < COLS; c += 8) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) { v[2 * e] = l2[c / 2 + e].x; v[2 * e + 1] = l2[c / 2 + e].y; }
            const float s = warp_sum8(v, lane);
            if ((lane & 3) == 0) my_part[c + (lane >> 2)] = s;
        }
        // O^T of the last products (in ALT of both groups)
        for (int i = max(n - kStep, 0); i < n; ++i)
            fail |= !wait_for(at(offsetof(Scalars, pv_done), i & 1), (uint32_t)((i >> 1) & 1), kRoleSoftmax | kBarPv | 0xffffu, failed);
        record(p.err, failed);
        if (barrier_any<L::kSoftmaxThreads>(5, fail)) { // sums and references of all groups are there
            sc->abort = 1;
        } else {
            tc_fence_after();
            const int dim = D == 128 ? 32 * q4 + lane : 16 * q4 + lane;
            const bool mine = D == 128 || lane < 16;
            auto row_sum = [&](int group, int r) {
                const float* s = sc->part + 4 * group * L::kPart + r;
                return (s[0] + s[L::kPart]) + (s[2 * L::kPart] + s[3 * L::kPart]);
            };
            if constexpr (ALT) {
                // Weights of the two groups' parts of a row; this group writes half of the rows.
                // A group that took no tile has nothing in O^T.
                constexpr int kHalf = COLS / 2;
                if (t < kHalf) {
                    const int r = gr * kHalf + t;
                    const float s0 = row_sum(0, r), s1 = row_sum(1, r);
                    const float m0 = -sc->neg_ref[r], m1 = -sc->neg_ref[64 + r];
                    const float m = fmaxf(s0 != 0.f ? m0 : -kNoKey, s1 != 0.f ? m1 : -kNoKey);
                    const float w0 = s0 != 0.f ? ex2(m0 - m) : 0.f, w1 = s1 != 0.f ? ex2(m1 - m) : 0.f;
                    const float s = s0 * w0 + s1 * w1;
                    sc->corr[r] = w0 * fabsf(unit);
                    sc->corr[64 + r] = w1 * fabsf(unit);
                    if (r < Rb)
                        *reinterpret_cast<float2*>(p.part_ml + (slot + r) * 2) =
                            make_float2(m == -kNoKey && s == 0.f ? -INFINITY : m, s);
                }
                group_sync(gr);
                float* dst = p.part_acc + (slot + gr * kHalf) * D + dim;
#pragma unroll 1
                for (int ch = 0; ch < kHalf / 8; ++ch, dst += 8 * D) {
                    uint32_t o0[8], o1[8];
                    const int base = gr * kHalf + 8 * ch;
                    tmem_ld8(lanes + L::kTmemO + (uint32_t)base, o0);
                    tmem_ld8(lanes + L::kTmemO + L::kNCols + (uint32_t)base, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int r = base + c;
                        const float w0 = sc->corr[r], w1 = sc->corr[64 + r];
                        const float y = __uint_as_float(o0[c]) * w0 + (n > 1 ? __uint_as_float(o1[c]) * w1 : 0.f);
                        if (mine && r < Rb) dst[c * D] = y;
                    }
                }
            } else {
                if (t < COLS && c0 + t < Rb) {
                    const float s = row_sum(gr, t), nr = neg_ref[t];
                    *reinterpret_cast<float2*>(p.part_ml + (slot + c0 + t) * 2) =
                        nr == kNoKey && s == 0.f ? make_float2(-INFINITY, 0.f) : make_float2(-nr, s);
                }
                float* dst = p.part_acc + (slot + c0) * D + dim;
#pragma unroll 1
                for (int ch = 0; ch < COLS / 8; ++ch, dst += 8 * D) {
                    uint32_t o[8];
                    tmem_ld8(o_base + (uint32_t)(8 * ch), o);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (mine && c0 + 8 * ch + c < Rb) dst[c * D] = __uint_as_float(o[c]) * fabsf(unit);
                }
            }
            const int flagged = sc->flagged;
            if (flagged > 0 && mine) {
                // V elements left out of the products reach the rows that see them
                const __nv_bfloat16* Vh = static_cast<const __nv_bfloat16*>(p.V) + bg * p.cap * D;
                const int64_t first = (int64_t)max(t_begin - keys.page_tiles, 0) * kQ8Tile;
                const int64_t last = min((int64_t)(t_end - keys.page_tiles) * kQ8Tile, tail_keys);
                const bool listed = flagged <= kFlagged;
                const int64_t m = listed ? flagged : last - first;
#pragma unroll 1
                for (int64_t f = 0; f < m; ++f) {
                    int64_t key = first + f;
                    if (listed) {
                        key = sc->flagged_at[f] / D;
                        if (sc->flagged_at[f] % D != dim) continue;
                    }
                    const float v = __bfloat162float(Vh[key * D + dim]);
                    if (fabsf(v) < INFINITY) continue;
                    const int64_t node = key - keys.tail;
#pragma unroll 1
                    for (int r = ALT ? gr * (COLS / 2) : c0; r < min(ALT ? (gr + 1) * (COLS / 2) : c0 + COLS, Rb); ++r) {
                        const int iq = (r0 + r) % p.n_q;
                        if (node < 0 || (p.mask ? p.mask[((int64_t)b * p.n_q + iq) * p.n_q + node] != 0
                                                : node <= iq))
                            p.part_acc[(slot + r) * D + dim] += v;
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == L::kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                     : "memory");
    }
}

// The pool as rows of 128 bytes; a page and head (K, then V) is d of them.
bool make_pool_map(CUtensorMap* m, const AttnQ8Params& p) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {128, (cuuint64_t)p.n_pages * p.Hkv * p.d};
    cuuint64_t strides[1] = {128};
    cuuint32_t box[2] = {128, (cuuint32_t)p.d};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p.pages), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int COLS, bool ALT>
cudaError_t launch_shape(const CUtensorMap& pool, const AttnQ8Params& p, int n_rb, int rows, cudaStream_t st) {
    using L = Plan<D, COLS, ALT>;
    auto kern = attn_q8_tc_kernel<D, COLS, ALT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.S * n_rb, p.Hkv, 1);
    cfg.blockDim = dim3(L::kThreads, 1, 1);
    cfg.dynamicSmemBytes = L::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, pool, p, n_rb, rows);
}

// N in steps of 16 as far as two groups that take the tiles in turn hold all rows, above it
// four groups with a quarter of the rows each, N in steps of 32.  Measured at 120K (us): 44 rows
// of 8 heads, in turn 45.9, four groups 59.5; 56 rows of 4 heads, in turn 43.8, four groups 40.6
// (38.1 since); 88 rows of 8 heads, N = 96 75.4, N = 128 86.4.  4 rows over 4K: N = 16 8.4, N = 48
// in turn 11.3, four groups 10.2.
template <int D>
cudaError_t launch_rows(const CUtensorMap& pool, const AttnQ8Params& p, cudaStream_t st) {
    const int n_rb = q8_row_blocks(p.R);
    const int rows = (p.R + n_rb - 1) / n_rb;
    if (rows <= 16) return launch_shape<D, 16, true>(pool, p, n_rb, rows, st);
    if (rows <= 32) return launch_shape<D, 32, true>(pool, p, n_rb, rows, st);
    if (rows <= 48) return launch_shape<D, 48, true>(pool, p, n_rb, rows, st);
    if (rows <= 64) return launch_shape<D, 16, false>(pool, p, n_rb, rows, st);
    if (rows <= 96) return launch_shape<D, 24, false>(pool, p, n_rb, rows, st);
    return launch_shape<D, 32, false>(pool, p, n_rb, rows, st);
}

}  // namespace

cudaError_t launch_attn_q8_tc(const AttnQ8Params& p, cudaStream_t st) {
    CUtensorMap pool;
    if (!make_pool_map(&pool, p)) return cudaErrorInvalidValue;
    return p.d == 128 ? launch_rows<128>(pool, p, st) : launch_rows<64>(pool, p, st);
}

}  // namespace rapid
