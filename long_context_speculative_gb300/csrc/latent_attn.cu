// Absorbed attention over a latent cache on tensor cores: verify attention whose keys are the
// cache rows (576 values, one row for all heads) and whose values are their first 512.
//
//   s_j = <q, [c_j, r_j]>,   O = sum_j softmax(scale s)_j c_j
//
// over the history rows and, as the chain or tree mask says, the n_q rows behind them.
//
// All H * n_q queries of a sequence share the rows, so one tile of rows in shared memory is read
// as both operands: by QK as K (64 keys x 576, K-major), by PV as V (64 keys x 512, MN-major).
// The accumulator is what decides the shape: 512 fp32 values for each query fill tensor memory
// at 128 queries, with no room for S.  So a CTA takes at most 64 queries, and forms
//   S[row, key]   = Q K^T           M = 64, N = 64, K = 576
//   O^T[dim, row] += V^T P^T        4 x (M = 128, N = rows, K = 64)
// the second product transposed: rows in N cost what they are (16, 32 or 64 of them), rows in M
// would leave half of the tensor unit's lanes idle.
//
// CTA = (sequence and split of its keys, block of rows).  Shared memory holds Q, two tiles of
// 64 keys and one P tile; a tile's room is refilled in five pieces (the key's 64 rotated values,
// then 128 values at a time) as soon as the products that read a piece are done, so copies run
// beside the products of the same tile.  Warps:
//   0-3    softmax: warp w has rows 16 w .. 16 w + 15 of S, and dimensions 32 w .. 32 w + 31 of
//          each 128 of O^T.  The running maximum moves only when a score passes it by more than
//          2^16 (the warps vote on a barrier); O^T is rescaled then
//   4      copies by TMA: Q; tiles of bf16 rows, the rotated part of 8-bit rows
//   5, 6   issue QK and PV
//   7-14   (8-bit rows) convert codes on their way from global memory to the tile: a thread has a
//          quarter of a key, and the next tile's are loaded once this one is stored.  A value is
//          code * scale in fp32, rounded to bf16, what rapid_latent_read gives: any scale will
//          do, and a NaN code is NaN
// P is rounded to bf16 (at most 2^-8 of each probability, and it averages out); sums are fp32.
//
// Rows that a query does not see have no effect on it, whatever they hold: in tiles that a mask
// touches, rows behind the step are zeroed in shared memory before they are read as values, and
// so are rows with a value that is not finite, whose probabilities become NaN where they are seen.
//
// Every wait is bounded in wall-clock time; after a failed wait the kernel records an error code,
// stops issuing, drains and returns.
//
// Measured with the join, calls back to back over inputs that do not stay in L2, SM clock 2070 MHz (us; floor
// by bytes at 6788 GB/s or operations at 1910 TFLOP/s): 128 heads, 11 queries over 120K bf16 rows 386 (197);
// 128 heads, 1 query over 120K 8-bit rows 55 (18), bf16 50 (21); 16 heads, a tree of 32 over four 8-bit
// histories of 32K to 96K 380 (153); 16 heads, 1 query over 120K bf16 rows 34 (21), over 1K 9.4 (0.2); 64
// sequences of 4K with 1 query of 16 heads 76 (45), 8 bits 74 (26), of 128 heads 122 (47), 8 bits 137 (38).
// With 64 rows the operands' reads from shared memory
// bound the products (128 B a clock: 36.7 clocks for M = N = 64, 52 for M = 128, N = 64, so 2153 a
// tile; a tile takes 2340, and sharing the copies of two row blocks in a cluster changes nothing).
// 8-bit rows take some 3300 clocks: the converters share issue slots and the shared-memory port with the softmax
// warps (16 converter warps are slower than 8, 68 us against 64 then).  One query of 16 heads takes
// 3650 a tile, 5.9 TB/s; of a short call, the start (lengths, first copies), the end and the join are
// 8 us.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "latent.cuh"
#include "tcgen05.cuh"

namespace rapid {

namespace {

constexpr int kKeys = 64;                        // keys of a tile
constexpr int kChunk = kKeys * 128;              // 64 values of a tile's keys: 8 KB
constexpr int kChunks = kLatentRow / 64;         // 9; the last is the rotated part
constexpr int kTile = kChunks * kChunk;
constexpr int kPieces = 5;                       // of a tile: rotated part, then 2 chunks at a time
constexpr int kProducerWarp = 4, kQkWarp = 5, kPvWarp = 6, kConvWarp = 7, kConvWarps = 8;
constexpr int kBarBytes = 1536;
// A row's reference (what its exponents are relative to) follows its maximum only when a score passes
// it by more than 2^kRise: P and the sums have fp32's exponents, and relative precision.
constexpr float kRise = 16.f;

template <int NR, bool Q8>
struct Plan {
    static constexpr int kThreads = 32 * (Q8 ? kConvWarp + kConvWarps : kPvWarp + 1);
    static constexpr int kQChunk = NR * 128;
    static constexpr int kOffQ = 0;
    static constexpr int kOffTile = kChunks * kQChunk;
    static constexpr int kOffP = kOffTile + 2 * kTile;
    static constexpr int kOffBar = kOffP + NR * 128;
    static constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;   // + alignment
    // tensor-memory columns: O^T (4 blocks of NR), two S buffers
    static constexpr uint32_t kTmemO = 0, kTmemS = 4 * NR;
    static constexpr uint32_t kTmemCols = 4 * NR + 2 * kKeys <= 256 ? 256 : 512;
    static constexpr uint32_t kIdescPV = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) |
                                         ((uint32_t)(NR >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
    static_assert(kSmemBytes <= 232448, "shared memory budget");
};
constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kKeys >> 3) << 17) |
                             ((uint32_t)(64 >> 4) << 24);

// Codes recorded by a timed-out wait: role << 24 | barrier << 16 | tile.
enum : unsigned int {
    kRoleProducer = 0x21u << 24, kRoleMma = 0x22u << 24, kRoleSoftmax = 0x23u << 24,
    kRoleConvert = 0x24u << 24,
    kBarFull = 1u << 16, kBarEmpty = 2u << 16, kBarS = 3u << 16, kBarPV = 4u << 16, kBarLast = 5u << 16
};

struct Slot {
    int b, s, S_b;           // sequence (-1: no work), split, splits of the sequence
    int t_begin, n;          // tiles of the split
    int P;                   // history of the sequence, clamped
};

struct Bars {
    uint64_t full[2][kPieces], empty[2][kPieces];
    uint64_t q_full, s_full[2], s_free[2], p_full, pv_done, drain[2];
    uint32_t tmem_base;
    int abort;
    Slot slot;
    uint32_t flagged[2];     // keys of a masked tile with a value that is not finite
    float factor[64];        // rescale factors of the rows, later 1 / sum
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block too small");

RAPID_DEVICE float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
RAPID_DEVICE uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
RAPID_DEVICE uint32_t times_zero(uint32_t x, uint32_t acc) {       // bf16 pairs: x * 0 + acc
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    return r;
}
// Two codes as floats.
RAPID_DEVICE float2 e4m3x2(uint16_t x) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(x, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
RAPID_DEVICE void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
RAPID_DEVICE void tma_load_3d(void* dst, const CUtensorMap* tm, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(tm), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
RAPID_DEVICE void tma_load_4d(void* dst, const CUtensorMap* tm, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(tm), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}
// 16 lanes x 64 columns -> 32 registers: 4 c .. 4 c + 3 of lane l are columns 8 c + 2 (l % 4), + 1
// of row l / 4, then of row l / 4 + 8.
RAPID_DEVICE void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// Barrier 1 of the four softmax warps: whether any thread says so.
RAPID_DEVICE bool softmax_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred.aligned q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

RAPID_DEVICE int clamped_len(const LatentAttnParams& p, int len) {
    return max(0, min(len, (int)p.cap - p.n_q));
}

// Which sequence and split a slot holds, worked out by one warp from the lengths: the least
// number of tiles a split for which all splits fit into the p.S slots.  (Tiles of all sequences are
// counted in 32 bits: B * cap / 64 stays below 2^31.)
RAPID_DEVICE Slot find_slot(const LatentAttnParams& p, int c, int lane) {
    if (p.S == p.B) {                             // one split each
        const int len = p.prefix_len[c], P = clamped_len(p, len);
        if (lane == 0 && p.err && len != P) atomicOr(p.err, kErrBadInput);
        return Slot{c, 0, 1, 0, (P + p.n_q + kKeys - 1) / kKeys, P};
    }
    // the first 32 sequences' tiles are kept in a register
    const int len0 = lane < p.B ? p.prefix_len[lane] : 0;
    const int mine = lane < p.B ? (clamped_len(p, len0) + p.n_q + kKeys - 1) / kKeys : 0;
    auto tiles_of = [&](int b) {
        return b < 32 ? mine : (clamped_len(p, p.prefix_len[b]) + p.n_q + kKeys - 1) / kKeys;
    };
    int total = 0, longest = 1;
    for (int b = lane; b < p.B; b += 32) {
        const int t = tiles_of(b);
        total += t;
        longest = max(longest, t);
    }
    total = __reduce_add_sync(0xffffffffu, total);
    longest = __reduce_max_sync(0xffffffffu, longest);
    int lo = (total + p.S - 1) / p.S, hi = max(lo, longest);
    if (p.B == 1) hi = lo;
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        int used = 0;
        for (int b = lane; b < p.B; b += 32) used += (tiles_of(b) + mid - 1) / mid;
        if (__reduce_add_sync(0xffffffffu, used) <= p.S) hi = mid; else lo = mid + 1;
    }
    int first = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        const int tiles = b < p.B ? tiles_of(b) : 0;
        const int S_b = (tiles + lo - 1) / lo;
        int upto = S_b;                           // inclusive scan
        if (p.B > 1) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
        }
        const uint32_t here = __ballot_sync(0xffffffffu, b < p.B && c < first + upto);
        if (here) {
            const int l = __ffs(here) - 1;
            Slot r;                               // (lane l's are the ones that count)
            r.b = b;
            r.S_b = S_b;
            r.s = c - first - (upto - S_b);
            r.t_begin = (int)((int64_t)r.s * tiles / max(S_b, 1));
            r.n = (int)((int64_t)(r.s + 1) * tiles / max(S_b, 1)) - r.t_begin;
            const int len = b < 32 ? len0 : p.prefix_len[b < p.B ? b : 0];
            r.P = clamped_len(p, len);
            if (lane == l && r.s == 0 && p.err && len != r.P) atomicOr(p.err, kErrBadInput);
            r.b = __shfl_sync(0xffffffffu, r.b, l);
            r.S_b = __shfl_sync(0xffffffffu, r.S_b, l);
            r.s = __shfl_sync(0xffffffffu, r.s, l);
            r.t_begin = __shfl_sync(0xffffffffu, r.t_begin, l);
            r.n = __shfl_sync(0xffffffffu, r.n, l);
            r.P = __shfl_sync(0xffffffffu, r.P, l);
            return r;
        }
        first += __shfl_sync(0xffffffffu, upto, 31);
    }
    return Slot{-1, 0, 1, 0, 0, 0};
}

template <int NR, bool Q8>
__global__ void __launch_bounds__(Plan<NR, Q8>::kThreads, 1)
latent_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmC,
                   const __grid_constant__ CUtensorMap tmR, const LatentAttnParams p) {
    using L = Plan<NR, Q8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Bars* bars = reinterpret_cast<Bars*>(smem + L::kOffBar);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    // Row blocks of one split are neighbours: they read the same tiles at the same time, once
    // from memory and then from L2.
    const int slot_idx = blockIdx.x / p.RB, rb = blockIdx.x - slot_idx * p.RB;
    const int R = p.H * p.n_q;
    const int r0 = rb * NR, Rb = min(NR, R - r0);
    if (tid == 0) {
        for (int u = 0; u < 2; ++u) {
            for (int g = 0; g < kPieces; ++g) {
                mbar_init(&bars->full[u][g], Q8 && g > 0 ? kConvWarps : 1);
                mbar_init(&bars->empty[u][g], 1);
            }
            mbar_init(&bars->s_full[u], 1);
            mbar_init(&bars->drain[u], 1);
            mbar_init(&bars->s_free[u], 4);
            bars->flagged[u] = 0;
        }
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->p_full, 4);
        mbar_init(&bars->pv_done, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == kQkWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&bars->tmem_base)),
                     "r"(L::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    griddep_wait();
    if (warp == 0) {
        const Slot sl = find_slot(p, slot_idx, lane);
        if (lane == 0) {
            bars->slot = sl;
            if (sl.b >= 0 && sl.s == 0 && rb == 0) {
                p.part_first[sl.b] = slot_idx;
                p.part_count[sl.b] = sl.S_b;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Slot sl = bars->slot;
    const int b = sl.b, t_begin = sl.t_begin, n = sl.n;
    const int64_t P = sl.P;
    const uint32_t tmem = bars->tmem_base;

    if (n <= 0) {
        // a slot that no split needs
    } else if (warp < 4) {
        // ------------------------------ softmax -------------------------------
        const bool rows_here = 16 * warp < NR;
        const int ra = 16 * warp + (lane >> 2), q4 = lane & 3;
        const bool live[2] = {rows_here && ra < Rb, rows_here && ra + 8 < Rb};
        uint64_t spec[2] = {0, 0};                // the step's rows that each row sees
        if ((int64_t)(t_begin + n) * kKeys > P) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = (r0 + ra + 8 * k) % p.n_q;
                if (!p.mask) {
                    spec[k] = (2ull << i) - 1;
                } else {
                    const uint8_t* m = p.mask + ((int64_t)b * p.n_q + i) * p.n_q;
                    for (int j = 16 * q4; j < min(16 * q4 + 16, p.n_q); ++j)
                        if (live[k] && m[j]) spec[k] |= 1ull << j;
                    spec[k] |= __shfl_xor_sync(0xffffffffu, spec[k], 1);
                    spec[k] |= __shfl_xor_sync(0xffffffffu, spec[k], 2);
                }
            }
        }
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * warp) << 16);
        const float c = p.scale_log2;
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
        bool dead = false;
        for (int j = 0; j < n; ++j) {
            const int buf = j & 1;
            if (!dead)
                dead = !__all_sync(0xffffffffu, mbar_wait_sleep(&bars->s_full[buf], (uint32_t)((j >> 1) & 1), p.err,
                                                          kRoleSoftmax | kBarS | (unsigned)(j & 0xffff)));
            uint32_t sr[32];
            float top[2];
            const int64_t base = (int64_t)(t_begin + j) * kKeys;
            const bool masked = base + kKeys > P;
            if (!dead) {
                tc_fence_after();
                if (rows_here) {
                    tmem_ld_16x256b_x8(lane_addr + L::kTmemS + (uint32_t)(buf * kKeys), sr);
                    tmem_wait_ld();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->s_free[buf]);
            }
            if (masked) {
                // The tile as values: two threads a key, 4 chunks each, 16-byte units in an order without
                // bank conflicts.  Only rows of the step can be hidden from some queries and seen by others.
                uint8_t* tile = smem + L::kOffTile + buf * kTile;
                const int key = tid >> 1, turn = key ^ ((tid & 1) << 2);
                uint8_t* mine = tile + 4 * (tid & 1) * kChunk + key * 128;
                const bool inside = base + key < P + p.n_q;
                uint64_t flagged = 0;
                if (!dead)                            // done long ago: what was copied is visible here
                    for (int g = 0; g < kPieces; ++g)
                        mbar_wait(&bars->full[buf][g], (uint32_t)((j >> 1) & 1), p.err, kRoleSoftmax | kBarFull);
                if (p.mask || p.n_q > 1) {
                    bool odd = false;
                    if (inside && base + key >= P && !dead) {
                        uint32_t acc[4] = {0, 0, 0, 0};       // value * 0 is NaN where it is not finite
#pragma unroll 8
                        for (int x = 0; x < 32; ++x) {
                            const uint4 v = *reinterpret_cast<const uint4*>(mine + (x >> 3) * kChunk + (((x ^ turn) & 7) << 4));
                            acc[0] = times_zero(v.x, acc[0]); acc[1] = times_zero(v.y, acc[1]);
                            acc[2] = times_zero(v.z, acc[2]); acc[3] = times_zero(v.w, acc[3]);
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            odd |= (acc[u] & 0x7fffu) > 0x7f80u || (acc[u] & 0x7fff0000u) > 0x7f800000u;
                    }
                    if (odd) atomicOr(&bars->flagged[key >> 5], 1u << (key & 31));
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    flagged = bars->flagged[0] | ((uint64_t)bars->flagged[1] << 32);
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    if (tid < 2) bars->flagged[tid] = 0;      // (set again only after the vote below)
                }
                if (!dead && (!inside || ((flagged >> key) & 1))) {
#pragma unroll 8
                    for (int x = 0; x < 32; ++x)
                        *reinterpret_cast<uint4*>(mine + (x >> 3) * kChunk + (((x ^ turn) & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                if (!dead && rows_here) {
                    const int64_t delta = P - base;       // < 64
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint64_t see = delta > 0 ? ((1ull << delta) - 1) | (spec[k] << delta)
                                                 : delta > -64 ? spec[k] >> -delta : 0;
                        if (!live[k]) see = 0;
                        const uint64_t here = see >> (2 * q4), odd = (flagged & see) >> (2 * q4);
#pragma unroll
                        for (int x = 0; x < 8; ++x)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t& s = sr[4 * x + 2 * k + e];
                                if (!((here >> (8 * x + e)) & 1)) s = 0xff800000u;          // -inf
                                if ((odd >> (8 * x + e)) & 1) s = 0x7fffffffu;              // NaN
                            }
                    }
                }
            }
            // Most tiles leave every reference alone: no lane's scores pass it by more than kRise.
            bool rises = false;
            if (!dead && rows_here) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        mx = fmaxf(mx, fmaxf(__uint_as_float(sr[4 * x + 2 * k]), __uint_as_float(sr[4 * x + 2 * k + 1])));
                    top[k] = mx * c;
                    rises |= live[k] && top[k] > m_run[k] + kRise;     // the first finite score too
                }
            }
            // (also keeps the warps within a tile of each other)
            if (softmax_any(rises || dead)) {
                if (!dead && rows_here) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float mx = top[k], fac = 1.f;
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        if (live[k] && mx > m_run[k] + kRise) {
                            fac = ex2(m_run[k] - mx);         // 0 where m_run is -inf
                            m_run[k] = mx;
                            l_run[k] *= fac;
                        }
                        if (q4 == 0) bars->factor[ra + 8 * k] = fac;
                    }
                }
                if (softmax_any(dead)) { dead = true; break; }
                // O^T is rescaled: after the product that last added to it
                if (j > 0) {
                    dead = !__all_sync(0xffffffffu, mbar_wait_sleep(&bars->pv_done, (uint32_t)((j - 1) & 1), p.err,
                                                              kRoleSoftmax | kBarPV | (unsigned)(j & 0xffff)));
                    if (!dead) {
                        tc_fence_after();
#pragma unroll 1
                        for (int x = 0; x < NR / 4; ++x) {    // 16 columns at a time
                            uint32_t o[16];
                            tmem_ld16(lane_addr + L::kTmemO + (uint32_t)(16 * x), o);
                            tmem_wait_ld();
                            const float* f = bars->factor + (16 * x) % NR;
#pragma unroll
                            for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f[u]);
                            tmem_st16(lane_addr + L::kTmemO + (uint32_t)(16 * x), o);
                        }
                        tmem_wait_st();
                    }
                }
                // the factors are written again no sooner than this
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            // (looked at before the exponentials, waited for behind them)
            const bool free = j == 0 || mbar_try_wait(&bars->pv_done, (uint32_t)((j - 1) & 1));
            uint32_t pk[16];
            if (!dead && rows_here) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float neg = m_run[k] == -INFINITY ? 0.f : -m_run[k];
                    const float2 c2 = make_float2(c, c), n2 = make_float2(neg, neg);
                    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const float2 y = fma2(make_float2(__uint_as_float(sr[4 * x + 2 * k]),
                                                          __uint_as_float(sr[4 * x + 2 * k + 1])), c2, n2);
                        const float2 e = make_float2(ex2(y.x), ex2(y.y));
                        sum = add2(sum, e);
                        pk[2 * x + k] = bf16x2(e.x, e.y);
                    }
                    l_run[k] += sum.x + sum.y;
                }
            }
            if (!dead && !__all_sync(0xffffffffu, free))     // the P tile has been read
                dead = !__all_sync(0xffffffffu, mbar_wait_sleep(&bars->pv_done, (uint32_t)((j - 1) & 1), p.err,
                                                          kRoleSoftmax | kBarPV | (unsigned)(j & 0xffff)));
            if (!dead) {
                if (rows_here) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint8_t* row = smem + L::kOffP + (ra + 8 * k) * 128 + 4 * q4;
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            *reinterpret_cast<uint32_t*>(row + ((x ^ (ra & 7)) << 4)) = pk[2 * x + k];
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->p_full);
            }
        }
        if (tid == 0) griddep_launch_dependents();
        if (!dead)
            dead = !__all_sync(0xffffffffu, mbar_wait_sleep(&bars->pv_done, (uint32_t)((n - 1) & 1), p.err,
                                                      kRoleSoftmax | kBarLast));
        if (rows_here) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                l_run[k] += __shfl_xor_sync(0xffffffffu, l_run[k], 1);
                l_run[k] += __shfl_xor_sync(0xffffffffu, l_run[k], 2);
            }
        }
        dead = softmax_any(dead);
        if (!dead) {
            tc_fence_after();
            const bool whole = sl.S_b == 1;
            if (rows_here && q4 == 0) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int r = ra + 8 * k;
                    if (!live[k]) continue;
                    if (whole) {
                        bars->factor[r] = l_run[k] == 0.f ? 0.f : 1.f / l_run[k];
                        p.LSE[(int64_t)b * R + r0 + r] =
                            l_run[k] == 0.f ? -INFINITY : (m_run[k] + log2f(l_run[k])) * kLn2;
                    } else {
                        float* ml = p.part_ml + ((int64_t)slot_idx * R + r0 + r) * 2;
                        ml[0] = m_run[k];
                        ml[1] = l_run[k];
                    }
                }
            }
            if (whole) asm volatile("bar.sync 1, 128;" ::: "memory");
            // lane = dimension, register = row
#pragma unroll 1
            for (int x0 = 0; x0 < NR / 4; x0 += 2) {
                uint32_t both[2][16];
                tmem_ld16(lane_addr + L::kTmemO + (uint32_t)(16 * x0), both[0]);
                tmem_ld16(lane_addr + L::kTmemO + (uint32_t)(16 * x0 + 16), both[1]);
                tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t (&o)[16] = both[y];
                const int x = x0 + y, blk = 16 * x / NR, col = 16 * x % NR;
                const int dim = 128 * blk + tid;
                if (whole) {
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.O) +
                                         ((int64_t)b * R + r0 + col) * kLatent + dim;
#pragma unroll
                    for (int u = 0; u < 16; ++u)
                        if (col + u < Rb)
                            dst[(int64_t)u * kLatent] = __float2bfloat16_rn(__uint_as_float(o[u]) *
                                                                            bars->factor[col + u]);
                } else {
                    float* dst = p.part_acc + ((int64_t)slot_idx * R + r0 + col) * kLatent + dim;
#pragma unroll
                    for (int u = 0; u < 16; ++u)
                        if (col + u < Rb) dst[(int64_t)u * kLatent] = __uint_as_float(o[u]);
                }
              }
            }
        }
        if (dead) bars->abort = 1;
    } else if (warp < kConvWarp) {
        if (warp == kProducerWarp) {
            // ------------------------------ copies --------------------------------
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars->q_full, kChunks * L::kQChunk);
                tma_load_3d(smem + L::kOffQ, &tmQ, 0, b * R + r0, 0, &bars->q_full);
                constexpr int kCopied = Q8 ? 1 : kPieces;      // pieces of a tile: 8-bit rows, the rotated part
                int issued = 0;
                bool ok = true;
                // 8-bit rows are asked into L2 two tiles ahead (the converters load a tile late, below)
                auto ahead = [&](int j) {
                    if (!Q8 || j >= n) return;
                    const int64_t row = (int64_t)(t_begin + j) * kKeys, rows = min((int64_t)kKeys, p.cap - row);
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                     p.cache + ((int64_t)b * p.cap + row) * kLatentQ8Row),
                                 "r"((uint32_t)(rows * kLatentQ8Row))
                                 : "memory");
                };
                ahead(1);
                for (int j = 0; j < n && ok; ++j) {
                    const int st = j & 1;
                    uint8_t* tile = smem + L::kOffTile + st * kTile;
                    const int y = (t_begin + j) * kKeys;
                    ahead(j + 2);
                    for (int g = 0; g < kCopied; ++g) {
                        if ((j >= 2 && !mbar_wait_sleep(&bars->empty[st][g], (uint32_t)(((j >> 1) + 1) & 1), p.err,
                                                        kRoleProducer | kBarEmpty | (unsigned)(j & 0xffff))) ||
                            *((volatile int*)&bars->abort)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&bars->full[st][g], g == 0 ? kChunk : 2 * kChunk);
                        if (Q8)
                            tma_load_3d(tile + 8 * kChunk, &tmC, 0, y, b, &bars->full[st][0]);
                        else
                            tma_load_4d(tile + (g == 0 ? 8 : 2 * (g - 1)) * kChunk, g == 0 ? &tmR : &tmC, 0, y,
                                        g == 0 ? 0 : 2 * (g - 1), b, &bars->full[st][g]);
                        ++issued;
                    }
                }
                if (!ok) bars->abort = 1;
                // The copies in flight land before the CTA exits, whichever role may have given up: the last
                // two tiles', the last phases of their barriers.
                for (int x = max(0, issued - 2 * kCopied); x < issued; ++x)
                    mbar_wait_sleep(&bars->full[(x / kCopied) & 1][x % kCopied], (uint32_t)((x / kCopied >> 1) & 1),
                                    p.err, kRoleProducer | kBarFull);
                mbar_wait_sleep(&bars->q_full, 0, p.err, kRoleProducer | kBarLast);
            }
        } else if (warp == kQkWarp || warp == kPvWarp) {
            // ------------------------------ products ------------------------------
            // A warp for each product: what they wait for is on barriers alone.  The whole warp runs
            // the loop (addresses and descriptors stay in uniform registers) and one lane issues.
            const uint32_t base = smem_u32(smem);
            const uint32_t tm = __reduce_or_sync(0xffffffffu, tmem);
            const uint32_t leader = elect_one();
            const int tiles = __reduce_max_sync(0xffffffffu, n);
            auto wait = [&](uint64_t* bar, int phase, unsigned code) {
                return __all_sync(0xffffffffu, mbar_wait_sleep(bar, (uint32_t)(phase & 1), p.err, kRoleMma | code)) != 0;
            };
            bool ok = true;
            if (warp == kQkWarp) {
                const uint64_t qd = sdesc(base + L::kOffQ, 16, 1024);
                const uint64_t kd0 = sdesc(base + L::kOffTile, 16, 1024);
                ok = wait(&bars->q_full, 0, kBarLast);
#pragma unroll 1
                for (int j = 0; ok && j < tiles; ++j) {
                    const int st = j & 1;
                    const uint32_t dS = tm + L::kTmemS + (uint32_t)(st * kKeys);
                    const uint64_t kd = kd0 + (uint64_t)(st * (kTile >> 4));
                    if (j >= 2) ok = wait(&bars->s_free[st], (j >> 1) + 1, kBarS | (unsigned)(j & 0xffff));
#pragma unroll
                    for (int g = 0; g < kPieces; ++g) {
                        ok = ok && wait(&bars->full[st][g], j >> 1, kBarFull | (unsigned)(j & 0xffff));
                        if (!ok) break;
                        tc_fence_after();
                        const int c0 = g == 0 ? 8 : 2 * (g - 1);      // first chunk of the piece
                        mma4_if<2, 2>(leader, dS, qd + (uint64_t)(c0 * L::kQChunk >> 4), kd + (uint64_t)(c0 * kChunk >> 4),
                                      kIdescS, g > 0 ? 1u : 0u);
                        if (g > 0)
                            mma4_if<2, 2>(leader, dS, qd + (uint64_t)((c0 + 1) * L::kQChunk >> 4),
                                          kd + (uint64_t)((c0 + 1) * kChunk >> 4), kIdescS, 1u);
                    }
                    if (!ok) break;
                    mma_commit_if(leader, &bars->empty[st][0]);
                    mma_commit_if(leader, &bars->s_full[st]);
                }
            } else {
                const uint64_t vd0 = sdesc(base + L::kOffTile, kChunk, 1024);
                const uint64_t pd = sdesc(base + L::kOffP, 16, 1024);
#pragma unroll 1
                for (int j = 0; j < tiles; ++j) {
                    const int st = j & 1;
                    const uint64_t vd = vd0 + (uint64_t)(st * (kTile >> 4));
                    ok = wait(&bars->p_full, j, kBarPV | (unsigned)(j & 0xffff));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t add = j > 0 ? 1u : 0u;
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        mma4_if<2048 / 16, 2>(leader, tm + L::kTmemO + (uint32_t)(m * NR),
                                              vd + (uint64_t)(2 * m * kChunk >> 4), pd, L::kIdescPV, add);
                        mma_commit_if(leader, &bars->empty[st][1 + m]);
                    }
                    mma_commit_if(leader, &bars->pv_done);
                }
            }
            if (!ok) bars->abort = 1;
            // nothing in flight when tensor memory is freed
            mma_commit_if(leader, &bars->drain[warp - kQkWarp]);
            mbar_wait(&bars->drain[warp - kQkWarp], 0, p.err, kRoleMma | kBarLast);
        }
    } else if constexpr (Q8) {
        // ------------------------------ conversion ----------------------------
        // Thread: a quarter of a key, 16 codes at a time: 16 bytes in, 32 out.
        const int ct = tid - 32 * kConvWarp, key = ct >> 2, q = ct & 3;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.cache + ((int64_t)b * p.cap + (int64_t)t_begin * kKeys + key) * kLatentQ8Row);
        int64_t left = p.cap - (int64_t)t_begin * kKeys - key;    // rows of the cache from this one on
        uint4 v[8], sc;
        auto load_tile = [&] {
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = left > 0 ? src[4 * u + q] : make_uint4(0, 0, 0, 0);
            sc = left > 0 ? src[kLatentQ8Scale / 16] : make_uint4(0, 0, 0, 0);
        };
        load_tile();
        // 16-byte units 2 q and 2 q + 1 of a chunk
        const uint32_t unit0 = smem_u32(smem) + L::kOffTile + (uint32_t)(key * 128 + (((2 * q) ^ (key & 7)) << 4));
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            const int st = j & 1;
            const float scale[4] = {__uint_as_float(sc.x), __uint_as_float(sc.y), __uint_as_float(sc.z),
                                    __uint_as_float(sc.w)};
            bool ok = true;
            // Two halves of 256 values, each converted while the room is still in use.  The last piece of a
            // half is free only after its others (the products that read them are issued in order).
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t o[4][8];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int u = 4 * half + x;
                    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float2 y = mul2(e4m3x2((uint16_t)(w[k >> 1] >> (16 * (k & 1)))),
                                              make_float2(scale[u >> 1], scale[u >> 1]));
                        o[x][k] = bf16x2(y.x, y.y);
                    }
                }
                if (j >= 2)
                    ok = __all_sync(0xffffffffu, mbar_wait_sleep(&bars->empty[st][2 + 2 * half], (uint32_t)(((j >> 1) + 1) & 1),
                                                                 p.err, kRoleConvert | kBarEmpty | (unsigned)(j & 0xffff)));
                if (!ok) break;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t to = unit0 + (uint32_t)(st * kTile + (4 * half + x) * kChunk);
                    sts128(to, o[x][0], o[x][1], o[x][2], o[x][3]);
                    sts128(to ^ 16u, o[x][4], o[x][5], o[x][6], o[x][7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars->full[st][1 + 2 * half]);
                    mbar_arrive(&bars->full[st][2 + 2 * half]);
                }
            }
            if (!ok) {
                bars->abort = 1;
                break;
            }
            // A proxy fence waits for the loads before it, so the next tile's are issued behind the tile's last
            // one.  (Non-coherent loads would not be waited for, but the rows may have been written while
            // this kernel was already there; those issued early and without the look ahead into L2: 385 us
            // for the tree against 380.)
            src += kKeys * kLatentQ8Row / 16;
            left -= kKeys;
            if (j + 1 < n) load_tile();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kQkWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kTmemCols)
                     : "memory");
    }
}

// Joins the splits of a row by log-sum-exp: one block for 128 dimensions of a row.  Its threads work
// out the splits' weights together, then its warps add up splits in turn, 8 loads in flight each.
// Many splits (few rows) get 16 warps: 152 splits of 16 rows take 4 us, 14 with 4 warps.
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS) latent_merge_kernel(const LatentAttnParams p) {
    extern __shared__ float weight[];             // [p.S]
    __shared__ float4 s_acc[WARPS][32];
    __shared__ float s_red[WARPS];
    griddep_wait();
    const int R = p.H * p.n_q;
    const int64_t row = blockIdx.x;
    const int b = (int)(row / R), r = (int)(row - (int64_t)b * R);
    const int count = p.part_count[b];
    if (count <= 1) return;                       // written by its only split
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = (int64_t)p.part_first[b] * R + r;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + first;
    auto block = [&](float x, bool sum) -> float {
        x = sum ? warp_sum(x) : warp_max(x);
        __syncthreads();
        if (lane == 0) s_red[warp] = x;
        __syncthreads();
        x = s_red[0];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) x = sum ? x + s_red[w] : fmaxf(x, s_red[w]);
        return x;
    };
    float M = -INFINITY;
    for (int s = threadIdx.x; s < count; s += 32 * WARPS) M = fmaxf(M, ml[(int64_t)s * R].x);
    M = block(M, false);
    const float ref = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    for (int s = threadIdx.x; s < count; s += 32 * WARPS) {
        const float2 x = ml[(int64_t)s * R];
        const float f = ex2(x.x - ref);
        weight[s] = f;
        l = fmaf(f, x.y, l);
    }
    l = block(l, true);
    const float* acc = p.part_acc + first * kLatent + 128 * blockIdx.y + 4 * lane;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = warp; s < count; s += WARPS) {
        const float f = weight[s];
        const float4 x = __ldcs(reinterpret_cast<const float4*>(acc + (int64_t)s * R * kLatent));
        a.x = fmaf(f, x.x, a.x); a.y = fmaf(f, x.y, a.y);
        a.z = fmaf(f, x.z, a.z); a.w = fmaf(f, x.w, a.w);
    }
    s_acc[warp][lane] = a;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
        const float4 x = s_acc[w][lane];
        a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint2* dst = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + row * kLatent + 128 * blockIdx.y) + lane;
    *dst = make_uint2(bf16x2(a.x * inv, a.y * inv), bf16x2(a.z * inv, a.w * inv));
    if (lane == 0 && blockIdx.y == 0) p.LSE[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

// Rows as chunks of 64 values: box_rows rows of box_chunks chunks, chunk by chunk.
bool make_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
              const cuuint64_t* strides, uint32_t box_rows, uint32_t box_chunks) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint32_t box[4] = {64, box_rows, box_chunks, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NR, bool Q8>
cudaError_t launch_rows(const CUtensorMap& tmQ, const CUtensorMap& tmC, const CUtensorMap& tmR,
                        const LatentAttnParams& p, cudaStream_t st) {
    auto kern = latent_attn_kernel<NR, Q8>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<NR, Q8>::kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.S * p.RB, 1, 1);
    cfg.blockDim = dim3(Plan<NR, Q8>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = Plan<NR, Q8>::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, tmQ, tmC, tmR, p);
    if (e != cudaSuccess || p.S == p.B) return e;
    cfg.gridDim = dim3((unsigned)((int64_t)p.B * p.H * p.n_q), kLatent / 128, 1);
    cfg.dynamicSmemBytes = (size_t)p.S * sizeof(float);
    if (p.S > 32) {
        cfg.blockDim = dim3(512, 1, 1);
        return cudaLaunchKernelEx(&cfg, latent_merge_kernel<16>, p);
    }
    cfg.blockDim = dim3(128, 1, 1);
    return cudaLaunchKernelEx(&cfg, latent_merge_kernel<4>, p);
}

}  // namespace

int latent_attn_block_rows(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : 64; }

// Slots for the splits: CTAs run one to an SM, in w waves; a wave costs its tiles and the start
// and end of a CTA (about 4 tiles' time).  Fewer slots than sequences: one for each.
int latent_attn_slots(int B, int R, int64_t cap) {
    const int nr = latent_attn_block_rows(R);
    const int64_t rb = (R + nr - 1) / nr, sms = sm_count(), tiles = (cap + kKeys - 1) / kKeys * B;
    int64_t S = B;
    double least = 1e30;
    for (int w = 1; w <= 4; ++w) {
        const int64_t slots = w * sms / rb;
        if (slots <= B) continue;
        const double cost = w * ((double)((tiles + slots - 1) / slots) + 4.);
        if (cost < least) { least = cost; S = slots; }
    }
    return (int)S;
}

cudaError_t launch_latent_attn(const LatentAttnParams& p, cudaStream_t st) {
    CUtensorMap tmQ, tmC, tmR;
    const int64_t R = (int64_t)p.H * p.n_q;
    const int nr = latent_attn_block_rows((int)R);
    const cuuint64_t q_dims[3] = {64, (cuuint64_t)(p.B * R), kChunks};
    const cuuint64_t q_strides[2] = {2 * kLatentRow, 128};
    if (!make_map(&tmQ, p.Q, 3, q_dims, q_strides, (uint32_t)nr, kChunks)) return cudaErrorInvalidValue;
    if (p.q8) {
        // the rotated part of the rows
        const cuuint64_t dims[3] = {64, (cuuint64_t)p.cap, (cuuint64_t)p.B};
        const cuuint64_t strides[2] = {kLatentQ8Row, (cuuint64_t)p.cap * kLatentQ8Row};
        if (!make_map(&tmC, p.cache + kLatentQ8Rope, 3, dims, strides, kKeys, 1)) return cudaErrorInvalidValue;
        if (nr == 16) return launch_rows<16, true>(tmQ, tmC, tmC, p, st);
        return nr == 32 ? launch_rows<32, true>(tmQ, tmC, tmC, p, st) : launch_rows<64, true>(tmQ, tmC, tmC, p, st);
    }
    const cuuint64_t dims[4] = {64, (cuuint64_t)p.cap, kChunks - 1, (cuuint64_t)p.B};
    const cuuint64_t strides[3] = {2 * kLatentRow, 128, (cuuint64_t)p.cap * 2 * kLatentRow};
    const cuuint64_t r_dims[4] = {64, (cuuint64_t)p.cap, 1, (cuuint64_t)p.B};
    if (!make_map(&tmC, p.cache, 4, dims, strides, kKeys, 2) ||
        !make_map(&tmR, p.cache + 2 * kLatent, 4, r_dims, strides, kKeys, 1))
        return cudaErrorInvalidValue;
    if (nr == 16) return launch_rows<16, false>(tmQ, tmC, tmR, p, st);
    return nr == 32 ? launch_rows<32, false>(tmQ, tmC, tmR, p, st) : launch_rows<64, false>(tmQ, tmC, tmR, p, st);
}

}  // namespace rapid
