// Expanded attention of a prompt chunk on tensor cores: keys of 128 values for each head and 64
// that all heads share, values of 128, causal behind a prefix.
//
//   s_ij = <q_i, [k_j, r_j]>,   O_i = sum_{j <= prefix + i} softmax(scale s_i)_j v_j
//
// CTA = 256 tokens of one head, as two tiles of 128 that share every tile of 128 keys.  In tensor
// memory each has S (128 columns) and O (128): all of it.  P (bf16) takes the place of the S that it
// is made from, so a tile's products and its softmax alternate, and the two tiles fill the
// tensor unit for each other:
//   S = Q K^T   M = 128, N = 128, K = 192       P V   M = 128, N = 2 x 64, K = 128, P from tensor memory
// Keys and values pass through a ring of eight 16 KB chunks (128 keys x 64 values: k 0, k 1, r, v 0,
// v 1 of each tile of keys), so the next keys come while this tile's values wait.  Warps:
//   0-3, 4-7  softmax of the two tiles: a thread has a token's 128 scores.  The running maximum
//             moves only when a score passes it by more than 2^16, and O is rescaled then
//   8         copies by TMA
//   9, 10     issue the products of the two tiles
//   11        cleans the values of key tiles that some token does not see whole (below)
// With few blocks of tokens (latent_prefill_ctas) the blocks' key tiles form one line, in the order
// (sequence, block, head, tile), and each of one wave of CTAs takes an equal run of it: parts of blocks
// leave (O, maximum, sum) in the workspace, joined by log-sum-exp, whole ones are written at once.
// P is rounded to bf16 (at most 2^-8 of each probability, and it averages out); sums are fp32.
//
// Keys that a token does not see have no effect on it, whatever they hold: in tiles of keys that some
// token of the CTA does not see whole, a warp zeroes the values of keys behind the chunk in shared memory,
// and of keys with a value that is not finite, whose probabilities become NaN for the tokens that see
// them.  It does so while the scores are formed.
//
// Every wait is bounded in wall-clock time; after a failed wait the kernel records an error code,
// stops issuing, drains and returns.
//
// Measured, calls back to back (us; floor by operations at 1910 TFLOP/s, by bytes at 6788 GB/s where that is
// more): 8192 tokens of 32 heads 455 (360), 1.51 PFLOP/s at the 1755 MHz that the power limit leaves, 417 for a
// call alone; of 128 heads 1804 (1439), 1640 alone; three ragged chunks of up to 999 tokens of 16 heads behind
// up to 12001 135 to 140 (61); 16 tokens of 16 heads behind 16000 40 (19.7 by bytes).
// A tile of keys takes 2850 clocks for both tiles of tokens, 2710 of them the
// tensor unit's (68 for M = N = 128, 36 for M = 128, N = 64 with P in tensor memory).  The ragged chunks
// lose 6000 clocks between two pieces of a CTA (Q, whose room is in use until the last scores, then
// its first scores) and 10 us in the join.
#include <algorithm>
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "latent.cuh"
#include "tcgen05.cuh"

namespace rapid {

namespace {

constexpr int kTile = 128;                       // tokens, and keys, of a tile
constexpr int kChunk = kTile * 128;              // 64 values of 128 rows: 16 KB
constexpr int kRing = 8;
constexpr int kOffQ = 0, kOffRing = 6 * kChunk, kOffBar = kOffRing + kRing * kChunk;
constexpr int kBarBytes = 2048;
constexpr int kMaxPairs = 352;                   // blocks of tokens of all sequences that a line can hold
constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;   // + alignment
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr int kProducerWarp = 8, kMmaWarp = 9, kCleanWarp = 11, kThreads = 384;
// A block starts with 168 registers a thread; its warpgroups share them out anew.
constexpr int kSoftmaxRegs = 184, kLastRegs = 136;
static_assert(2 * kSoftmaxRegs + kLastRegs <= 3 * 168, "registers of a block");
constexpr uint32_t kTmemS = 0, kTmemO = 256;     // + 128 for the second tile
constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kTile >> 3) << 17) |
                             ((uint32_t)(128 >> 4) << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(64 >> 3) << 17) |
                              ((uint32_t)(128 >> 4) << 24);

enum : unsigned int {
    kRoleProducer = 0x31u << 24, kRoleMma = 0x32u << 24, kRoleSoftmax = 0x33u << 24, kRoleClean = 0x34u << 24,
    kBarFull = 1u << 16, kBarEmpty = 2u << 16, kBarS = 3u << 16, kBarP = 4u << 16, kBarPV = 5u << 16,
    kBarLast = 6u << 16, kBarClean = 7u << 16
};

// A run of the line: from tile j0 of head h of block `pair` (sequence * blocks + block) on.
struct Run {
    int pair, h, j0;
    int left;                // tiles
};

struct Bars {
    uint64_t full[kRing], empty[kRing];
    uint64_t q_full[2], s_full[2], pv_done[2], drain[2];
    uint64_t q_free;         // the products of a piece have read Q (of both tiles: it also keeps them in one piece)
    uint64_t lead;           // the first tile's first scores of a piece are there
    uint64_t o_free[2];      // O of a piece (that has one) has been read
    uint64_t p_full[2][2];   // P of a tile's first and second 64 keys
    uint32_t tmem_base;
    int abort;
    Run run;
    Run softmax_run[8];      // each softmax warp's, while its registers hold scores
    int tiles[kMaxPairs];    // key tiles of each block
    // Masked tiles, four in turn: the values are there; they are clean; keys with one that is not finite
    uint64_t dirty[4], clean[4];
    uint32_t flagged[4][4];
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block too small");

RAPID_DEVICE float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
RAPID_DEVICE float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
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
// 32 bytes at once (a whole sector)
RAPID_DEVICE void stg256(void* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
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

// Key tiles of block qb of sequence b (0: no tokens there, or a refused sequence).
RAPID_DEVICE int block_tiles(const LatentPrefillParams& p, int b, int qb) {
    const int count = p.n_rows ? p.n_rows[b] : p.n;
    const int64_t P = p.prefix_len[b];
    if (count < 0 || count > p.n || P < 0 || P + count > p.kv_rows) return 0;
    const int last = min(2 * kTile * (qb + 1), count) - 1;
    return last < 2 * kTile * qb ? 0 : (int)((P + last) / kTile + 1);
}

// CTAs that have a run of a line of T tiles: at least one tile each.
RAPID_DEVICE int line_ctas(const LatentPrefillParams& p, int64_t T) { return T < p.ctas ? (int)T : p.ctas; }

// CTA c's run of the line of all blocks' key tiles, worked out by one warp; the blocks' tiles go to
// `tiles`, where they start and how long the line is to the workspace (by CTA 0).
RAPID_DEVICE Run find_run(const LatentPrefillParams& p, int blocks, int c, int lane, int* tiles) {
    const int pairs = p.B * blocks;
    int total = 0;
    for (int x = lane; x < pairs; x += 32) total += tiles[x] = block_tiles(p, x / blocks, x % blocks);
    __syncwarp();
    const int64_t T = (int64_t)__reduce_add_sync(0xffffffffu, total) * p.H;
    const int ctas = line_ctas(p, T);
    const int64_t from = c * T / max(ctas, 1), to = (c + 1) * T / max(ctas, 1);
    Run r{0, 0, 0, c < ctas ? (int)(to - from) : 0};
    int64_t start = 0;                            // of the pairs of this round
    for (int x0 = 0; x0 < pairs; x0 += 32) {
        const int x = x0 + lane;
        const int64_t here = x < pairs ? (int64_t)tiles[x] * p.H : 0;
        int64_t upto = here;                      // inclusive scan
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        if (c == 0 && x < pairs) p.part_first[x] = start + upto - here;
        const uint32_t hit = __ballot_sync(0xffffffffu, from >= start + upto - here && from < start + upto);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int64_t at = from - (start + __shfl_sync(0xffffffffu, upto - here, l));
            r.pair = x0 + l;
            r.h = (int)(at / tiles[r.pair]);
            r.j0 = (int)(at % tiles[r.pair]);
        }
        start += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (c == 0 && lane == 0) p.part_first[pairs] = T;
    return r;
}
// The CTA whose run holds tile x of a line of T.
RAPID_DEVICE int cta_of(int64_t x, int64_t T, int ctas) { return (int)(((x + 1) * ctas - 1) / T); }

// SPLIT: the grid is p.ctas runs of the line; else a CTA for every block of tokens.
template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
latent_prefill_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmR,
                      const LatentPrefillParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int blocks = (p.n + 2 * kTile - 1) / (2 * kTile);
    griddep_wait();
    Run run;
    if constexpr (SPLIT) {
        if (warp == 0) {
            run = find_run(p, blocks, blockIdx.x, lane, bars->tiles);
            if (lane == 0) bars->run = run;
            if (blockIdx.x == 0 && p.err)         // refused sequences
                for (int b = lane; b < p.B; b += 32) {
                    const int count = p.n_rows ? p.n_rows[b] : p.n;
                    const int64_t P = p.prefix_len[b];
                    if (count < 0 || count > p.n || P < 0 || P + count > p.kv_rows) atomicOr(p.err, kErrBadInput);
                }
        }
        __syncthreads();
        run = bars->run;
        if (run.left == 0) return;
    } else {
        // Groups of heads, and in a group the last blocks of all heads first, which are the longest: short ones
        // fill the end, and the keys and values in use stay in L2.  The last group takes the heads left over,
        // so that its end is filled too.  8K tokens, in calls after each other: 32 heads 453 us, 128 heads 1781
        // (all heads as one group 464 and 2070; the blocks of a head as neighbours 491 and 1804).
        const int heads = p.B * p.H, groups = heads / p.group, gi = min((int)blockIdx.x / (p.group * blocks), groups - 1);
        const int first = gi * p.group, width = gi + 1 < groups ? p.group : heads - first;
        const int at = blockIdx.x - first * blocks, row = at / width, bh = first + at - row * width;
        const int b = bh / p.H, qb = blocks - 1 - row;
        run = Run{b * blocks + qb, bh % p.H, 0, block_tiles(p, b, qb)};
        if (run.left == 0) {
            const int count = p.n_rows ? p.n_rows[b] : p.n;
            const int64_t P = p.prefix_len[b];
            if (qb == 0 && run.h == 0 && tid == 0 && p.err && (count < 0 || count > p.n || P < 0 || P + count > p.kv_rows))
                atomicOr(p.err, kErrBadInput);    // refused: left alone
            return;
        }
        if (tid == 0) bars->tiles[0] = run.left;
    }
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->q_full[t], 1);
            mbar_init(&bars->s_full[t], 1);
            for (int u = 0; u < 2; ++u) mbar_init(&bars->p_full[t][u], 4);
            mbar_init(&bars->pv_done[t], 1);
            mbar_init(&bars->o_free[t], 4);
            mbar_init(&bars->drain[t], 1);
        }
        mbar_init(&bars->lead, 1);
        mbar_init(&bars->q_free, 2);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars->dirty[i], 1);
            mbar_init(&bars->clean[i], 1);
        }
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&bars->tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    // The run's pieces, each of one block and head; every role goes through them.
    struct Piece {
        int b, h, i0;                             // sequence, head, first token
        int count;                                // tokens of the sequence
        int j0, n, seen;                          // its key tiles: from j0, n of `seen`
        int nt0, nt1;                             // ... of the block's two tiles of tokens
        int first_masked;                         // tile (of n) from which on some token does not see all keys
        int64_t P;
    };
    auto piece_of = [&](const Run& r) -> Piece {
        Piece q;
        q.b = r.pair / blocks;
        q.h = r.h;
        q.i0 = (r.pair - q.b * blocks) * 2 * kTile;
        q.count = p.n_rows ? p.n_rows[q.b] : p.n;
        q.P = p.prefix_len[q.b];
        q.seen = bars->tiles[SPLIT ? r.pair : 0];
        q.j0 = r.j0;
        q.n = min(q.seen - r.j0, r.left);
        q.first_masked = (int)((q.P + q.i0 + 1) / kTile) - q.j0;
        auto seen_by = [&](int t) {
            const int last = min(q.i0 + kTile * (t + 1), q.count) - 1;
            const int sees = last < q.i0 + kTile * t ? 0 : (int)((q.P + last) / kTile + 1);
            return max(0, min(sees - q.j0, q.n));
        };
        q.nt0 = seen_by(0);
        q.nt1 = seen_by(1);
        return q;
    };
    auto next_piece = [&](Run& r, int n) {
        r.left -= n;
        r.j0 = 0;
        if (r.left > 0 && ++r.h == p.H) {
            r.h = 0;
            do ++r.pair; while (bars->tiles[r.pair] == 0);
        }
    };

    if (warp < 8) {
        // ------------------------------ softmax -------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int t = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t s_addr = lane_addr + kTmemS + (uint32_t)(kTile * t);
        const uint32_t o_addr = lane_addr + kTmemO + (uint32_t)(kTile * t);
        const float c = p.scale_log2;
        bool dead = false;
        int at = 0, cleaned = 0;                  // tiles of this role, and masked ones, of earlier pieces
        auto wait = [&](uint64_t* bar, int phase, unsigned code) {
            return __all_sync(0xffffffffu, mbar_wait_sleep(bar, (uint32_t)(phase & 1), p.err, kRoleSoftmax | code)) != 0;
        };
#pragma unroll 1
        do {
            // What the loop needs of the piece; the rest is worked out again behind it (the scores take most
            // registers).  In tile j this token sees columns <= sees - 128 j, and from first_masked on
            // some token of the block does not see all.
            int nt, n, sees, first_masked;
            {
                const Piece pc = piece_of(run);
                nt = t ? pc.nt1 : pc.nt0;
                n = pc.n;
                if (SPLIT && lane == 0) bars->softmax_run[warp] = run;
                sees = (int)(pc.P + pc.i0 + kTile * t + row - (int64_t)pc.j0 * kTile);
                first_masked = pc.first_masked;
            }
            float m_run = -INFINITY, l_run = 0.f;
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const bool masked = j >= first_masked;
                const bool mine = j < nt;
                uint32_t s[4][32];
                if (mine && !dead) {
                    dead = !wait(&bars->s_full[t], at + j, kBarS | (unsigned)(j & 0xffff));
                    if (!dead) {
                        tc_fence_after();
#pragma unroll
                        for (int x = 0; x < 4; ++x) tmem_ld32(s_addr + (uint32_t)(32 * x), s[x]);
                        tmem_wait_ld();
                    }
                }
                if (masked && mine && !dead) {
                    const int m = cleaned + j - max(first_masked, 0), lim = sees - j * kTile;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {             // columns <= lim are seen
                        const uint32_t see = lim >= 32 * x + 31 ? 0xffffffffu : lim < 32 * x ? 0u : (2u << (lim - 32 * x)) - 1;
#pragma unroll
                        for (int u = 0; u < 32; ++u)
                            if (!((see >> u) & 1)) s[x][u] = 0xff800000u;           // -inf
                    }
                    dead = !wait(&bars->clean[m & 3], m >> 2, kBarClean | (unsigned)(j & 0xffff));
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t f = bars->flagged[m & 3][x];
                        if (f == 0) continue;
#pragma unroll
                        for (int u = 0; u < 32; ++u)
                            if (((f >> u) & 1) && 32 * x + u <= lim) s[x][u] = 0x7fffffffu;   // NaN
                    }
                }
                if (!mine || dead) continue;
                float mx[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    mx[x] = __uint_as_float(s[x][0]);
#pragma unroll
                    for (int u = 1; u < 31; u += 2)
                        mx[x] = fmax3(mx[x], __uint_as_float(s[x][u]), __uint_as_float(s[x][u + 1]));
                    mx[x] = fmaxf(mx[x], __uint_as_float(s[x][31]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                float fac = 1.f;
                bool moved = false;
                if (top > m_run + 16.f) {              // the first finite score too
                    fac = ex2(m_run - top);           // 0 where m_run is -inf
                    m_run = top;
                    l_run *= fac;
                    moved = j > 0;
                }
                if (__any_sync(0xffffffffu, moved)) {
                    // O is rescaled (S of this tile was issued behind the product that last added to O)
#pragma unroll 1
                    for (int x = 0; x < 8; ++x) {
                        uint32_t o[16];
                        tmem_ld16(o_addr + (uint32_t)(16 * x), o);
                        tmem_wait_ld();
#pragma unroll
                        for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * fac);
                        tmem_st16(o_addr + (uint32_t)(16 * x), o);
                    }
                }
                const float neg = m_run == -INFINITY ? 0.f : -m_run;
                const float2 c2 = make_float2(c, c), n2 = make_float2(neg, neg);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t pk[16];
#pragma unroll
                    for (int u = 0; u < 16; ++u) {
                        const float2 y = fma2(make_float2(__uint_as_float(s[x][2 * u]), __uint_as_float(s[x][2 * u + 1])), c2, n2);
                        const float2 e = make_float2(ex2(y.x), ex2(y.y));
                        sum = add2(sum, e);
                        pk[u] = bf16x2(e.x, e.y);
                    }
                    tmem_st16(s_addr + (uint32_t)(16 * x), pk);
                    if (x & 1) {                      // 64 keys' product can start
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars->p_full[t][x >> 1]);
                    }
                }
                l_run += sum.x + sum.y;
            }
            if (!dead && nt > 0) dead = !wait(&bars->pv_done[t], at + nt - 1, kBarLast);
            __syncwarp();
            if constexpr (SPLIT) run = bars->softmax_run[warp];
            const Piece pc = piece_of(run);
            const int i = pc.i0 + kTile * t + row;
            // A block's first part (the end of the run) and a later part (its start) have slots of their own.
            const bool part = SPLIT && pc.n < pc.seen;
            const int64_t part_row = (int64_t)(2 * blockIdx.x + (pc.j0 == 0)) * 2 * kTile + kTile * t + row;
            if (part && !dead) {
                p.part_ml[part_row * 2] = m_run;      // (no keys: -inf and 0, and no O)
                p.part_ml[part_row * 2 + 1] = l_run;
            }
            if (!dead && nt > 0) {
                tc_fence_after();
                const float inv = part ? 1.f : l_run == 0.f ? 0.f : 1.f / l_run;
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.O) +
                                                      (((int64_t)pc.b * p.n + i) * p.H + pc.h) * kLatentHead);
                // a part's O: [32 dimensions of 4][256 tokens], so that a warp's stores are whole lines
                float4* acc = reinterpret_cast<float4*>(p.part_acc) +
                              (int64_t)(2 * blockIdx.x + (pc.j0 == 0)) * 32 * 2 * kTile + kTile * t + row;
                const bool whole_sectors = (reinterpret_cast<uintptr_t>(p.O) & 31) == 0;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    uint32_t o[16];
                    tmem_ld16(o_addr + (uint32_t)(16 * x), o);
                    tmem_wait_ld();
                    if (part && i < pc.count) {
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            acc[(4 * x + u) * 2 * kTile] =
                                make_float4(__uint_as_float(o[4 * u]), __uint_as_float(o[4 * u + 1]),
                                            __uint_as_float(o[4 * u + 2]), __uint_as_float(o[4 * u + 3]));
                    } else if (i < pc.count) {
                        uint32_t w[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            w[u] = bf16x2(__uint_as_float(o[2 * u]) * inv, __uint_as_float(o[2 * u + 1]) * inv);
                        if (whole_sectors) {
                            stg256(dst + 2 * x, w);
                        } else {
                            dst[2 * x] = make_uint4(w[0], w[1], w[2], w[3]);
                            dst[2 * x + 1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                }
                if (i < pc.count && !part)
                    p.LSE[((int64_t)pc.b * p.H + pc.h) * p.n + i] = l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && nt > 0) mbar_arrive(&bars->o_free[t]);
            at += nt;
            cleaned += n - min(n, max(first_masked, 0));
            next_piece(run, n);
        } while (SPLIT && run.left > 0);
        if (dead) bars->abort = 1;
        if (tid == 0) griddep_launch_dependents();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLastRegs));
        if (warp == kProducerWarp) {
            // ------------------------------ copies ----------------------------
            if (lane == 0) {
                int ch = 0, k = 0, q_loads = 0;   // chunks, pieces, loads of Q
                bool ok = true;
                while (ok && run.left > 0) {
                    const Piece pc = piece_of(run);
                    auto load_q = [&] {
                        for (int t = 0; t < 2; ++t) {
                            mbar_arrive_expect_tx(&bars->q_full[t], 3 * kChunk);
                            for (int x = 0; x < 3; ++x)
                                tma_load_4d(smem + kOffQ + (3 * t + x) * kChunk, &tmQ, 64 * x, pc.i0 + kTile * t, pc.h,
                                            pc.b, &bars->q_full[t]);
                        }
                        ++q_loads;
                    };
                    if (k == 0) load_q();
                    for (int j = 0; j < pc.n && ok; ++j) {
                        const int y = (pc.j0 + j) * kTile;
                        for (int x = 0; x < 5; ++x) {
                            if (j == 0 && x == 3 && k > 0) {      // behind the keys: Q is in use a little longer
                                ok = mbar_wait_sleep(&bars->q_free, (uint32_t)((k - 1) & 1), p.err, kRoleProducer | kBarLast);
                                if (!ok) break;
                                load_q();
                            }
                            const int sl = ch % kRing;
                            if ((ch >= kRing && !mbar_wait_sleep(&bars->empty[sl], (uint32_t)((ch / kRing + 1) & 1), p.err,
                                                                 kRoleProducer | kBarEmpty | (unsigned)(j & 0xffff))) ||
                                *((volatile int*)&bars->abort)) {
                                ok = false;
                                break;
                            }
                            mbar_arrive_expect_tx(&bars->full[sl], kChunk);
                            uint8_t* dst = smem + kOffRing + sl * kChunk;
                            if (x < 2) tma_load_4d(dst, &tmK, 64 * x, y, pc.h, pc.b, &bars->full[sl]);
                            else if (x == 2) tma_load_3d(dst, &tmR, 0, y, pc.b, &bars->full[sl]);
                            else tma_load_4d(dst, &tmV, 64 * (x - 3), y, pc.h, pc.b, &bars->full[sl]);
                            ++ch;
                        }
                    }
                    ++k;
                    next_piece(run, pc.n);
                }
                if (!ok) bars->abort = 1;
                // The copies in flight land before the CTA exits, whichever role may have given up: the last
                // chunks of the ring, the last phases of their barriers.
                for (int c = max(0, ch - kRing); c < ch; ++c)
                    mbar_wait_sleep(&bars->full[c % kRing], (uint32_t)((c / kRing) & 1), p.err, kRoleProducer | kBarFull);
                for (int t = 0; t < 2; ++t)
                    mbar_wait_sleep(&bars->q_full[t], (uint32_t)((q_loads - 1) & 1), p.err, kRoleProducer | kBarLast);
            }
        } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            // ------------------------------ products --------------------------
            // The whole warp runs the loop (addresses and descriptors stay in uniform registers)
            // and one lane issues.
            const int t = warp - kMmaWarp;
            const uint32_t base = smem_u32(smem);
            const uint32_t tm = __reduce_or_sync(0xffffffffu, tmem);
            const uint32_t leader = elect_one();
            const uint32_t dS = tm + kTmemS + (uint32_t)(kTile * t), dO = tm + kTmemO + (uint32_t)(kTile * t);
            const uint64_t qd = sdesc(base + kOffQ + 3 * t * kChunk, 16, 1024);
            const uint64_t rd = sdesc(base + kOffRing, 16, 1024);
            const uint64_t vd = sdesc(base + kOffRing, kChunk, 1024);
            auto wait = [&](uint64_t* bar, int phase, unsigned code) {
                return __all_sync(0xffffffffu, mbar_wait_sleep(bar, (uint32_t)(phase & 1), p.err, kRoleMma | code)) != 0;
            };
            auto chunk = [&](int ch) { return wait(&bars->full[ch % kRing], ch / kRing, kBarFull | (unsigned)(ch & 0xffff)); };
            // m >= 0: the values of masked tile m, whose chunks start at ch, are there to be cleaned
            auto have_cleaned = [&](int m, int ch) -> bool {
                if (m < 0) return true;
                if (!chunk(ch + 3) || !chunk(ch + 4)) return false;
                if (lane == 0) mbar_arrive(&bars->dirty[m & 3]);
                __syncwarp();                     // products and commits are issued by a whole warp
                return true;
            };
            auto scores = [&](int ch) -> bool {   // of the keys whose chunks start at ch
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    const int sl = (ch + x) % kRing;
                    if (!chunk(ch + x)) return false;
                    tc_fence_after();
                    mma4_if<2, 2>(leader, dS, qd + (uint64_t)(x * kChunk >> 4), rd + (uint64_t)(sl * (kChunk >> 4)),
                                  kIdescS, x > 0 ? 1u : 0u);
                    mma_commit_if(leader, &bars->empty[sl]);
                }
                mma_commit_if(leader, &bars->s_full[t]);
                return true;
            };
            bool ok = true;
            int at = 0, ch = 0, cleaned = 0;      // tiles of this role, chunks and masked tiles of earlier pieces
            int k = 0, with_o = 0, left = __reduce_max_sync(0xffffffffu, run.left);
#pragma unroll 1
            do {                                  // (on a condition that is known to be the warp's)
                const Piece pc = piece_of(run);
                const int nt = __reduce_max_sync(0xffffffffu, t ? pc.nt1 : pc.nt0), n = __reduce_max_sync(0xffffffffu, pc.n);
                const int first_masked = __reduce_max_sync(0xffffffffu, max(pc.first_masked, 0));
                ok = wait(&bars->q_full[t], k, kBarLast);
                // The second tile starts a product later: the tiles then run half a period apart, one in its
                // softmax while the other has the tensor unit (in step they take a quarter more).
                if (t == 1) ok = ok && wait(&bars->lead, k, kBarLast);
                // the first tile of tokens that sees a masked tile of keys has it cleaned
                auto to_clean = [&](int j) { return j >= first_masked && (t == 0 || j >= pc.nt0) ? cleaned + j - first_masked : -1; };
                if (nt > 0) ok = ok && have_cleaned(to_clean(0), ch) && scores(ch);
                if (t == 0) mma_commit_if(leader, &bars->lead);
                if (nt <= 1) mma_commit_if(leader, &bars->q_free);
                // O of the last piece that had one has been read
                if (nt > 0 && ++with_o > 1) ok = ok && wait(&bars->o_free[t], with_o - 2, kBarLast);
#pragma unroll 1
                for (int j = 0; ok && j < nt; ++j) {
                    const int c0 = ch + 5 * j + 3;
                    ok = chunk(c0) && chunk(c0 + 1);
                    if (j >= first_masked) {
                        const int m = cleaned + j - first_masked;
                        ok = ok && wait(&bars->clean[m & 3], m >> 2, kBarClean | (unsigned)(j & 0xffff));
                    }
                    const int sl0 = c0 % kRing, sl1 = (c0 + 1) % kRing;
                    const uint64_t v0 = vd + (uint64_t)(sl0 * (kChunk >> 4)), v1 = vd + (uint64_t)(sl1 * (kChunk >> 4));
#pragma unroll
                    for (int u = 0; u < 2; ++u) {         // 64 keys at a time
                        ok = ok && wait(&bars->p_full[t][u], at + j, kBarP | (unsigned)(j & 0xffff));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t add = u > 0 || j > 0 ? 1u : 0u;
                        mma4_ta_if<128>(leader, dO, dS + (uint32_t)(32 * u), v0 + (uint64_t)(512 * u), kIdescPV, add);
                        mma4_ta_if<128>(leader, dO + 64, dS + (uint32_t)(32 * u), v1 + (uint64_t)(512 * u), kIdescPV, add);
                    }
                    if (!ok) break;
                    mma_commit_if(leader, &bars->empty[sl0]);
                    mma_commit_if(leader, &bars->empty[sl1]);
                    mma_commit_if(leader, &bars->pv_done[t]);
                    if (j + 1 < nt) {
                        ok = have_cleaned(to_clean(j + 1), ch + 5 * (j + 1)) && scores(ch + 5 * (j + 1));
                        if (j + 2 == nt) mma_commit_if(leader, &bars->q_free);
                    }
                }
                // keys that only the other tile sees: their chunks are free for this one at once
                for (int c = ch + 5 * nt; ok && c < ch + 5 * n; ++c) {
                    ok = chunk(c);
                    if (ok && lane == 0) mbar_arrive(&bars->empty[c % kRing]);
                    __syncwarp();
                }
                at += nt;
                ch += 5 * n;
                cleaned += n - min(n, first_masked);
                next_piece(run, n);
                left -= n;
                ++k;
            } while (SPLIT && ok && left > 0);
            if (!ok) bars->abort = 1;
            // nothing in flight when tensor memory is freed
            mma_commit_if(leader, &bars->drain[t]);
            mbar_wait(&bars->drain[t], 0, p.err, kRoleMma | kBarLast);
        } else if (warp == kCleanWarp) {
            // ------------------------------ cleaning --------------------------
            bool ok = true;
            int ch = 0, m = 0;                    // chunks, and masked tiles, of earlier pieces
            do {
                const Piece pc = piece_of(run);
                const int there = (int)(pc.P + pc.count - (int64_t)pc.j0 * kTile);   // keys of the piece that are there
                for (int j = max(pc.first_masked, 0); ok && j < pc.n; ++j) {
                    const int c0 = ch + 5 * j + 3;
                    ok = __all_sync(0xffffffffu, mbar_wait_sleep(&bars->dirty[m & 3], (uint32_t)((m >> 2) & 1), p.err,
                                                                 kRoleClean | kBarFull | (unsigned)(j & 0xffff)));
                    if (!ok) break;
                    uint8_t* v[2] = {smem + kOffRing + (c0 % kRing) * kChunk, smem + kOffRing + ((c0 + 1) % kRing) * kChunk};
#pragma unroll 2
                    for (int r = 0; r < 4; ++r) {             // a lane's key; its 16-byte units in an order without
                        const int key = 32 * r + lane;        // bank conflicts
                        const bool inside = j * kTile + key < there;
                        uint32_t acc[4] = {0, 0, 0, 0};       // value * 0 is NaN where it is not finite
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const uint4 w = *reinterpret_cast<const uint4*>(v[x >> 3] + key * 128 + (((x ^ lane) & 7) << 4));
                            acc[0] = times_zero(w.x, acc[0]); acc[1] = times_zero(w.y, acc[1]);
                            acc[2] = times_zero(w.z, acc[2]); acc[3] = times_zero(w.w, acc[3]);
                        }
                        bool odd = false;
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            odd |= (acc[u] & 0x7fffu) > 0x7f80u || (acc[u] & 0x7fff0000u) > 0x7f800000u;
                        odd = odd && inside;
                        const uint32_t bits = __ballot_sync(0xffffffffu, odd);
                        if (lane == 0) bars->flagged[m & 3][r] = bits;
                        if (odd || !inside) {
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                *reinterpret_cast<uint4*>(v[x >> 3] + key * 128 + (((x ^ lane) & 7) << 4)) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->clean[m & 3]);
                    ++m;
                }
                ch += 5 * pc.n;
                next_piece(run, pc.n);
            } while (SPLIT && ok && run.left > 0);
            if (!ok) bars->abort = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// Joins the parts of a block's tokens by log-sum-exp: 32 tokens of a block and head, one to a lane; a warp
// adds up 16 dimensions of the parts, and the rows are written through shared memory.
constexpr int kMergeRows = 32;

__global__ void __launch_bounds__(256) latent_prefill_merge_kernel(const LatentPrefillParams p) {
    __shared__ float s_o[kMergeRows][kLatentHead + 4];
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, blocks = (p.n + 2 * kTile - 1) / (2 * kTile);
    const int pair = blockIdx.x / p.H, h = blockIdx.x - pair * p.H, b = pair / blocks, qb = pair - b * blocks;
    const int tiles = block_tiles(p, b, qb);
    if (tiles == 0) return;
    const int count = p.n_rows ? p.n_rows[b] : p.n;
    const int r = blockIdx.y * kMergeRows + lane, i0 = qb * 2 * kTile + blockIdx.y * kMergeRows;
    if (i0 >= count) return;
    const int64_t T = p.part_first[p.B * blocks];
    const int64_t start = p.part_first[pair] + (int64_t)h * tiles;
    const int ctas = line_ctas(p, T), c0 = cta_of(start, T, ctas), S = cta_of(start + tiles - 1, T, ctas) - c0 + 1;
    if (S <= 1) return;                           // written by its only CTA
    // part s: slot 2 c0 + 1, then 2 (c0 + s)
    auto slot_of = [&](int s) { return (int64_t)(2 * (c0 + s) + (s == 0)); };
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + r;
    const float4* acc = reinterpret_cast<const float4*>(p.part_acc) + 4 * warp * 2 * kTile + r;
    const bool live = i0 + lane < count;
    float M = -INFINITY;
#pragma unroll 4
    for (int s = 0; s < S; ++s) M = fmaxf(M, live ? ml[slot_of(s) * 2 * kTile].x : -INFINITY);
    const float ref = M == -INFINITY ? 0.f : M;
    float4 a[4] = {};
    float l = 0.f;
#pragma unroll 2
    for (int s = 0; s < S; ++s) {
        const float2 x = live ? ml[slot_of(s) * 2 * kTile] : make_float2(0.f, 0.f);
        if (x.y == 0.f) continue;                 // saw no key: left no O
        const float f = ex2(x.x - ref);
        l = fmaf(f, x.y, l);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float4 v = __ldcs(acc + slot_of(s) * 32 * 2 * kTile + u * 2 * kTile);
            a[u].x = fmaf(f, v.x, a[u].x); a[u].y = fmaf(f, v.y, a[u].y);
            a[u].z = fmaf(f, v.z, a[u].z); a[u].w = fmaf(f, v.w, a[u].w);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int u = 0; u < 4; ++u)
        *reinterpret_cast<float4*>(&s_o[lane][16 * warp + 4 * u]) =
            make_float4(a[u].x * inv, a[u].y * inv, a[u].z * inv, a[u].w * inv);
    if (warp == 0 && live)
        p.LSE[((int64_t)b * p.H + h) * p.n + i0 + lane] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMergeRows / 8; ++k) {
        const int i = i0 + warp * (kMergeRows / 8) + k;
        if (i >= count) break;
        const float4 o = *reinterpret_cast<const float4*>(&s_o[i - i0][4 * lane]);
        reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + (((int64_t)b * p.n + i) * p.H + h) * kLatentHead)[lane] =
            make_uint2(bf16x2(o.x, o.y), bf16x2(o.z, o.w));
    }
}

// Rows of `width` values with element strides for the outer dimensions (rows first); the
// stride of a dimension of size 1 means nothing, and the encoder wants one.
bool make_map(CUtensorMap* m, const void* base, int rank, const int64_t* dims, const int64_t* strides) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t d[4], s[3];
    cuuint32_t box[4] = {64, kTile, 1, 1}, estr[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) d[i] = (cuuint64_t)dims[i];
    for (int i = 0; i + 1 < rank; ++i) s[i] = (cuuint64_t)(strides[i] > 0 ? 2 * strides[i] : 16);
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, s, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Heads whose blocks are in flight together: their keys and values stay in L2 (48 MB of it, 8 to 32 heads).
int head_group(int heads, int64_t kv_rows) {
    const int64_t fit = ((int64_t)48 << 20) / (kv_rows * 2 * 2 * kLatentHead);
    return (int)std::min(std::min(std::max(fit, (int64_t)8), (int64_t)32), (int64_t)heads);
}

}  // namespace

cudaError_t launch_latent_prefill(LatentPrefillParams p, cudaStream_t st) {
    p.group = head_group(p.B * p.H, p.kv_rows);
    CUtensorMap tmQ, tmK, tmV, tmR;
    const int64_t qd[4] = {kLatentHead + kLatentRope, p.n, p.H, p.B}, kd[4] = {kLatentHead, p.kv_rows, p.H, p.B};
    const int64_t rd[3] = {kLatentRope, p.kv_rows, p.B};
    const int64_t qs[3] = {p.q_stride[1], p.q_stride[2], p.q_stride[0]};
    const int64_t ks[3] = {p.k_stride[1], p.k_stride[2], p.k_stride[0]};
    const int64_t vs[3] = {p.v_stride[1], p.v_stride[2], p.v_stride[0]};
    const int64_t rs[2] = {p.r_stride[1], p.r_stride[0]};
    if (!make_map(&tmQ, p.Q, 4, qd, qs) || !make_map(&tmK, p.K, 4, kd, ks) || !make_map(&tmV, p.V, 4, kd, vs) ||
        !make_map(&tmR, p.K_rope, 3, rd, rs))
        return cudaErrorInvalidValue;
    const int64_t grid = p.ctas ? p.ctas : (int64_t)p.B * p.H * ((p.n + 2 * kTile - 1) / (2 * kTile));
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    auto kern = p.ctas ? latent_prefill_kernel<true> : latent_prefill_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, tmQ, tmK, tmV, tmR, p);
    if (e != cudaSuccess || !p.ctas) return e;
    cfg.gridDim = dim3((unsigned)(p.B * ((p.n + 2 * kTile - 1) / (2 * kTile)) * p.H), 2 * kTile / kMergeRows, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, latent_prefill_merge_kernel, p);
}

// CTAs that share a line of all key tiles, or 0: every block of tokens its own CTA.
int latent_prefill_ctas(int B, int n, int H, int64_t kv_rows) {
    const int64_t pairs = (int64_t)B * ((n + 2 * kTile - 1) / (2 * kTile)), sms = sm_count();
    return pairs <= kMaxPairs && pairs * H <= 2 * sms && kv_rows > 4 * kTile ? (int)sms : 0;
}

size_t latent_prefill_block_rows() { return 2 * kTile; }

}  // namespace rapid
