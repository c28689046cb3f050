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
// Few blocks of tokens, or blocks behind long prefixes (latent_prefill_slots), share their keys out: a split
// takes a run of key tiles and leaves (O, maximum, sum) in the workspace, joined by log-sum-exp.
// P is rounded to bf16 (2^-9 of each probability, and it averages out); sums are fp32.
//
// Keys that a token does not see have no effect on it, whatever they hold: in tiles of keys that
// some token of the CTA does not see whole, values of keys behind the chunk become zeros in shared
// memory, and so do keys with a value that is not finite, whose probabilities become NaN for the
// tokens that see them.
//
// Every wait is bounded in wall-clock time; after a failed wait the kernel records an error code,
// stops issuing, drains and returns.
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
constexpr int kBarBytes = 1024;
constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;   // + alignment
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr int kProducerWarp = 8, kMmaWarp = 9, kThreads = 384;
// A block starts with 168 registers a thread; its warpgroups share them out anew.
constexpr int kSoftmaxRegs = 208, kLastRegs = 88;
static_assert(2 * kSoftmaxRegs + kLastRegs <= 3 * 168, "registers of a block");
constexpr uint32_t kTmemS = 0, kTmemO = 256;     // + 128 for the second tile
constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kTile >> 3) << 17) |
                             ((uint32_t)(128 >> 4) << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(64 >> 3) << 17) |
                              ((uint32_t)(128 >> 4) << 24);

enum : unsigned int {
    kRoleProducer = 0x31u << 24, kRoleMma = 0x32u << 24, kRoleSoftmax = 0x33u << 24,
    kBarFull = 1u << 16, kBarEmpty = 2u << 16, kBarS = 3u << 16, kBarP = 4u << 16, kBarPV = 5u << 16,
    kBarLast = 6u << 16
};

struct Piece {
    int b, h, qb;            // block of tokens of a head (b = -1: no work)
    int s, S;                // split, splits of the block
    int slot;                // first split's slot
};

struct Bars {
    uint64_t full[kRing], empty[kRing];
    uint64_t q_full[2], s_full[2], pv_done[2], drain[2];
    uint64_t p_full[2][2];   // P of a tile's first and second 64 keys
    uint32_t tmem_base;
    int abort;
    Piece piece;
    uint32_t flagged[4];     // keys of a tile with a value that is not finite
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

// Which block and split a slot holds, worked out by one warp: the least number of key tiles a split
// for which all splits fit into p.slots.  Splits lie in the order (sequence, block, head, split).
RAPID_DEVICE Piece find_piece(const LatentPrefillParams& p, int blocks, int c, int lane) {
    const int pairs = p.B * blocks;
    int longest = 1;
    int64_t total = 0;
    for (int x = lane; x < pairs; x += 32) {
        const int t = block_tiles(p, x / blocks, x % blocks);
        total += (int64_t)t * p.H;
        longest = max(longest, t);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
    }
    int lo = max(1, (int)((total + p.slots - 1) / p.slots)), hi = max(lo, longest);
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        int used = 0;
        for (int x = lane; x < pairs; x += 32) used += (block_tiles(p, x / blocks, x % blocks) + mid - 1) / mid;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) used += __shfl_xor_sync(0xffffffffu, used, o);
        if (used * p.H <= p.slots) hi = mid; else lo = mid + 1;
    }
    int first = 0;
    for (int x0 = 0; x0 < pairs; x0 += 32) {
        const int x = x0 + lane;
        const int S = x < pairs ? (block_tiles(p, x / blocks, x % blocks) + lo - 1) / lo : 0;
        int upto = S * p.H;                       // inclusive scan
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, c < first + upto);
        if (here) {
            const int l = __ffs(here) - 1;
            Piece r;
            r.S = __shfl_sync(0xffffffffu, S, l);
            const int start = first + __shfl_sync(0xffffffffu, upto, l) - r.S * p.H;
            r.b = (x0 + l) / blocks;
            r.qb = (x0 + l) % blocks;
            r.h = (c - start) / r.S;
            r.s = (c - start) % r.S;
            r.slot = start;
            return r;
        }
        first += __shfl_sync(0xffffffffu, upto, 31);
    }
    return Piece{-1, 0, 0, 0, 1, 0};
}

// SPLIT: the grid is p.slots pieces of key runs; else a CTA for every block of tokens.
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
    Piece pc;
    if constexpr (SPLIT) {
        if (warp == 0) {
            pc = find_piece(p, blocks, blockIdx.x, lane);
            if (lane == 0) bars->piece = pc;
            if (blockIdx.x == 0 && p.err)         // refused sequences
                for (int b = lane; b < p.B; b += 32) {
                    const int count = p.n_rows ? p.n_rows[b] : p.n;
                    const int64_t P = p.prefix_len[b];
                    if (count < 0 || count > p.n || P < 0 || P + count > p.kv_rows) atomicOr(p.err, kErrBadInput);
                }
        }
        __syncthreads();
        pc = bars->piece;
        if (pc.b < 0) return;
        if (tid == 0 && pc.h == 0 && pc.s == 0) {
            p.part_first[pc.b * blocks + pc.qb] = pc.slot;
            p.part_count[pc.b * blocks + pc.qb] = pc.S;
        }
    } else {
        // The blocks of a head are neighbours (their keys stay in L2), the longest first.
        const int bh = blockIdx.x / blocks;
        pc = Piece{bh / p.H, bh % p.H, blocks - 1 - (int)(blockIdx.x - bh * blocks), 0, 1, 0};
    }
    const int b = pc.b, h = pc.h, i0 = pc.qb * 2 * kTile;   // first token of the CTA
    const int count = p.n_rows ? p.n_rows[b] : p.n;
    const int64_t P = p.prefix_len[b];
    if (!SPLIT && (count < 0 || count > p.n || P < 0 || P + count > p.kv_rows)) {   // refused: left alone
        if (pc.qb == 0 && h == 0 && tid == 0 && p.err) atomicOr(p.err, kErrBadInput);
        return;
    }
    if (i0 >= count) return;
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
            mbar_init(&bars->drain[t], 1);
        }
        for (int i = 0; i < 4; ++i) bars->flagged[i] = 0;
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
    // tiles of keys that tile t of the CTA sees any of
    auto key_tiles = [&](int t) -> int {
        const int last = min(i0 + kTile * (t + 1), count) - 1;
        return last < i0 + kTile * t ? 0 : (int)((P + last) / kTile + 1);
    };
    const int seen0 = key_tiles(0), seen1 = key_tiles(1), seen = max(seen0, seen1);
    // the split's run of them, from j0 on, and the first that some token does not see whole
    const int j0 = (int)((int64_t)pc.s * seen / pc.S), j1 = (int)((int64_t)(pc.s + 1) * seen / pc.S);
    const int n = j1 - j0, n0 = max(0, min(seen0 - j0, n)), n1 = max(0, min(seen1 - j0, n));
    const int first_masked = (int)((P + i0 + 1) / kTile) - j0;

    if (warp < 8) {
        // ------------------------------ softmax -------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int t = warp >> 2, row = 32 * (warp & 3) + lane, nt = t ? n1 : n0;
        const int i = i0 + kTile * t + row;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t s_addr = lane_addr + kTmemS + (uint32_t)(kTile * t);
        const uint32_t o_addr = lane_addr + kTmemO + (uint32_t)(kTile * t);
        const float c = p.scale_log2;
        float m_run = -INFINITY, l_run = 0.f;
        bool dead = false;
        auto wait = [&](uint64_t* bar, int phase, unsigned code) {
            return __all_sync(0xffffffffu, mbar_wait_sleep(bar, (uint32_t)(phase & 1), p.err, kRoleSoftmax | code)) != 0;
        };
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            const bool masked = j >= first_masked;
            if (!masked && dead) continue;        // (the barriers below are for all)
            const bool mine = j < nt;
            uint32_t s[4][32];
            if (mine && !dead) {
                dead = !wait(&bars->s_full[t], j, kBarS | (unsigned)(j & 0xffff));
                if (!dead) {
                    tc_fence_after();
#pragma unroll
                    for (int x = 0; x < 4; ++x) tmem_ld32(s_addr + (uint32_t)(32 * x), s[x]);
                    tmem_wait_ld();
                }
            }
            if (masked) {
                // all 256 softmax threads: half a key's values each.  Only a tile that has S of
                // these keys knows which lap of the ring they are in, and waits for both.
                const int ch = 5 * j + 3 + (tid & 1), key = tid >> 1;
                if (mine && !dead) dead = !wait(&bars->full[(5 * j + 3) % kRing], (5 * j + 3) / kRing, kBarFull) ||
                                          !wait(&bars->full[(5 * j + 4) % kRing], (5 * j + 4) / kRing, kBarFull);
                asm volatile("bar.sync 1, 256;" ::: "memory");
                uint8_t* v = smem + kOffRing + (ch % kRing) * kChunk + key * 128;
                const bool inside = (int64_t)(j0 + j) * kTile + key < P + count;
                bool odd = false;
                if (inside && !dead) {
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const uint4 w4 = *reinterpret_cast<const uint4*>(v + 16 * x);
                        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            odd |= (w[u] & 0x7f80u) == 0x7f80u || (w[u] & 0x7f800000u) == 0x7f800000u;
                    }
                }
                if (odd) atomicOr(&bars->flagged[key >> 5], 1u << (key & 31));
                asm volatile("bar.sync 1, 256;" ::: "memory");
                const uint32_t f[4] = {bars->flagged[0], bars->flagged[1], bars->flagged[2], bars->flagged[3]};
                uint32_t mine_f = f[0];
#pragma unroll
                for (int u = 1; u < 4; ++u) mine_f = key >> 5 == u ? f[u] : mine_f;
                if (!dead && (!inside || ((mine_f >> (key & 31)) & 1))) {
#pragma unroll
                    for (int x = 0; x < 8; ++x) *reinterpret_cast<uint4*>(v + 16 * x) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (tid < 4) bars->flagged[tid] = 0;
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (mine && !dead) {
                    const int64_t lim = P + i - (int64_t)(j0 + j) * kTile;       // columns <= lim are seen
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int u = 0; u < 32; ++u) {
                            if (32 * x + u > lim) s[x][u] = 0xff800000u;            // -inf
                            else if ((f[x] >> u) & 1) s[x][u] = 0x7fffffffu;        // NaN
                        }
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
        if (!dead && nt > 0) dead = !wait(&bars->pv_done[t], nt - 1, kBarLast);
        const bool part = SPLIT && pc.S > 1;
        const int64_t part_row = (int64_t)blockIdx.x * 2 * kTile + kTile * t + row;
        if (part && !dead) {
            p.part_ml[part_row * 2] = m_run;      // (no keys: -inf and 0, and no O)
            p.part_ml[part_row * 2 + 1] = l_run;
        }
        if (!dead && nt > 0) {
            tc_fence_after();
            const float inv = part ? 1.f : l_run == 0.f ? 0.f : 1.f / l_run;
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.O) +
                                                  (((int64_t)b * p.n + i) * p.H + h) * kLatentHead);
            float4* acc = reinterpret_cast<float4*>(p.part_acc + part_row * kLatentHead);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                uint32_t o[16];
                tmem_ld16(o_addr + (uint32_t)(16 * x), o);
                tmem_wait_ld();
                if (i >= count) continue;
                if (part) {
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        acc[4 * x + u] = make_float4(__uint_as_float(o[4 * u]), __uint_as_float(o[4 * u + 1]),
                                                     __uint_as_float(o[4 * u + 2]), __uint_as_float(o[4 * u + 3]));
                    continue;
                }
                uint32_t w[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    w[u] = bf16x2(__uint_as_float(o[2 * u]) * inv, __uint_as_float(o[2 * u + 1]) * inv);
                dst[2 * x] = make_uint4(w[0], w[1], w[2], w[3]);
                dst[2 * x + 1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
            if (i < count && !part)
                p.LSE[((int64_t)b * p.H + h) * p.n + i] = l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
        }
        if (dead) bars->abort = 1;
        if (tid == 0) griddep_launch_dependents();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLastRegs));
        if (warp == kProducerWarp) {
            // ------------------------------ copies ----------------------------
            if (lane == 0) {
                auto load_q = [&](int t) {
                    mbar_arrive_expect_tx(&bars->q_full[t], 3 * kChunk);
                    for (int x = 0; x < 3; ++x)
                        tma_load_4d(smem + kOffQ + (3 * t + x) * kChunk, &tmQ, 64 * x, i0 + kTile * t, h, b, &bars->q_full[t]);
                };
                load_q(0);
                int issued = 0;
                bool ok = true;
                for (int j = 0; j < n && ok; ++j) {
                    for (int x = 0; x < 5; ++x) {
                        const int ch = 5 * j + x, sl = ch % kRing;
                        if ((ch >= kRing && !mbar_wait_sleep(&bars->empty[sl], (uint32_t)((ch / kRing + 1) & 1), p.err,
                                                             kRoleProducer | kBarEmpty | (unsigned)(j & 0xffff))) ||
                            *((volatile int*)&bars->abort)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&bars->full[sl], kChunk);
                        uint8_t* dst = smem + kOffRing + sl * kChunk;
                        if (x < 2) tma_load_4d(dst, &tmK, 64 * x, (j0 + j) * kTile, h, b, &bars->full[sl]);
                        else if (x == 2) tma_load_3d(dst, &tmR, 0, (j0 + j) * kTile, b, &bars->full[sl]);
                        else tma_load_4d(dst, &tmV, 64 * (x - 3), (j0 + j) * kTile, h, b, &bars->full[sl]);
                        ++issued;
                    }
                    if (j == 0) load_q(1);
                }
                if (!ok) {
                    bars->abort = 1;
                    // let the copies in flight land before the CTA exits
                    for (int ch = max(0, issued - kRing); ch < issued; ++ch)
                        mbar_wait(&bars->full[ch % kRing], (uint32_t)((ch / kRing) & 1), p.err, kRoleProducer | kBarFull);
                }
                mbar_wait_sleep(&bars->q_full[0], 0, p.err, kRoleProducer | kBarLast);
                mbar_wait_sleep(&bars->q_full[1], 0, p.err, kRoleProducer | kBarLast);
            }
        } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            // ------------------------------ products --------------------------
            // The whole warp runs the loop (addresses and descriptors stay in uniform registers)
            // and one lane issues.
            const int t = warp - kMmaWarp;
            const uint32_t base = smem_u32(smem);
            const uint32_t tm = __reduce_or_sync(0xffffffffu, tmem);
            const uint32_t leader = elect_one();
            const int nt = __reduce_max_sync(0xffffffffu, t ? n1 : n0), all = __reduce_max_sync(0xffffffffu, n);
            const uint32_t dS = tm + kTmemS + (uint32_t)(kTile * t), dO = tm + kTmemO + (uint32_t)(kTile * t);
            const uint64_t qd = sdesc(base + kOffQ + 3 * t * kChunk, 16, 1024);
            const uint64_t rd = sdesc(base + kOffRing, 16, 1024);
            const uint64_t vd = sdesc(base + kOffRing, kChunk, 1024);
            auto wait = [&](uint64_t* bar, int phase, unsigned code) {
                return __all_sync(0xffffffffu, mbar_wait_sleep(bar, (uint32_t)(phase & 1), p.err, kRoleMma | code)) != 0;
            };
            auto chunk = [&](int ch) { return wait(&bars->full[ch % kRing], ch / kRing, kBarFull | (unsigned)(ch & 0xffff)); };
            auto scores = [&](int j) -> bool {
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    const int sl = (5 * j + x) % kRing;
                    if (!chunk(5 * j + x)) return false;
                    tc_fence_after();
                    mma4_if<2, 2>(leader, dS, qd + (uint64_t)(x * kChunk >> 4), rd + (uint64_t)(sl * (kChunk >> 4)),
                                  kIdescS, x > 0 ? 1u : 0u);
                    mma_commit_if(leader, &bars->empty[sl]);
                }
                mma_commit_if(leader, &bars->s_full[t]);
                return true;
            };
            bool ok = nt == 0 || (wait(&bars->q_full[t], 0, kBarLast) && scores(0));
#pragma unroll 1
            for (int j = 0; ok && j < nt; ++j) {
                ok = chunk(5 * j + 3) && chunk(5 * j + 4);
                const int sl0 = (5 * j + 3) % kRing, sl1 = (5 * j + 4) % kRing;
                const uint64_t v0 = vd + (uint64_t)(sl0 * (kChunk >> 4)), v1 = vd + (uint64_t)(sl1 * (kChunk >> 4));
#pragma unroll
                for (int u = 0; u < 2; ++u) {         // 64 keys at a time
                    ok = ok && wait(&bars->p_full[t][u], j, kBarP | (unsigned)(j & 0xffff));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t add = u > 0 || j > 0 ? 1u : 0u;
                    mma4_ta_if<128>(leader, dO, dS + (uint32_t)(32 * u), v0 + (uint64_t)(512 * u), kIdescPV, add);
                    mma4_ta_if<128>(leader, dO + 64, dS + (uint32_t)(32 * u), v1 + (uint64_t)(512 * u), kIdescPV, add);
                }
                if (!ok) break;
                mma_commit_if(leader, &bars->empty[sl0]);
                mma_commit_if(leader, &bars->empty[sl1]);
                if (!ok) break;
                mma_commit_if(leader, &bars->pv_done[t]);
                if (j + 1 < nt) ok = scores(j + 1);
            }
            // keys that only the other tile sees: their chunks are free for this one at once
            for (int ch = 5 * nt; ok && ch < 5 * all; ++ch) {
                ok = chunk(ch);
                if (ok && lane == 0) mbar_arrive(&bars->empty[ch % kRing]);
            }
            if (!ok) bars->abort = 1;
            // nothing in flight when tensor memory is freed
            mma_commit_if(leader, &bars->drain[t]);
            mbar_wait(&bars->drain[t], 0, p.err, kRoleMma | kBarLast);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// Joins the splits of a token and head by log-sum-exp: one warp each.
__global__ void __launch_bounds__(128) latent_prefill_merge_kernel(const LatentPrefillParams p) {
    griddep_wait();
    const int lane = threadIdx.x & 31, blocks = (p.n + 2 * kTile - 1) / (2 * kTile);
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);   // (b, i, h)
    const int h = (int)(unit % p.H), b = (int)(unit / p.H / p.n), i = (int)(unit / p.H % p.n);
    if (b >= p.B) return;
    const int qb = i / (2 * kTile), count = p.n_rows ? p.n_rows[b] : p.n;
    if (i >= count || block_tiles(p, b, qb) == 0) return;
    const int S = p.part_count[b * blocks + qb];
    if (S <= 1) return;                           // written by its only split
    const int64_t row = ((int64_t)p.part_first[b * blocks + qb] + (int64_t)h * S) * 2 * kTile + i % (2 * kTile);
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + row;
    float M = -INFINITY;
    for (int s = lane; s < S; s += 32) M = fmaxf(M, ml[(int64_t)s * 2 * kTile].x);
    M = warp_max(M);
    const float ref = M == -INFINITY ? 0.f : M;
    const float4* acc = reinterpret_cast<const float4*>(p.part_acc + row * kLatentHead) + lane;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int s = 0; s < S; ++s) {
        const float2 x = ml[(int64_t)s * 2 * kTile];
        if (x.y == 0.f) continue;                 // saw no key: left no O
        const float f = ex2(x.x - ref);
        const float4 v = __ldcs(acc + (int64_t)s * 2 * kTile * (kLatentHead / 4));
        l = fmaf(f, x.y, l);
        a.x = fmaf(f, v.x, a.x); a.y = fmaf(f, v.y, a.y);
        a.z = fmaf(f, v.z, a.z); a.w = fmaf(f, v.w, a.w);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + (((int64_t)b * p.n + i) * p.H + h) * kLatentHead)[lane] =
        make_uint2(bf16x2(a.x * inv, a.y * inv), bf16x2(a.z * inv, a.w * inv));
    if (lane == 0) p.LSE[((int64_t)b * p.H + h) * p.n + i] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
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

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillParams& p, cudaStream_t st) {
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
    const int64_t grid = p.slots ? p.slots : (int64_t)p.B * p.H * ((p.n + 2 * kTile - 1) / (2 * kTile));
    const int64_t rows = ((int64_t)p.B * p.n * p.H + 3) / 4;
    if (grid > 0x7fffffff || rows > 0x7fffffff) return cudaErrorInvalidValue;
    auto kern = p.slots ? latent_prefill_kernel<true> : latent_prefill_kernel<false>;
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
    if (e != cudaSuccess || !p.slots) return e;
    cfg.gridDim = dim3((unsigned)rows, 1, 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, latent_prefill_merge_kernel, p);
}

// Slots for splits, or 0: every block of tokens its own CTA.  With no more blocks than SMs the longest
// of them alone would decide the time: one wave of pieces of equal length (16 tokens of 16 heads
// behind 16000, 41 us; two waves of shorter pieces 53).  Up to twice as many, two waves, if the
// blocks are about equally long because most keys are earlier ones (three ragged chunks of up to 999
// behind up to 12001, 192 blocks: 159 us, 259 unsplit; but 256 blocks of 1000 behind 1000 take
// 101, and 88 unsplit).  Few keys stay whole.
int latent_prefill_slots(int B, int n, int H, int64_t kv_rows) {
    const int64_t units = (int64_t)B * H * ((n + 2 * kTile - 1) / (2 * kTile)), sms = sm_count();
    if (kv_rows <= 4 * kTile) return 0;
    if (units <= sms) return (int)sms;
    return units <= 2 * sms && kv_rows >= 4 * (int64_t)n ? (int)(2 * sms) : 0;
}

size_t latent_prefill_block_rows() { return 2 * kTile; }

}  // namespace rapid
