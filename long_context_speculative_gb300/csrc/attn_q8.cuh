// Verify attention over an 8-bit history: shared parameter block, the split plan and kernel
// entry points.
//
// The keys of a sequence are its sealed pages (64 tokens each, e4m3 values with one scale
// for each page, KV head and side), then its tail rows, then the n_q speculative rows of the
// step, which follow the tail rows in the tail caches.  A history kernel splits them over
// CTAs that each leave an un-normalised partial (acc, m, l); a merge kernel combines the
// partials by log-sum-exp.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kv_seal.cuh"

namespace rapid {

// Keys of a tile, the unit of the split plan: two pages or 128 tail rows on tensor cores, one
// page or 64 tail rows on CUDA cores.
constexpr int kQ8Tile = 128;
constexpr int kQ8SimtTile = 64;

struct AttnQ8Params {
    const void* Q;               // [B, Hq, n_q, d]
    const void* K;               // [B, Hkv, cap, d] tail caches
    const void* V;
    const uint8_t* pages;        // [n_pages, Hkv, 2, 64, d] e4m3
    const float* scales;         // [n_pages, Hkv, 2]
    const int32_t* page_table;   // [B, max_pages]
    const int32_t* sealed_len;   // [B]
    const int32_t* tail_len;     // [B]
    const uint8_t* mask;         // [B, n_q, n_q] or nullptr (chain)
    void* O;                     // [B, Hq, n_q, d]
    float* LSE;                  // [B, Hq, n_q]
    // Partials of (KV head, slot, group row): acc [.., d], (m, l) with m in the log2 domain.
    // Sequence b's splits sit at slots part_first[b * Hkv + g] .. + part_count[..] - 1.
    float* part_acc;             // [Hkv, S, R, d]
    float* part_ml;              // [Hkv, S, R, 2]
    int* part_first;             // [B * Hkv]
    int* part_count;             // [B * Hkv]
    unsigned int* err;
    int64_t cap;                 // rows of a tail cache
    int B, Hq, Hkv, d, n_q, G, R;
    int max_pages, n_pages;
    int S;                       // (sequence, split) slots per KV head, at least B
    float scale_log2;            // softmax scale * log2(e)
};

// Lengths of one sequence, clamped so that every access stays in bounds (the merge kernel
// flags a value that had to be clamped).
struct Q8Keys {
    int pages;                   // sealed pages
    int64_t tail;                // tail rows
    int page_tiles, tiles;
};

template <int TILE>
__device__ __forceinline__ Q8Keys q8_keys(const AttnQ8Params& p, int b) {
    Q8Keys k;
    int pages = p.sealed_len[b] / kPageTokens;
    if (pages < 0) pages = 0;
    k.pages = pages > p.max_pages ? p.max_pages : pages;
    int64_t tail = p.tail_len[b];
    if (tail < 0) tail = 0;
    if (tail > p.cap - p.n_q) tail = p.cap - p.n_q;
    k.tail = tail;
    k.page_tiles = (k.pages + TILE / kPageTokens - 1) / (TILE / kPageTokens);
    k.tiles = k.page_tiles + (int)((tail + p.n_q + TILE - 1) / TILE);
    return k;
}

// Page id of block j of sequence b, clamped into the pool and flagged where it is outside.
__device__ __forceinline__ int q8_page(const AttnQ8Params& p, int b, int j) {
    const int id = p.page_table[(int64_t)b * p.max_pages + j];
    if (id >= 0 && id < p.n_pages) return id;
    if (p.err) atomicOr(p.err, kErrBadInput);
    return 0;
}

struct Q8Split {
    int b;               // sequence, or -1 where the slot has no work
    int t_begin, t_end;  // its tiles
    int first, count;    // slots of the sequence's splits
};

// The (sequence, split) of slot c, worked out by one whole warp from the device-side
// lengths: the smallest number of tiles per split whose splits fit into the S slots, so
// that short and long sequences of a ragged batch finish together.  Lanes take sequences
// lane, lane + 32, ..., so a large batch costs B / 32 reads a round.
template <int TILE>
static __device__ __noinline__ Q8Split q8_split_of_many(const AttnQ8Params& p, int c) {
    const int lane = threadIdx.x & 31;
    const int mine = lane < p.B ? q8_keys<TILE>(p, lane).tiles : 0;   // of the first 32 sequences
    auto tiles_of = [&](int b) { return b == lane ? mine : q8_keys<TILE>(p, b).tiles; };
    int total = 0, longest = 1;
#pragma unroll 1
    for (int b = lane; b < p.B; b += 32) {
        const int t = tiles_of(b);
        total += t;
        longest = t > longest ? t : longest;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    longest = __reduce_max_sync(0xffffffffu, longest);
    int lo = (total + p.S - 1) / p.S;
    if (lo < 1) lo = 1;
    // sum of ceil(t / m) <= (total - B) / m + B, so this many tiles are enough
    int hi = longest > lo ? longest : lo;
    if (p.S > p.B) {
        const int enough = (total - p.B + p.S - p.B - 1) / (p.S - p.B);
        hi = enough < lo ? lo : enough < hi ? enough : hi;
    }
#pragma unroll 1
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        int used = 0;
#pragma unroll 1
        for (int b = lane; b < p.B; b += 32) used += (tiles_of(b) + mid - 1) / mid;
        used = __reduce_add_sync(0xffffffffu, used);
        if (used <= p.S) hi = mid; else lo = mid + 1;
    }
    int first = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        const int tiles = b < p.B ? tiles_of(b) : 0;
        const int n = (tiles + lo - 1) / lo;
        int end = n;                                  // inclusive scan over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, c < first + end);
        if (hit) {
            const int w = __ffs(hit) - 1;
            const int count = __shfl_sync(0xffffffffu, n, w);
            const int f = first + __shfl_sync(0xffffffffu, end, w) - count;
            const int t0 = (c - f) * lo;              // below the sequence's tiles: count is tiles / lo, up
            return Q8Split{b0 + w, t0, min(t0 + lo, __shfl_sync(0xffffffffu, tiles, w)), f, count};
        }
        first += __shfl_sync(0xffffffffu, end, 31);
    }
    return Q8Split{-1, 0, 0, 0, 0};
}

// The same with the sequence's lengths; one sequence needs no search.
template <int TILE>
__device__ __forceinline__ Q8Split q8_split_of(const AttnQ8Params& p, int c, Q8Keys* keys) {
    Q8Split sp{0, 0, 0, 0, 0};
    if (p.B > 1) sp = q8_split_of_many<TILE>(p, c);
    *keys = q8_keys<TILE>(p, sp.b < 0 ? 0 : sp.b);
    if (p.B == 1) {
        const int budget = (keys->tiles + p.S - 1) / p.S;
        sp.t_begin = c * budget;
        sp.t_end = min(sp.t_begin + budget, keys->tiles);
        sp.count = (keys->tiles + budget - 1) / budget;
        if (c >= sp.count) sp.b = -1;
    }
    return sp;
}

// Group rows that one CTA of the history kernels takes.
constexpr int kQ8SimtRows = 64;
constexpr int kQ8TcRows = 128;
__host__ __device__ __forceinline__ int q8_row_blocks(int R) { return (R + kQ8TcRows - 1) / kQ8TcRows; }

cudaError_t launch_attn_q8_tc(const AttnQ8Params& p, cudaStream_t s);   // bf16
cudaError_t launch_attn_q8_simt(const AttnQ8Params& p, cudaStream_t s); // fp32
cudaError_t launch_attn_q8_merge(const AttnQ8Params& p, int dtype, cudaStream_t s);

}  // namespace rapid
