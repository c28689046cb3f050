// Verify attention over an 8-bit history on CUDA cores (fp32 queries and tails), and the
// merge of the partials of either history kernel.
//
// Pages hold x = code * scale, so a page's scores are scale_K (q . code) and its part of the
// output scale_V sum p code; both are applied to the values as they are unpacked.  One pass
// with the running maximum and sum of the softmax, in the log2 domain and fp32.
//
// The history kernel is bound by the CUDA cores' fp32 products and, on short histories, by the
// latency of a tile's loads, unpacking and two barriers.  Tiles are half a page, a key for each
// lane, so that a short history still splits over many CTAs: 5 queries of 4 heads over one KV
// head, d = 64, 1K of history takes 19.5 us, with tiles of 128 keys 33.6.
#include <cuda_fp16.h>

#include "attn_q8.cuh"
#include "common.cuh"

namespace rapid {

namespace {

constexpr int kSimtThreads = 128;                   // 4 warps
constexpr int kRowsPerWarp = kQ8SimtRows / 4;
constexpr int kKeys = kQ8SimtTile;                  // keys of a tile, one per lane

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 16 elements of a page row, scaled.
__device__ __forceinline__ void load_page16(const uint8_t* src, float scale, float (&x)[16]) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = e4m3x2_to_float2(w[i] & 0xffffu), c = e4m3x2_to_float2(w[i] >> 16);
        x[4 * i] = a.x * scale;
        x[4 * i + 1] = a.y * scale;
        x[4 * i + 2] = c.x * scale;
        x[4 * i + 3] = c.y * scale;
    }
}

__device__ __forceinline__ void load_row16(const float* src, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = reinterpret_cast<const float4*>(src)[i];
        x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
    }
}
// CTA = (slot and block of up to 64 group rows, KV head).  Each lane owns one key of a
// 32-key step for the scores and d / 32 output columns for the products with V.
template <int D>
__global__ void __launch_bounds__(kSimtThreads) attn_q8_simt_kernel(const AttnQ8Params p) {
    constexpr int DP = D + 4;                 // padded K pitch: conflict-free float4 rows
    constexpr int NC = D / 32;                // output columns per lane
    extern __shared__ float4 smem_f4[];
    float* sQ = reinterpret_cast<float*>(smem_f4);   // [64][D], times scale * log2(e)
    float* sK = sQ + kQ8SimtRows * D;                // [32][DP]
    float* sV = sK + kKeys * DP;                     // [32][D]
    __shared__ Q8Split s_split;
    __shared__ Q8Keys s_keys;

    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_rb = (p.R + kQ8SimtRows - 1) / kQ8SimtRows;
    const int slot_idx = blockIdx.x / n_rb, rb = blockIdx.x - slot_idx * n_rb;
    const int g = blockIdx.y;
    if (warp == 0) {
        Q8Keys k;
        const Q8Split sp = q8_split_of<kQ8SimtTile>(p, slot_idx, &k);
        if (lane == 0) {
            s_split = sp;
            s_keys = k;
        }
    }
    __syncthreads();
    const Q8Split sp = s_split;
    if (sp.b < 0) return;
    const int b = sp.b;
    const int64_t bg = (int64_t)b * p.Hkv + g;
    if (threadIdx.x == 0 && sp.s == 0 && rb == 0) {
        p.part_first[bg] = sp.first;
        p.part_count[bg] = sp.count;
    }
    const Q8Keys keys = s_keys;
    const int t_begin = (int)((int64_t)sp.s * keys.tiles / sp.count);
    const int t_end = (int)((int64_t)(sp.s + 1) * keys.tiles / sp.count);
    const int r0 = rb * kQ8SimtRows;
    const int nrows = min(kQ8SimtRows, p.R - r0);

    const float* Qg = static_cast<const float*>(p.Q) + ((int64_t)b * p.Hq + (int64_t)g * p.G) * p.n_q * D;
    for (int idx = threadIdx.x; idx < kQ8SimtRows * D; idx += kSimtThreads) {
        const int r = idx / D, k = idx - r * D;
        sQ[idx] = r < nrows ? Qg[(int64_t)(r0 + r) * D + k] * p.scale_log2 : 0.f;
    }
    float acc[kRowsPerWarp][NC];
    float m[kRowsPerWarp], l[kRowsPerWarp];
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[i][c] = 0.f;
    }
    const float* Kh = static_cast<const float*>(p.K) + bg * p.cap * D;
    const float* Vh = static_cast<const float*>(p.V) + bg * p.cap * D;
    const int64_t tail_keys = keys.tail + p.n_q;

    for (int tile = t_begin; tile < t_end; ++tile) {
        // key of lane 0: a page key, or a tail row once the page tiles are through
        const bool paged = tile < keys.page_tiles;
        const int64_t k0 = (int64_t)(paged ? tile : tile - keys.page_tiles) * kKeys;
        const int64_t k_end = paged ? (int64_t)keys.pages * kPageTokens : tail_keys;
        const int nk = (int)(k_end - k0 < kKeys ? k_end - k0 : kKeys);
        int64_t head = 0;                      // (page, head): one page holds the whole tile
        if (paged) head = (int64_t)q8_page(p, b, (int)(k0 / kPageTokens)) * p.Hkv + g;
        __syncthreads();
        for (int idx = threadIdx.x; idx < kKeys * (D / 16); idx += kSimtThreads) {
            const int key = idx / (D / 16), e = (idx - key * (D / 16)) * 16;
            float x[16], y[16];
            if (key >= nk) {
#pragma unroll
                for (int u = 0; u < 16; ++u) { x[u] = 0.f; y[u] = 0.f; }
            } else if (paged) {
                const int64_t row = k0 % kPageTokens + key;
                load_page16(p.pages + (head * 2 * kPageTokens + row) * D + e, p.scales[head * 2], x);
                load_page16(p.pages + ((head * 2 + 1) * kPageTokens + row) * D + e,
                            p.scales[head * 2 + 1], y);
            } else {
                load_row16(Kh + (k0 + key) * D + e, x);
                load_row16(Vh + (k0 + key) * D + e, y);
            }
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                sK[key * DP + e + u] = x[u];
                sV[key * D + e + u] = y[u];
            }
        }
        __syncthreads();
        const int64_t node = paged ? -1 : k0 + lane - keys.tail;   // speculative node of this lane's key
        float sc[kRowsPerWarp];
#pragma unroll
        for (int i = 0; i < kRowsPerWarp; ++i) sc[i] = 0.f;
#pragma unroll 4
        for (int k = 0; k < D; k += 4) {
            const float4 kv = *reinterpret_cast<const float4*>(&sK[lane * DP + k]);
#pragma unroll
            for (int i = 0; i < kRowsPerWarp; ++i) {
                const int r = warp + 4 * i;
                if (r < nrows) {
                    const float4 qv = *reinterpret_cast<const float4*>(&sQ[r * D + k]);
                    sc[i] = fmaf(qv.x, kv.x, sc[i]);
                    sc[i] = fmaf(qv.y, kv.y, sc[i]);
                    sc[i] = fmaf(qv.z, kv.z, sc[i]);
                    sc[i] = fmaf(qv.w, kv.w, sc[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRowsPerWarp; ++i) {
            const int r = warp + 4 * i;
            if (r >= nrows) continue;
            bool seen = lane < nk;
            if (node >= 0 && seen) {
                const int iq = (r0 + r) % p.n_q;
                seen = p.mask ? p.mask[((int64_t)b * p.n_q + iq) * p.n_q + node] != 0 : node <= iq;
            }
            const float si = seen ? sc[i] : -INFINITY;
            const float mnew = fmaxf(m[i], warp_max(si));
            // a row that has seen no key yet keeps p = 0 instead of exp(-inf + inf)
            const float ref = mnew == -INFINITY ? 0.f : mnew;
            const float corr = exp2f(m[i] - ref);
            const float pj = exp2f(si - ref);
            l[i] = l[i] * corr + warp_sum(pj);
            m[i] = mnew;
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[i][c] *= corr;
            sc[i] = pj;
        }
        for (int j = 0; j < nk; ++j) {
            float vv[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) vv[c] = sV[j * D + lane + 32 * c];
#pragma unroll
            for (int i = 0; i < kRowsPerWarp; ++i) {
                if (warp + 4 * i >= nrows) break;
                const float pj = __shfl_sync(0xffffffffu, sc[i], j);
                if (pj == 0.f) continue;       // a hidden row's V may hold anything
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[i][c] = fmaf(pj, vv[c], acc[i][c]);
            }
        }
    }
    const int64_t slot = ((int64_t)g * p.S + slot_idx) * p.R;
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        const int r = warp + 4 * i;
        if (r >= nrows) continue;
        float* dst = p.part_acc + (slot + r0 + r) * D;
#pragma unroll
        for (int c = 0; c < NC; ++c) dst[lane + 32 * c] = acc[i][c];
        if (lane == 0)
            *reinterpret_cast<float2*>(p.part_ml + (slot + r0 + r) * 2) = make_float2(m[i], l[i]);
    }
}

// One CTA of 128 threads per query row:
//   M = max m_s;  L = sum l_s 2^(m_s - M);  O = sum acc_s 2^(m_s - M) / L;
//   LSE = (M + log2 L) ln 2,
// over the splits s of the row's sequence.  Warps split the partials, lanes the d columns.
// Bound by latency: (m, l), the weights and the partial rows follow one another, about 4 us
// behind the history kernel; the first 32 partial rows are fetched before the weights are known.
constexpr int kMergeThreads = 128;
constexpr int kMergeMaxS = 1024;

template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) attn_q8_merge_kernel(const AttnQ8Params p) {
    constexpr int VPL = D / 32;                 // columns per lane
    constexpr int kPre = 8;                     // partial rows per warp held in registers
    __shared__ float s_w[kMergeMaxS];           // weights 2^(m_s - M)
    __shared__ float2 s_ml[kMergeMaxS];
    __shared__ float s_red[4][D];
    __shared__ float s_scal[4][2];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = blockIdx.x;
    const int bg = blockIdx.y;
    const int b = bg / p.Hkv, g = bg - b * p.Hkv;
    const int h = g * p.G + r / p.n_q, i = r % p.n_q;
    if (tid == 0 && g == 0 && r == 0 && p.err) {   // the lengths that the host cannot check
        const int64_t S = p.sealed_len[b], P = p.tail_len[b];
        if (S < 0 || S % kPageTokens || S / kPageTokens > p.max_pages || P < 0 || P > p.cap - p.n_q)
            atomicOr(p.err, kErrBadInput);
    }
    const int count = min(p.part_count[bg], kMergeMaxS);
    const int64_t first = (int64_t)g * p.S + p.part_first[bg];
    const float* ml = p.part_ml + (first * p.R + r) * 2;
    const float* pa = p.part_acc + (first * p.R + r) * D + lane * VPL;
    const int64_t mls = (int64_t)p.R * 2, pas = (int64_t)p.R * D;

    // the first partial rows on their way while (m, l) are reduced
    float v[kPre][VPL];
#pragma unroll
    for (int u = 0; u < kPre; ++u) {
        const int s = warp + 4 * u;
#pragma unroll
        for (int c = 0; c < VPL; ++c) v[u][c] = s < count ? pa[s * pas + c] : 0.f;
    }
    float top = -INFINITY;
    for (int s = tid; s < count; s += kMergeThreads) {
        const float2 x = *reinterpret_cast<const float2*>(ml + s * mls);
        s_ml[s] = x;
        if (x.y != 0.f) top = fmaxf(top, x.x);  // a NaN sum counts: it is the row's result
    }
    top = warp_max(top);
    if (lane == 0) s_scal[warp][0] = top;
    __syncthreads();
    const float M = fmaxf(fmaxf(s_scal[0][0], s_scal[1][0]), fmaxf(s_scal[2][0], s_scal[3][0]));
    float sum = 0.f;
    for (int s = tid; s < count; s += kMergeThreads) {
        const float2 x = s_ml[s];
        const float w = x.y != 0.f ? exp2f(x.x - M) : 0.f;
        s_w[s] = w;
        sum = fmaf(w, x.y, sum);
    }
    sum = warp_sum(sum);
    if (lane == 0) s_scal[warp][1] = sum;
    __syncthreads();
    const float L = (s_scal[0][1] + s_scal[1][1]) + (s_scal[2][1] + s_scal[3][1]);
    float acc[VPL];
#pragma unroll
    for (int c = 0; c < VPL; ++c) acc[c] = 0.f;
#pragma unroll
    for (int u = 0; u < kPre; ++u) {
        const int s = warp + 4 * u;
        const float w = s < count ? s_w[s] : 0.f;
#pragma unroll
        for (int c = 0; c < VPL; ++c) acc[c] = fmaf(w, w != 0.f ? v[u][c] : 0.f, acc[c]);
    }
    for (int s = warp + 4 * kPre; s < count; s += 4) {
        const float w = s_w[s];
        if (w == 0.f) continue;
#pragma unroll
        for (int c = 0; c < VPL; ++c) acc[c] = fmaf(w, pa[s * pas + c], acc[c]);
    }
#pragma unroll
    for (int c = 0; c < VPL; ++c) s_red[warp][lane * VPL + c] = acc[c];
    __syncthreads();
    if (warp != 0) return;
    const int64_t row = ((int64_t)b * p.Hq + h) * p.n_q + i;
    T* Orow = static_cast<T*>(p.O) + row * D;
    const float inv = L != 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (int c = 0; c < VPL; ++c) {
        const int col = lane * VPL + c;
        Orow[col] = from_float<T>(((s_red[0][col] + s_red[1][col]) + (s_red[2][col] + s_red[3][col])) * inv);
    }
    if (lane == 0) p.LSE[row] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

template <int D>
cudaError_t simt_typed(const AttnQ8Params& p, cudaStream_t st) {
    const int smem = (kQ8SimtRows * D + kKeys * (D + 4) + kKeys * D) * (int)sizeof(float);
    auto kern = attn_q8_simt_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int n_rb = (p.R + kQ8SimtRows - 1) / kQ8SimtRows;
    kern<<<dim3(p.S * n_rb, p.Hkv, 1), kSimtThreads, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t merge_typed(const AttnQ8Params& p, cudaStream_t st) {
    if (p.S - p.B + 1 > kMergeMaxS) return cudaErrorNotSupported;   // splits of one sequence
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.R, p.B * p.Hkv, 1);
    cfg.blockDim = dim3(kMergeThreads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_q8_merge_kernel<T, D>, p);
}

}  // namespace

cudaError_t launch_attn_q8_simt(const AttnQ8Params& p, cudaStream_t s) {
    return p.d == 128 ? simt_typed<128>(p, s) : simt_typed<64>(p, s);
}

cudaError_t launch_attn_q8_merge(const AttnQ8Params& p, int dtype, cudaStream_t s) {
    if (dtype == 1)
        return p.d == 128 ? merge_typed<__nv_bfloat16, 128>(p, s) : merge_typed<__nv_bfloat16, 64>(p, s);
    return p.d == 128 ? merge_typed<float, 128>(p, s) : merge_typed<float, 64>(p, s);
}

}  // namespace rapid
