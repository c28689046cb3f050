// Verify attention over an 8-bit history on CUDA cores (fp32 queries and tails), and the
// merge of the partials of either history kernel.
//
// Pages hold x = code * scale, so a page's scores are scale_K (q . code) and its part of the
// output scale_V sum p code; both are applied to the values as they are unpacked.  One pass
// with the running maximum and sum of the softmax, in the log2 domain and fp32.
//
// The history kernel is bound by the CUDA cores and shared memory (two packed products, or one
// 16-byte read of K, V or P, for 4 to 8 multiplications), on short histories by the latency of
// a tile: unpacking, two barriers, the two products one after the other.  Measured with the merge:
// 5 queries of 4 heads over one KV head, d = 64, 1K of history 7.8 us; 10 queries of 16 heads,
// d = 64, six histories of 1.6K 39 us; 60 queries of 64 heads over 8, d = 128, 512 of history 66 us.
// With a key to a lane, rows over the warps and P handed round by shuffles these took 19.4, 206
// and 183.
#include <cuda_fp16.h>

#include "attn_q8.cuh"
#include "common.cuh"

namespace rapid {

namespace {

constexpr int kSimtThreads = 256;
constexpr int kKeys = kQ8SimtTile;                  // keys of a tile: a page, or 64 tail rows
static_assert(kKeys == kPageTokens, "a tile is a page");

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four codes, scaled.
__device__ __forceinline__ float4 page4(uint32_t w, float scale) {
    const float2 a = e4m3x2_to_float2(w & 0xffffu), c = e4m3x2_to_float2(w >> 16);
    return make_float4(a.x * scale, a.y * scale, c.x * scale, c.y * scale);
}

// CTA = (slot and block of up to 64 group rows, KV head).  A tile is unpacked into shared
// memory while the next page's codes are on their way into registers.  16 lanes own TR rows
// (tr + 16 i) in both products: 4 keys each of the scores, d / 16 columns each of the output, so
// that P and the running maxima never leave the warp.
template <int D, int TR>
__global__ void __launch_bounds__(kSimtThreads, TR == 4 ? 1 : 2) attn_q8_simt_kernel(const AttnQ8Params p) {
    constexpr int ROWS = 16 * TR;
    constexpr int KP = D + 4;                 // pitches of K and P: conflict-free
    constexpr int PP = kKeys + 4;
    constexpr int W = kKeys * D / 4 / kSimtThreads;   // words of codes a thread holds, each side
    constexpr int NV = D / 64;                // float4 columns per lane: 4 kg + 64 h
    extern __shared__ float4 smem_f4[];
    float* sQ = reinterpret_cast<float*>(smem_f4);   // [ROWS][D], times scale * log2(e)
    float* sK = sQ + ROWS * D;                       // [64][KP]
    float* sV = sK + kKeys * KP;                     // [64][D]
    float* sP = sV + kKeys * D;                      // [ROWS][PP]
    __shared__ Q8Split s_split;
    __shared__ Q8Keys s_keys;

    griddep_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kg = tid & 15, tr = tid >> 4;
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
    if (tid == 0 && sp.t_begin == 0 && rb == 0) {
        p.part_first[bg] = sp.first;
        p.part_count[bg] = sp.count;
    }
    const Q8Keys keys = s_keys;
    const int t_begin = sp.t_begin, t_end = sp.t_end;
    const int r0 = rb * kQ8SimtRows;
    const int nrows = min(kQ8SimtRows, p.R - r0);

    const float4* Qg = reinterpret_cast<const float4*>(
        static_cast<const float*>(p.Q) + (((int64_t)b * p.Hq + (int64_t)g * p.G) * p.n_q + r0) * D);
    for (int x = tid; x < ROWS * D / 4; x += kSimtThreads) {
        float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < nrows * (D / 4)) q = Qg[x];
        reinterpret_cast<float4*>(sQ)[x] =
            make_float4(q.x * p.scale_log2, q.y * p.scale_log2, q.z * p.scale_log2, q.w * p.scale_log2);
    }
    float2 acc[TR][2 * NV];
    float m[TR], l[TR];                       // l: this lane's keys only
#pragma unroll
    for (int i = 0; i < TR; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < 2 * NV; ++c) acc[i][c] = make_float2(0.f, 0.f);
    }
    const float* Kh = static_cast<const float*>(p.K) + bg * p.cap * D;
    const float* Vh = static_cast<const float*>(p.V) + bg * p.cap * D;
    const int64_t tail_keys = keys.tail + p.n_q;

    uint32_t kc[W], vc[W];                    // a page's codes, and its scales
    float k_scale = 0.f, v_scale = 0.f;
    auto fetch = [&](int tile) {
        const int64_t head = (int64_t)q8_page(p, b, tile) * p.Hkv + g;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.pages + head * 2 * kPageTokens * D);
#pragma unroll
        for (int u = 0; u < W; ++u) {
            kc[u] = __ldg(src + u * kSimtThreads + tid);
            vc[u] = __ldg(src + kPageTokens * D / 4 + u * kSimtThreads + tid);
        }
        k_scale = __ldg(p.scales + head * 2);
        v_scale = __ldg(p.scales + head * 2 + 1);
    };
    if (t_begin < t_end && t_begin < keys.page_tiles) fetch(t_begin);

#pragma unroll 1
    for (int tile = t_begin; tile < t_end; ++tile) {
        const bool paged = tile < keys.page_tiles;
        const int64_t k0 = (int64_t)(tile - keys.page_tiles) * kKeys;   // tail tile's first row
        __syncthreads();
        if (paged) {
#pragma unroll
            for (int u = 0; u < W; ++u) {
                const int x = u * kSimtThreads + tid, key = x / (D / 4), c = x - key * (D / 4);
                *reinterpret_cast<float4*>(sK + key * KP + 4 * c) = page4(kc[u], k_scale);
                *reinterpret_cast<float4*>(sV + key * D + 4 * c) = page4(vc[u], v_scale);
            }
            if (tile + 1 < t_end && tile + 1 < keys.page_tiles) fetch(tile + 1);
        } else {
#pragma unroll 2
            for (int x = tid; x < kKeys * D / 4; x += kSimtThreads) {
                const int key = x / (D / 4), c = x - key * (D / 4);
                float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
                if (k0 + key < tail_keys) {
                    kv = *reinterpret_cast<const float4*>(Kh + (k0 + key) * D + 4 * c);
                    vv = *reinterpret_cast<const float4*>(Vh + (k0 + key) * D + 4 * c);
                }
                *reinterpret_cast<float4*>(sK + key * KP + 4 * c) = kv;
                *reinterpret_cast<float4*>(sV + key * D + 4 * c) = vv;
            }
        }
        __syncthreads();
        if (2 * warp >= nrows) continue;      // no row in this warp
        float2 s2[TR][4];
#pragma unroll
        for (int i = 0; i < TR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
        for (int k = 0; k < D; k += 4) {
            float4 kv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(sK + (kg + 16 * j) * KP + k);
#pragma unroll
            for (int i = 0; i < TR; ++i) {
                const float4 q = *reinterpret_cast<const float4*>(sQ + (tr + 16 * i) * D + k);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s2[i][j] = fma2(make_float2(q.x, q.y), make_float2(kv[j].x, kv[j].y), s2[i][j]);
                    s2[i][j] = fma2(make_float2(q.z, q.w), make_float2(kv[j].z, kv[j].w), s2[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < TR; ++i) {
            const int r = tr + 16 * i;
            float s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = s2[i][j].x + s2[i][j].y;
            if (!paged) {
                const int iq = (r0 + min(r, nrows - 1)) % p.n_q;
                const uint8_t* seen = p.mask ? p.mask + ((int64_t)b * p.n_q + iq) * p.n_q : nullptr;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t key = k0 + kg + 16 * j, node = key - keys.tail;
                    if (key >= tail_keys || (node >= 0 && !(seen ? seen[node] != 0 : node <= iq))) s[j] = -INFINITY;
                }
            }
            float top = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float mnew = fmaxf(m[i], top);
            // a row that has seen no key yet keeps p = 0 instead of exp(-inf + inf)
            const float ref = mnew == -INFINITY ? 0.f : mnew;
            const float corr = exp2f(m[i] - ref);
            m[i] = mnew;
            l[i] *= corr;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = exp2f(s[j] - ref);
                l[i] += e;
                sP[r * PP + kg + 16 * j] = e;
            }
#pragma unroll
            for (int c = 0; c < 2 * NV; ++c) acc[i][c] = mul2(acc[i][c], make_float2(corr, corr));
        }
        __syncwarp();
        const int j_end = paged ? kKeys : (int)min(tail_keys - k0, (int64_t)kKeys);
#pragma unroll 1
        for (int j0 = 0; j0 < j_end; j0 += 4) {
            float4 pr[TR];
#pragma unroll
            for (int i = 0; i < TR; ++i) pr[i] = *reinterpret_cast<const float4*>(sP + (tr + 16 * i) * PP + j0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float4 v[NV];
#pragma unroll
                for (int h = 0; h < NV; ++h)
                    v[h] = *reinterpret_cast<const float4*>(sV + (j0 + e) * D + 4 * kg + 64 * h);
#pragma unroll
                for (int i = 0; i < TR; ++i) {
                    const float w = e == 0 ? pr[i].x : e == 1 ? pr[i].y : e == 2 ? pr[i].z : pr[i].w;
                    if (!paged && w == 0.f) continue;   // a hidden row's V may hold anything
                    const float2 w2 = make_float2(w, w);
#pragma unroll
                    for (int h = 0; h < NV; ++h) {
                        acc[i][2 * h] = fma2(w2, make_float2(v[h].x, v[h].y), acc[i][2 * h]);
                        acc[i][2 * h + 1] = fma2(w2, make_float2(v[h].z, v[h].w), acc[i][2 * h + 1]);
                    }
                }
            }
        }
    }
    const int64_t slot = ((int64_t)g * p.S + slot_idx) * p.R;
#pragma unroll
    for (int i = 0; i < TR; ++i) {
        const int r = tr + 16 * i;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
        if (r >= nrows) continue;
        float* dst = p.part_acc + (slot + r0 + r) * D + 4 * kg;
#pragma unroll
        for (int h = 0; h < NV; ++h)
            *reinterpret_cast<float4*>(dst + 64 * h) =
                make_float4(acc[i][2 * h].x, acc[i][2 * h].y, acc[i][2 * h + 1].x, acc[i][2 * h + 1].y);
        if (kg == 0)
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

template <int D, int TR>
cudaError_t simt_rows(const AttnQ8Params& p, cudaStream_t st) {
    constexpr int smem = (16 * TR * D + kKeys * (D + 4) + kKeys * D + 16 * TR * (kKeys + 4)) * (int)sizeof(float);
    auto kern = attn_q8_simt_kernel<D, TR>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int n_rb = (p.R + kQ8SimtRows - 1) / kQ8SimtRows;
    kern<<<dim3(p.S * n_rb, p.Hkv, 1), kSimtThreads, smem, st>>>(p);
    return cudaGetLastError();
}
// As few rows a lane as hold the group.
template <int D>
cudaError_t simt_typed(const AttnQ8Params& p, cudaStream_t st) {
    if (p.R <= 16) return simt_rows<D, 1>(p, st);
    if (p.R <= 32) return simt_rows<D, 2>(p, st);
    return simt_rows<D, 4>(p, st);
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
