// Absorbed attention over a latent cache: verify attention whose keys are the cache rows (576
// values, one row for all heads) and whose values are their first 512.
//
//   s_j = <q, [c_j, r_j]>,   O = sum_j softmax(scale s)_j c_j
//
// over the history rows and, as the chain or tree mask says, the n_q rows behind them.
// One block per query; its warps take keys in turn, a lane holds 18 values of the query and 16
// of the output.
#include <cuda_fp8.h>

#include "common.cuh"
#include "latent.cuh"

namespace rapid {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

RAPID_DEVICE void unpack8(uint4 r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__global__ void __launch_bounds__(kThreads) latent_attn_kernel(const LatentAttnParams p) {
    __shared__ float s_acc[kWarps][kLatent];
    __shared__ float s_m[kWarps], s_l[kWarps];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;                  // (b, h, i)
    const int i = (int)(row % p.n_q);
    const int b = (int)(row / p.n_q / p.H);
    int64_t P = p.prefix_len[b];
    if (P < 0 || P > p.cap - p.n_q) {
        if (threadIdx.x == 0 && p.err) atomicOr(p.err, kErrBadInput);
        P = P < 0 ? 0 : p.cap - p.n_q;
    }
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.Q) + row * kLatentRow;
    float qv[18], acc[16], m = -INFINITY, l = 0.f;
    unpack8(reinterpret_cast<const uint4*>(q)[2 * lane], qv);
    unpack8(reinterpret_cast<const uint4*>(q)[2 * lane + 1], qv + 8);
    qv[16] = __bfloat162float(q[kLatent + 2 * lane]);
    qv[17] = __bfloat162float(q[kLatent + 2 * lane + 1]);
#pragma unroll
    for (int u = 0; u < 16; ++u) acc[u] = 0.f;
    const int rb = p.q8 ? kLatentQ8Row : 2 * kLatentRow;
    for (int64_t j = warp; j < P + p.n_q; j += kWarps) {
        if (j >= P) {
            const int jj = (int)(j - P);
            if (p.mask ? p.mask[((int64_t)b * p.n_q + i) * p.n_q + jj] == 0 : jj > i) continue;
        }
        const uint8_t* kr = p.cache + ((int64_t)b * p.cap + j) * rb;
        float k[18];
        if (p.q8) {
            const float scale = reinterpret_cast<const float*>(kr + kLatentQ8Scale)[lane >> 3];
            const uint4 c = reinterpret_cast<const uint4*>(kr)[lane];
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const __half_raw h = __nv_cvt_fp8_to_halfraw((w[u / 4] >> (8 * (u % 4))) & 0xff, __NV_E4M3);
                k[u] = __half2float(*reinterpret_cast<const __half*>(&h)) * scale;
            }
        } else {
            unpack8(reinterpret_cast<const uint4*>(kr)[2 * lane], k);
            unpack8(reinterpret_cast<const uint4*>(kr)[2 * lane + 1], k + 8);
        }
        const __nv_bfloat16* rope = reinterpret_cast<const __nv_bfloat16*>(kr + (p.q8 ? kLatentQ8Rope : 2 * kLatent));
        k[16] = __bfloat162float(rope[2 * lane]);
        k[17] = __bfloat162float(rope[2 * lane + 1]);
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < 18; ++u) s = fmaf(qv[u], k[u], s);
        s = warp_sum(s) * p.scale_log2;
        const float mn = fmaxf(m, s), corr = m == -INFINITY ? 0.f : exp2f(m - mn);
        const float w = s == -INFINITY ? 0.f : exp2f(s - mn);
        m = s != s ? s : mn;
        l = l * corr + w;
#pragma unroll
        for (int u = 0; u < 16; ++u) acc[u] = fmaf(w, k[u], acc[u] * corr);
    }
#pragma unroll
    for (int u = 0; u < 16; ++u) s_acc[warp][16 * lane + u] = acc[u];
    if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
    float f[kWarps];
    for (int w = 0; w < kWarps; ++w) {
        f[w] = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - M);
        L += s_l[w] * f[w];
    }
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.O) + row * kLatent;
    for (int c = threadIdx.x; c < kLatent; c += kThreads) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w) x += f[w] * s_acc[w][c];
        o[c] = __float2bfloat16_rn(M == -INFINITY ? 0.f : x / L);
    }
    if (threadIdx.x == 0) p.LSE[row] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * kLn2;
}

}  // namespace

cudaError_t launch_latent_attn(const LatentAttnParams& p, cudaStream_t st) {
    latent_attn_kernel<<<(unsigned)((int64_t)p.B * p.H * p.n_q), kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace rapid
