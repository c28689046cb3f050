// Expanded attention of a prompt chunk: keys of 128 values for each head and 64 that all heads
// share, values of 128, causal behind a prefix.
//
//   s_ij = <q_i, [k_j, r_j]>,   O_i = sum_{j <= prefix + i} softmax(scale s_i)_j v_j
//
// One warp per query; a lane holds 4 + 2 values of the query and 4 of the output.
#include "common.cuh"
#include "latent.cuh"

namespace rapid {

namespace {

__global__ void __launch_bounds__(128) latent_prefill_kernel(const LatentPrefillParams p) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);   // (b, i, h)
    if (unit >= (int64_t)p.B * p.n * p.H) return;
    const int h = (int)(unit % p.H), i = (int)(unit / p.H % p.n), b = (int)(unit / p.H / p.n);
    const int count = p.n_rows ? p.n_rows[b] : p.n;
    const int64_t P = p.prefix_len[b];
    if (count < 0 || count > p.n || P < 0 || P + count > p.kv_rows) {
        if (lane == 0 && i == 0 && h == 0 && p.err) atomicOr(p.err, kErrBadInput);
        return;
    }
    if (i >= count) return;
    auto two = [](const __nv_bfloat16* x) { return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(x)); };
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.Q) + b * p.q_stride[0] + i * p.q_stride[1] + h * p.q_stride[2];
    const __nv_bfloat16* K = static_cast<const __nv_bfloat16*>(p.K) + b * p.k_stride[0] + h * p.k_stride[2];
    const __nv_bfloat16* V = static_cast<const __nv_bfloat16*>(p.V) + b * p.v_stride[0] + h * p.v_stride[2];
    const __nv_bfloat16* R = static_cast<const __nv_bfloat16*>(p.K_rope) + b * p.r_stride[0];
    const float2 q0 = two(q + 4 * lane), q1 = two(q + 4 * lane + 2), q2 = two(q + 128 + 2 * lane);
    float a0 = 0, a1 = 0, a2 = 0, a3 = 0, m = -INFINITY, l = 0.f;
    for (int64_t j = 0; j <= P + i; ++j) {
        const __nv_bfloat16* k = K + j * p.k_stride[1];
        const float2 k0 = two(k + 4 * lane), k1 = two(k + 4 * lane + 2), k2 = two(R + j * p.r_stride[1] + 2 * lane);
        float s = q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y + q2.x * k2.x + q2.y * k2.y;
        s = warp_sum(s) * p.scale_log2;
        const float mn = fmaxf(m, s), corr = m == -INFINITY ? 0.f : exp2f(m - mn);
        const float w = s == -INFINITY ? 0.f : exp2f(s - mn);
        m = mn;
        l = l * corr + w;
        const __nv_bfloat16* v = V + j * p.v_stride[1];
        const float2 v0 = two(v + 4 * lane), v1 = two(v + 4 * lane + 2);
        a0 = a0 * corr + w * v0.x; a1 = a1 * corr + w * v0.y;
        a2 = a2 * corr + w * v1.x; a3 = a3 * corr + w * v1.y;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(
        static_cast<__nv_bfloat16*>(p.O) + (((int64_t)b * p.n + i) * p.H + h) * 128 + 4 * lane);
    o[0] = __floats2bfloat162_rn(a0 * inv, a1 * inv);
    o[1] = __floats2bfloat162_rn(a2 * inv, a3 * inv);
    if (lane == 0) p.LSE[((int64_t)b * p.H + h) * p.n + i] = (m + log2f(l)) * kLn2;
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillParams& p, cudaStream_t st) {
    latent_prefill_kernel<<<(unsigned)(((int64_t)p.B * p.n * p.H + 3) / 4), 128, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace rapid
