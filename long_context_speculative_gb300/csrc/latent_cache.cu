// Rows of a latent cache: append with norm, rotation and quantisation, read back, commit.
//
// Append: for each token, of the projection row [c, r] (512 and 64 values)
//   c := c / sqrt(mean(c^2) + eps) * w,   r := r rotated by the token's position,
// held as 576 bf16, or with each 128 values of c as e4m3 codes of one power of two
//   scale = 2^ceil(log2(max|c| / 448)),   code = e4m3(c / scale),
// and the 64 last values of every query head rotated by the same angles.  A power of two costs
// a floating-point code no precision, and dividing and multiplying by it is exact.  All
// arithmetic is fp32, rounded once at the store.
//
// Loads are coherent ones: a kernel may be there before its predecessor has ended, and read what that wrote
// once griddep_wait() has returned.
//
// All three kernels copy: no value is read twice.  A row is one warp's work: lane l holds values
// 16 l .. 16 l + 15 of the latent vector (a scale group is 8 lanes) and pair l of the key.
//
// Measured, calls back to back over inputs that do not stay in L2 (us; floor by bytes at 6788 GB/s): three ragged
// chunks of up to 4095 tokens with 32 heads 19.1 (14.2), 8-bit rows 19.2 (13.6), 15.4 where the 97 MB stay in L2
// (28 before the pairs' layout was a template parameter, when the lanes' registers were indexed in memory);
// 8192 tokens of 128 heads, 8-bit rows 50.4 (41.7); 11 tokens of 128 heads 2.1.  Reading a 120K history in
// 8 bits back 37.1 (32.7); committing 16 sequences' paths of 60 layers 9.8 (5.5), 6.0 where they stay in L2.
#include <cuda_fp8.h>

#include "common.cuh"
#include "latent.cuh"
#include "rope.cuh"

namespace rapid {

namespace {

RAPID_DEVICE void unpack8(uint4 r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
RAPID_DEVICE uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
RAPID_DEVICE uint4 pack8(const float* x) {
    return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}

template <typename K, typename P>
cudaError_t launch(K kern, dim3 grid, int threads, const P& p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

constexpr int kAppendThreads = 128;
constexpr int kAppendWarps = kAppendThreads / 32;

// One power of two for max: the smallest 2^e with max <= 448 * 2^e, e >= -64; 1 for zeros.
RAPID_DEVICE float group_scale(float amax) {
    if (!(amax > 0.f)) return 1.f;
    const uint32_t bits = __float_as_uint(amax);
    int e = (int)(bits >> 23) - 127 - 8;             // amax = m 2^(e + 8), 1 <= m < 2
    if ((bits & 0x7fffffu) > 0x600000u) ++e;         // m > 1.75 = 448 / 256
    if (e < -64) e = -64;                            // (a subnormal amax too)
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// The latent vector and the key of one token by one warp.
RAPID_DEVICE void append_row(const LatentAppendParams& p, int b, int i, int64_t pos, uint8_t* row,
                             int lane) {
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.kv) + b * p.kv_batch + i * p.kv_token;
    const uint4 r0 = reinterpret_cast<const uint4*>(src)[2 * lane];
    const uint4 r1 = reinterpret_cast<const uint4*>(src)[2 * lane + 1];
    const int ka = p.interleaved ? 2 * lane : lane, kb = p.interleaved ? 2 * lane + 1 : lane + 32;
    const float ra = __bfloat162float(src[kLatent + ka]), rb = __bfloat162float(src[kLatent + kb]);
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    if (p.weight) {
        w0 = static_cast<const uint4*>(p.weight)[2 * lane];
        w1 = static_cast<const uint4*>(p.weight)[2 * lane + 1];
    }
    float sn, cs;
    sincos_turn(turns_per_position(p.inv_freq[lane]), pos, &sn, &cs);
    float x[16];
    unpack8(r0, x);
    unpack8(r1, x + 8);
    if (p.weight) {
        // The squares are taken of c 2^-k, 2^k the size of the largest value or of sqrt(eps), so that
        // they stay in fp32's range whatever the row's size.
        float big = sqrtf(p.eps);
#pragma unroll
        for (int u = 0; u < 16; ++u) big = fmaxf(big, fabsf(x[u]));
        const int k = min((int)(__reduce_max_sync(0xffffffffu, __float_as_uint(big)) >> 23), 253) - 127;
        const float down = __uint_as_float((uint32_t)(127 - max(k, -126)) << 23);
        float ss = 0.f;
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            x[u] *= down;
            ss = fmaf(x[u], x[u], ss);
        }
        const float inv = rsqrtf(warp_sum(ss) * (1.f / kLatent) + p.eps * down * down);
        float w[16];
        unpack8(w0, w);
        unpack8(w1, w + 8);
#pragma unroll
        for (int u = 0; u < 16; ++u) x[u] = x[u] * inv * w[u];
    }
    __nv_bfloat16* rope = reinterpret_cast<__nv_bfloat16*>(row + (p.q8 ? kLatentQ8Rope : 2 * kLatent));
    rope[ka] = __float2bfloat16_rn(ra * cs - rb * sn);
    rope[kb] = __float2bfloat16_rn(rb * cs + ra * sn);
    if (!p.q8) {
        reinterpret_cast<uint4*>(row)[2 * lane] = pack8(x);
        reinterpret_cast<uint4*>(row)[2 * lane + 1] = pack8(x + 8);
        return;
    }
    // A value that is not finite makes its group NaN (by the scale): whoever attends to the row
    // gets NaN, as with the value itself.
    float amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        bad |= !isfinite(x[u]);
        amax = fmaxf(amax, fabsf(x[u]));
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const uint32_t bads = __ballot_sync(0xffffffffu, bad);
    bad = (bads >> (lane & 24)) & 0xff;
    const float scale = bad ? __int_as_float(0x7fffffff) : group_scale(amax);
    const float inv = bad ? 0.f : __uint_as_float((254u << 23) - __float_as_uint(scale));   // 2^-e, exact
    uint32_t c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[4 * u + 1] * inv), "f"(x[4 * u] * inv));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[4 * u + 3] * inv), "f"(x[4 * u + 2] * inv));
        c[u] = bad ? 0u : (uint32_t)lo | ((uint32_t)hi << 16);
    }
    reinterpret_cast<uint4*>(row)[lane] = make_uint4(c[0], c[1], c[2], c[3]);
    if ((lane & 7) == 0) reinterpret_cast<float*>(row + kLatentQ8Scale)[lane >> 3] = scale;
}

// Units of one warp: token * (slices + 1) + slice; slice `slices` is the token's cache row, the
// others share its query heads, 8 heads (4 lanes each) a step.
template <bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads) latent_append_kernel(const LatentAppendParams p) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    const int64_t token = unit / (p.slices + 1);
    const int slice = (int)(unit - token * (p.slices + 1));
    if (token >= (int64_t)p.B * p.n) return;
    const int b = (int)(token / p.n), i = (int)(token - (int64_t)b * p.n);
    const int count = p.n_rows ? p.n_rows[b] : p.n;
    const int64_t P = p.prefix_len[b];
    if (count < 0 || count > p.n || P < 0 || P + count > p.cap) {   // refused: left alone
        if (i == 0 && slice == p.slices && lane == 0 && p.err) atomicOr(p.err, kErrBadInput);
        return;
    }
    if (i >= count) return;
    const int64_t pos = P + (p.row_offset ? p.row_offset[(int64_t)b * p.n + i] : i);
    if (slice == p.slices) {
        append_row(p, b, i, pos, p.cache + ((int64_t)b * p.cap + P + i) * (p.q8 ? kLatentQ8Row : 2 * kLatentRow),
                   lane);
        return;
    }
    // Lane l % 4 of a head holds two pieces of 8 values: c and c + 4 (their elements rotate into
    // each other), or 2 c and 2 c + 1 (interleaved pairs stay inside a piece): pairs 8 c .. 8 c + 7
    // either way.  The 8 heads of a step share the angles: each works out one pair a lane.
    const int c = lane & 3, sub = lane >> 2;
    float my_sn, my_cs, sn[8], cs[8];
    sincos_turn(turns_per_position(p.inv_freq[8 * c + sub]), pos, &my_sn, &my_cs);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        sn[u] = __shfl_sync(0xffffffffu, my_sn, 4 * u + c);
        cs[u] = __shfl_sync(0xffffffffu, my_cs, 4 * u + c);
    }
    const int p0 = INTERLEAVED ? 2 * c : c, p1 = INTERLEAVED ? 2 * c + 1 : c + 4;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + b * p.q_batch + i * p.q_token;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.q_out) + b * p.o_batch + i * p.o_token;
    const int steps = (p.H + 7) / 8;
    auto load = [&](int it, uint4& r0, uint4& r1) {
        const int h = it * 8 + sub;
        r0 = r1 = make_uint4(0, 0, 0, 0);
        if (h >= p.H) return;
        const uint4* s = reinterpret_cast<const uint4*>(q + h * p.q_head);   // may be rewritten in place
        r0 = s[p0];
        r1 = s[p1];
    };
    auto finish = [&](int it, uint4 r0, uint4 r1) {
        const int h = it * 8 + sub;
        float x[16], y[16];
        unpack8(r0, x);
        unpack8(r1, x + 8);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int ia = INTERLEAVED ? 2 * u : u, ib = INTERLEAVED ? 2 * u + 1 : u + 8;
            y[u] = x[ia] * cs[u] - x[ib] * sn[u];
            y[u + 8] = x[ib] * cs[u] + x[ia] * sn[u];
        }
        if (h >= p.H) return;
        if (INTERLEAVED) {
#pragma unroll
            for (int u = 0; u < 8; ++u) { x[2 * u] = y[u]; x[2 * u + 1] = y[u + 8]; }
        } else {
#pragma unroll
            for (int u = 0; u < 16; ++u) x[u] = y[u];
        }
        uint4* d = reinterpret_cast<uint4*>(o + h * p.o_head);
        d[p0] = pack8(x);
        d[p1] = pack8(x + 8);
    };
    for (int it = slice; it < steps; it += 2 * p.slices) {   // two steps' loads in flight
        const int next = it + p.slices;
        uint4 r0, r1, n0, n1;
        load(it, r0, r1);
        if (next < steps) load(next, n0, n1);
        finish(it, r0, r1);
        if (next < steps) finish(next, n0, n1);
    }
}

// Read back: a warp takes four rows at a time, 16 codes (or 16 values) a lane and row.
constexpr int kReadRows = 4;

template <bool Q8>
__global__ void __launch_bounds__(128) latent_read_kernel(const LatentReadParams p) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int per = (p.n - 1) / kReadRows + 1;            // units of a sequence
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int b = (int)(unit / per);
    if (b >= p.B) return;
    const int i0 = (int)(unit - (int64_t)b * per) * kReadRows;
    const int count = p.n_rows ? p.n_rows[b] : p.n;
    const int64_t f = p.first ? p.first[b] : 0;
    if (count < 0 || count > p.n || f < 0 || f + count > p.cap) {   // refused: left alone
        if (i0 == 0 && lane == 0 && p.err) atomicOr(p.err, kErrBadInput);
        return;
    }
    constexpr int kRow = Q8 ? kLatentQ8Row : 2 * kLatentRow;
    const uint8_t* src = p.cache + ((int64_t)b * p.cap + f + i0) * kRow;
    uint8_t* dst = p.rows + ((int64_t)b * p.n + i0) * 2 * kLatentRow;
    const int m = min(kReadRows, count - i0);
    uint4 x[kReadRows], y[kReadRows], z[kReadRows];
    float scale[kReadRows];
#pragma unroll
    for (int r = 0; r < kReadRows; ++r) {
        if (r >= m) continue;
        const uint4* s = reinterpret_cast<const uint4*>(src + (int64_t)r * kRow);
        x[r] = s[lane];
        if (!Q8) y[r] = s[32 + lane];
        if (lane < 8) z[r] = s[(Q8 ? 32 : 64) + lane];
        if (Q8) scale[r] = reinterpret_cast<const float*>(s + kLatentQ8Scale / 16)[lane >> 3];
    }
#pragma unroll
    for (int r = 0; r < kReadRows; ++r) {
        if (r >= m) continue;
        uint4* d = reinterpret_cast<uint4*>(dst + (int64_t)r * 2 * kLatentRow);
        if (Q8) {
            const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
            float v[16];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const __half2_raw q = __nv_cvt_fp8x2_to_halfraw2(
                        (__nv_fp8x2_storage_t)(w[u] >> (16 * h)), __NV_E4M3);
                    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&q));
                    v[4 * u + 2 * h] = t.x * scale[r];
                    v[4 * u + 2 * h + 1] = t.y * scale[r];
                }
            }
            d[2 * lane] = pack8(v);
            d[2 * lane + 1] = pack8(v + 8);
        } else {
            d[lane] = x[r];
            d[32 + lane] = y[r];
        }
        if (lane < 8) d[64 + lane] = z[r];
    }
}

// Commit: thread c moves 16-byte column c of the accepted rows, in path order.  A path
// increases, so row 1 + k is never behind a source that is still to be read: no staging, and
// kMove rows are read before the first of them is written.
constexpr int kMove = 8;

__global__ void __launch_bounds__(96) latent_commit_kernel(const LatentCommitParams p) {
    __shared__ int s_src[64];
    __shared__ int s_flags;             // bit 0: invalid input, bit 1: some row moves
    griddep_wait();
    const int t = threadIdx.x, b = blockIdx.x, layer = blockIdx.y;
    const int n = p.n_acc[b];
    const int64_t P = p.prefix_len[b];
    if (t == 0) s_flags = n >= 0 && n <= p.n_q - 1 && P >= 0 && P + p.n_q <= p.cap ? 0 : 1;
    __syncthreads();
    const bool fits = (s_flags & 1) == 0;
    __syncthreads();
    if (fits && t < n) {
        const int src = p.path[(int64_t)b * p.n_q + t];
        const int prev = t > 0 ? p.path[(int64_t)b * p.n_q + t - 1] : 0;
        int f = 0;
        if (src < t + 1 || src > p.n_q - 1 || src <= prev) f |= 1;   // not a valid increasing path
        if (src != t + 1) f |= 2;
        s_src[t] = src;
        if (f) atomicOr(&s_flags, f);
    }
    __syncthreads();
    const int flags = s_flags;
    if (flags & 1) {
        if (t == 0 && layer == 0 && p.err) atomicOr(p.err, kErrBadInput);
        return;
    }
    if (!(flags & 2) || t >= p.row_bytes / 16) return;
    uint8_t* base = p.cache[layer] + ((int64_t)b * p.cap + P) * p.row_bytes + 16 * t;
    for (int k0 = 0; k0 < n; k0 += kMove) {
        uint4 x[kMove];
#pragma unroll
        for (int u = 0; u < kMove; ++u)
            if (k0 + u < n) x[u] = *reinterpret_cast<const uint4*>(base + (int64_t)s_src[k0 + u] * p.row_bytes);
#pragma unroll
        for (int u = 0; u < kMove; ++u)
            if (k0 + u < n) *reinterpret_cast<uint4*>(base + (int64_t)(1 + k0 + u) * p.row_bytes) = x[u];
    }
}

}  // namespace

cudaError_t launch_latent_append(LatentAppendParams p, cudaStream_t st) {
    const int steps = p.q ? (p.H + 7) / 8 : 0;
    const int64_t tokens = (int64_t)p.B * p.n;
    // few tokens: a token's heads spread over more warps, up to 32 an SM
    int64_t slices = ((int64_t)sm_count() * 32 + tokens - 1) / tokens;
    if (slices > steps) slices = steps;
    p.slices = (int)slices;
    const int64_t blocks = (tokens * (p.slices + 1) + kAppendWarps - 1) / kAppendWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return p.interleaved ? launch(latent_append_kernel<true>, dim3((unsigned)blocks), kAppendThreads, p, st)
                         : launch(latent_append_kernel<false>, dim3((unsigned)blocks), kAppendThreads, p, st);
}

cudaError_t launch_latent_read(const LatentReadParams& p, cudaStream_t st) {
    const int64_t units = (int64_t)p.B * ((p.n - 1) / kReadRows + 1);
    const int64_t blocks = (units + 3) / 4;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return p.q8 ? launch(latent_read_kernel<true>, dim3((unsigned)blocks), 128, p, st)
                : launch(latent_read_kernel<false>, dim3((unsigned)blocks), 128, p, st);
}

cudaError_t launch_latent_commit(const LatentCommitParams& p, int layers, int B, cudaStream_t st) {
    return launch(latent_commit_kernel, dim3(B, layers), 96, p, st);
}

}  // namespace rapid
