// Per-head norm, rotary positions and the append to the KV cache, in one pass over the
// projection rows of a verify step or a prefill chunk.
//
//   y = x / sqrt(mean(x^2) + eps) * w          (where a norm weight is given)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq[pair]
//
// Queries go to [B, Hq, n, d], the layout verify attention reads; keys and values to their
// cache rows.  All arithmetic is in fp32 and rounded once, at the store.
//
// The angle is formed in fixed point: inv_freq / (2 pi) becomes a 64-bit fraction of a
// turn, its product with the integer position wraps modulo one turn exactly, and the top
// 32 bits go to sincospi.  An fp32 product would be off by 2^-24 of the angle, 0.008 rad at
// position 131072.
//
// The work is copying: d elements in and out for each head row, no reuse.  A head row is
// read by d / 16 lanes, each with the two 16-byte (bf16) pieces whose elements rotate into
// each other, so a rotated pair never leaves its lane; a warp takes one token and some of
// its heads, with the sines and cosines of its lanes' pairs kept in registers over all of
// them.
//
// Measured: 8192 tokens of 32 + 8 + 8 heads of 128, bf16, with norms, 35.8 us for 201 MB (5.6
// TB/s, 0.83 of a plain copy); 3 ragged chunks of 1999 tokens, fp32, d = 64, 21.1 us (0.77);
// 11 tokens 2.5 us.  Each warp has two steps' loads in flight before it works on the first, in
// place of one (45.6 us), and 28 warps an SM, in place of 20 (40.4 us); with bf16 that is 72 registers
// a thread and 2 to 4 of them spilled.
#include "common.cuh"
#include "qkv_append.cuh"

namespace rapid {

namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendWarps = kAppendThreads / 32;

// inv_freq / (2 pi) modulo one turn as a fraction of 2^64.  |f| = m 2^(e - 23) with m a
// 24-bit integer, and 1 / (2 pi) = C 2^-66 to 64 bits, so the fraction is m C 2^(e - 25).
__device__ __forceinline__ uint64_t turns_per_position(float f) {
    constexpr uint64_t kInvTwoPi = 0xa2f9836e4e441529ull;   // 2^66 / (2 pi), rounded down
    const uint32_t bits = __float_as_uint(f);
    const int field = (int)((bits >> 23) & 0xff);
    if (field == 0xff) return 0;                            // inf or NaN: no rotation is defined
    const uint64_t m = (bits & 0x7fffffu) | (field ? 0x800000u : 0u);
    const int right = 25 - ((field ? field : 1) - 127);     // fraction = (hi : lo) >> right
    const uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
    uint64_t x;
    if (right >= 128) x = 0;
    else if (right >= 64) x = hi >> (right - 64);
    else if (right > 0) x = (lo >> right) | (hi << (64 - right));
    else x = right > -64 ? lo << -right : 0;
    return (bits >> 31) ? 0 - x : x;
}

__device__ __forceinline__ void sincos_turn(uint64_t per_pos, int64_t pos, float* s, float* c) {
    const uint64_t t = per_pos * (uint64_t)pos;             // modulo one turn
    const int32_t top = (int32_t)((t + 0x80000000ull) >> 32);
    sincospif((float)top * 4.656612873077392578125e-10f, s, c);   // top 2^-31 half turns
}

template <typename T> struct Piece;                         // 8 elements
template <> struct Piece<__nv_bfloat16> { uint4 a; };
template <> struct Piece<float> { float4 a, b; };

__device__ __forceinline__ void load_piece(const __nv_bfloat16* p, Piece<__nv_bfloat16>& r) {
    r.a = __ldg(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void load_piece(const float* p, Piece<float>& r) {
    r.a = __ldg(reinterpret_cast<const float4*>(p));
    r.b = __ldg(reinterpret_cast<const float4*>(p) + 1);
}
__device__ __forceinline__ void store_piece(__nv_bfloat16* p, const Piece<__nv_bfloat16>& r) {
    *reinterpret_cast<uint4*>(p) = r.a;
}
__device__ __forceinline__ void store_piece(float* p, const Piece<float>& r) {
    reinterpret_cast<float4*>(p)[0] = r.a;
    reinterpret_cast<float4*>(p)[1] = r.b;
}
__device__ __forceinline__ void unpack(const Piece<__nv_bfloat16>& r, float (&x)[8]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const Piece<float>& r, float (&x)[8]) {
    x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
    x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
__device__ __forceinline__ void pack(const float (&x)[8], Piece<__nv_bfloat16>& r) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float (&x)[8], Piece<float>& r) {
    r.a = make_float4(x[0], x[1], x[2], x[3]);
    r.b = make_float4(x[4], x[5], x[6], x[7]);
}

// CTAs of an SM: 28 warps (bf16) or 16 (fp32) with two head rows a lane group in flight.
template <typename T> constexpr int kAppendCtas = sizeof(T) == 2 ? 7 : 4;

template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas<T>) qkv_append_kernel(const QkvAppendParams p) {
    constexpr int kLanes = D / 16;                  // lanes of one head row
    constexpr int kRows = 32 / kLanes;              // head rows a warp handles at a time
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, l = lane - sub * kLanes;
    const int64_t unit = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    const int64_t token = unit / p.slices;
    const int slice = (int)(unit - token * p.slices);
    if (token >= (int64_t)p.B * p.n) return;
    const int b = (int)(token / p.n), i = (int)(token - (int64_t)b * p.n);

    const int count = p.n_rows ? p.n_rows[b] : p.n;
    const int64_t P = p.prefix_len[b];
    if (count < 0 || count > p.n || P < 0 || P + count > p.cap) {   // refused: left alone
        if (i == 0 && slice == 0 && lane == 0 && p.err) atomicOr(p.err, kErrBadInput);
        return;
    }
    if (i >= count) return;
    int64_t pos = P + (p.row_offset ? p.row_offset[(int64_t)b * p.n + i] : i);
    if (p.pos_offset) pos += p.pos_offset[b];

    // The lane's two pieces.  Rotated halves: piece c pairs with piece c + rot / 16; the
    // pieces past rot are not rotated.  Interleaved pairs sit inside a piece.
    const int half = p.rot / 16;
    int c0, c1;
    if (INTERLEAVED || l < half) { c0 = l; c1 = l + (INTERLEAVED ? kLanes : half); }
    else { c0 = 2 * l; c1 = 2 * l + 1; }
    const bool turn = !INTERLEAVED && l < half;
    // Sines and cosines of the lane's 8 pairs.  The lanes of a token's other rows need the same
    // ones, so each row's lanes work out their share and the rest comes by shuffles.
    constexpr int kShare = 8 / kRows;
    float my_sn[kShare], my_cs[kShare], sn[8], cs[8];
#pragma unroll
    for (int e = 0; e < kShare; ++e) {
        const int u = sub * kShare + e;             // interleaved: u < 4 pairs of piece c0, else of c1
        const int pair = INTERLEAVED ? (u < 4 ? c0 : c1) * 4 + (u & 3) : 8 * c0 + u;
        my_sn[e] = 0.f;
        my_cs[e] = 1.f;
        if (INTERLEAVED ? 2 * pair < p.rot : turn)
            sincos_turn(turns_per_position(__ldg(p.inv_freq + pair)), pos, &my_sn[e], &my_cs[e]);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        sn[u] = __shfl_sync(0xffffffffu, my_sn[u % kShare], u / kShare * kLanes + l);
        cs[u] = __shfl_sync(0xffffffffu, my_cs[u % kShare], u / kShare * kLanes + l);
    }

    // Steps of kRows heads: first the queries', then the keys', then the values'.  Rows of
    // queries and of the caches are q_step and kv_step elements apart.
    const int q_steps = (p.Hq + kRows - 1) / kRows, kv_steps = (p.Hkv + kRows - 1) / kRows;
    const int steps = q_steps + 2 * kv_steps;
    const T* q = static_cast<const T*>(p.q) + b * p.q_batch + i * p.q_token;
    const T* k = static_cast<const T*>(p.k) + b * p.k_batch + i * p.k_token;
    const T* v = static_cast<const T*>(p.v) + b * p.v_batch + i * p.v_token;
    T* Q = static_cast<T*>(p.Q) + ((int64_t)b * p.Hq * p.n + i) * D;
    const int64_t cache = ((int64_t)b * p.Hkv * p.cap + P + i) * D;
    const int64_t q_step = (int64_t)p.n * D, kv_step = p.cap * D;

    auto load_step = [&](int it, Piece<T>& r0, Piece<T>& r1) {
        const bool is_q = it < q_steps, is_k = it < q_steps + kv_steps;
        const int h = (is_q ? it : is_k ? it - q_steps : it - q_steps - kv_steps) * kRows + sub;
        r0 = {};
        r1 = {};
        if (h >= (is_q ? p.Hq : p.Hkv)) return;
        const T* src = (is_q ? q : is_k ? k : v) + h * D;
        load_piece(src + 8 * c0, r0);
        load_piece(src + 8 * c1, r1);
    };
    auto finish_step = [&](int it, Piece<T>& r0, Piece<T>& r1) {
        const bool is_q = it < q_steps, is_k = it < q_steps + kv_steps;   // one kind for the warp
        const int h = (is_q ? it : is_k ? it - q_steps : it - q_steps - kv_steps) * kRows + sub;
        if (is_k) {                                 // a query or a key
            float x[8], y[8];
            unpack(r0, x);
            unpack(r1, y);
            const T* w = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
            if (w) {
                Piece<T> w0, w1;
                load_piece(w + 8 * c0, w0);
                load_piece(w + 8 * c1, w1);
                float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int u = 0; u < 8; u += 2) {
                    const float2 a = make_float2(x[u], x[u + 1]), c = make_float2(y[u], y[u + 1]);
                    s2 = fma2(a, a, fma2(c, c, s2));
                }
                float ss = s2.x + s2.y;
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = rsqrtf(ss * (1.f / D) + p.eps);
                const float2 i2 = make_float2(inv, inv);
                float wx[8], wy[8];
                unpack(w0, wx);
                unpack(w1, wy);
#pragma unroll
                for (int u = 0; u < 8; u += 2) {
                    const float2 a = mul2(mul2(make_float2(x[u], x[u + 1]), i2), make_float2(wx[u], wx[u + 1]));
                    const float2 c = mul2(mul2(make_float2(y[u], y[u + 1]), i2), make_float2(wy[u], wy[u + 1]));
                    x[u] = a.x; x[u + 1] = a.y;
                    y[u] = c.x; y[u + 1] = c.y;
                }
            }
            if (INTERLEAVED) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float a = x[2 * u], c = x[2 * u + 1], e = y[2 * u], f = y[2 * u + 1];
                    x[2 * u] = a * cs[u] - c * sn[u];
                    x[2 * u + 1] = c * cs[u] + a * sn[u];
                    y[2 * u] = e * cs[4 + u] - f * sn[4 + u];
                    y[2 * u + 1] = f * cs[4 + u] + e * sn[4 + u];
                }
            } else if (turn) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float a = x[u], c = y[u];
                    x[u] = a * cs[u] - c * sn[u];
                    y[u] = c * cs[u] + a * sn[u];
                }
            }
            pack(x, r0);
            pack(y, r1);
        }
        if (h < (is_q ? p.Hq : p.Hkv)) {
            T* dst = is_q ? Q + h * q_step : static_cast<T*>(is_k ? p.K : p.V) + cache + h * kv_step;
            store_piece(dst + 8 * c0, r0);
            store_piece(dst + 8 * c1, r1);
        }
    };
    // two steps at a time, both on their way before the first is worked on
    for (int it = slice; it < steps; it += 2 * p.slices) {
        const int next = it + p.slices;
        Piece<T> r0, r1, n0, n1;
        load_step(it, r0, r1);
        if (next < steps) load_step(next, n0, n1);
        finish_step(it, r0, r1);
        if (next < steps) finish_step(next, n0, n1);
    }
}

template <typename T, int D>
cudaError_t launch_typed(QkvAppendParams p, cudaStream_t st) {
    constexpr int kRows = 32 / (D / 16);
    const int steps = (p.Hq + kRows - 1) / kRows + 2 * ((p.Hkv + kRows - 1) / kRows);
    const int64_t tokens = (int64_t)p.B * p.n;
    // few tokens: spread each one's heads over several warps, up to 32 an SM (up to 64: the
    // sines of a token are worked out more often, 37.3 us where 32 and 16 take 35.8)
    int64_t slices = ((int64_t)sm_count() * 32 + tokens - 1) / tokens;
    if (slices > steps) slices = steps;
    p.slices = (int)(slices < 1 ? 1 : slices);
    const int64_t blocks = (tokens * p.slices + kAppendWarps - 1) / kAppendWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    cfg.blockDim = dim3(kAppendThreads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return p.interleaved ? cudaLaunchKernelEx(&cfg, qkv_append_kernel<T, D, true>, p)
                         : cudaLaunchKernelEx(&cfg, qkv_append_kernel<T, D, false>, p);
}

}  // namespace

cudaError_t launch_qkv_append(QkvAppendParams p, int dtype, cudaStream_t st) {
    if (dtype == 1)
        return p.d == 128 ? launch_typed<__nv_bfloat16, 128>(p, st) : launch_typed<__nv_bfloat16, 64>(p, st);
    return p.d == 128 ? launch_typed<float, 128>(p, st) : launch_typed<float, 64>(p, st);
}

}  // namespace rapid
