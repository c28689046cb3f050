// Sealing: whole blocks of 64 committed tail rows become pages of 8-bit values.
//
// A block of one KV head and side (K or V) has one scale, the smallest power of two that
// brings its largest magnitude into e4m3's range,
//   scale = 2^ceil(log2(max|x| / 448)),   code = e4m3(x / scale)  (nearest, ties to even).
// e4m3 is a floating-point format, so a power of two costs nothing in relative precision
// against max / 448 (only the subnormal end shifts by less than one bit), and it makes the
// division, and the product that undoes it, exact.  A value that is not finite is stored as
// e4m3's NaN and takes no part in the maximum; an all-zero block has scale 1; the exponent
// is at least -64, so values below 2^-74 become zero.
//
// What bounds it, while few rows stay, is the copy: 2 (or 4) bytes read and 1 written for each
// element, the rows that stay read and written once.  A CTA holds a whole block (K and V of one
// head) in registers between the maximum and the store, so the block is read once.  The blocks that
// the rows which stay will overwrite, and the moving of those rows, are one CTA's work for each head,
// 64 rows after 64: with about half of the tail kept it does all of it, and few heads leave most of
// the machine idle.
//
// Measured: 33 blocks of 8 heads on 32 layers, d = 128, bf16 66.3 us for 420 MB (0.93 of a plain
// copy), fp32 110 (0.94); at most one block of each of 4 sequences on 32 layers, bf16 4.9 us (floor
// 2.3: the lengths, the page ids and the rows are read one after the other), fp32 7.8 (3.9).  4096
// tail rows of which 2000 stay: 32 layers 171 us (139), one layer 60 (4.3; 19 with none kept).  Held
// as fp32 instead of packed, a bf16 block leaves room for two CTAs an SM instead of four: 95 us.
#include "common.cuh"
#include "kv_seal.cuh"

namespace rapid {

namespace {

constexpr int kSealThreads = 256;
constexpr int kSideThreads = kSealThreads / 2;   // threads 0..127: K, 128..255: V

// Blocks that sequence b seals now, or -1 where its device-side inputs are invalid (the
// sequence is then left alone).  Every thread of the CTA calls it.
__device__ __forceinline__ int seal_blocks(const SealPlan& p, int b) {
    const int64_t P = p.tail_len[b], S = p.sealed_len[b];
    bool ok = P >= 0 && P <= p.cap && S >= 0 && (S % kPageTokens) == 0;
    const int64_t stay = P < p.keep ? P : p.keep;
    const int64_t n_b = ok ? (P - stay) / kPageTokens : 0;
    const int64_t first = S / kPageTokens;
    if (ok && n_b > 0 && first + n_b > p.max_pages) ok = false;
    if (ok) {
        const int32_t* ids = p.page_table + (int64_t)b * p.max_pages + first;
        for (int64_t j = threadIdx.x; j < n_b; j += blockDim.x) {
            const int id = ids[j];
            if (id < 0 || id >= p.n_pages) ok = false;
        }
    }
    return __syncthreads_and(ok) ? (int)n_b : -1;
}

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// A unit is 16 consecutive elements, held as they are: 2 (bf16) or 4 (fp32) 16-byte pieces.
// Magnitudes are compared as integers, which order finite values as floats do and put what
// is not finite above them.
template <typename T> struct Unit;
template <> struct Unit<__nv_bfloat16> {
    static constexpr uint32_t kFirstOdd = 0x7f80u;      // least magnitude that is not finite
    uint4 v[2];
    __device__ __forceinline__ void top(uint32_t& m) const {   // two running maxima in m
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    }
    static __device__ __forceinline__ uint32_t join(uint32_t m) { return max(m & 0xffffu, m >> 16); }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m << 16; }   // as fp32
    __device__ __forceinline__ void to_float(float (&x)[16]) const {
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <> struct Unit<float> {
    static constexpr uint32_t kFirstOdd = 0x7f800000u;
    uint4 v[4];
    __device__ __forceinline__ void top(uint32_t& m) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = max(max(max(m, v[i].x & 0x7fffffffu), max(v[i].y & 0x7fffffffu, v[i].z & 0x7fffffffu)),
                    v[i].w & 0x7fffffffu);
    }
    static __device__ __forceinline__ uint32_t join(uint32_t m) { return m; }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m; }
    __device__ __forceinline__ void to_float(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[4 * i] = __uint_as_float(v[i].x); x[4 * i + 1] = __uint_as_float(v[i].y);
            x[4 * i + 2] = __uint_as_float(v[i].z); x[4 * i + 3] = __uint_as_float(v[i].w);
        }
    }
};

// Maximum over the four warps of a side.
__device__ __forceinline__ uint32_t side_max(uint32_t m, uint32_t (&s)[4], int warp, int lane) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) s[warp] = m;
    __syncthreads();
    return max(max(s[0], s[1]), max(s[2], s[3]));
}

// CTAs of an SM: what a block held in registers leaves room for.
template <typename T> constexpr int kSealCtas = sizeof(T) == 2 ? 4 : 2;

// grid: (parts, B * Hkv, layers).  Part 0 seals the blocks that the rows which stay will
// overwrite and then moves those rows to the front; the other blocks are shared out over
// the parts.  So no row is overwritten before its one reader has read it.
template <typename T, int D>
__global__ void __launch_bounds__(kSealThreads, kSealCtas<T>) kv_seal_kernel(const __grid_constant__ SealParams p) {
    constexpr int kUnits = kPageTokens * D / 16 / kSideThreads;   // 16-element units a thread holds
    constexpr int kPiece = 16 / sizeof(T);                        // elements of 16 bytes
    constexpr int kRowPieces = D / kPiece;
    constexpr int kMovePieces = kPageTokens * kRowPieces / kSideThreads;   // 64 rows at a time
    __shared__ uint32_t s_max[2][4];
    griddep_wait();
    const int part = blockIdx.x;
    const int b = blockIdx.y / p.Hkv, g = blockIdx.y - b * p.Hkv;
    const SealLayer& layer = p.layer[blockIdx.z];
    const int n_b = seal_blocks(p.plan, b);
    if (n_b < 0) {
        if (threadIdx.x == 0 && part == 0 && g == 0 && blockIdx.z == 0 && p.err)
            atomicOr(p.err, kErrBadInput);
        return;
    }
    if (n_b == 0) return;
    const int side = threadIdx.x / kSideThreads, t = threadIdx.x - side * kSideThreads;
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    T* rows = static_cast<T*>(side ? layer.V : layer.K) + ((int64_t)b * p.Hkv + g) * p.plan.cap * D;
    const int64_t rest = p.plan.tail_len[b] - (int64_t)n_b * kPageTokens;
    const int64_t over = (rest + kPageTokens - 1) / kPageTokens;   // blocks the move overwrites
    const int first = (int)(over < n_b ? over : n_b);
    const int32_t* ids = p.plan.page_table + (int64_t)b * p.plan.max_pages +
                         p.plan.sealed_len[b] / kPageTokens;

    for (int j = 0; j < n_b; ++j) {
        const int owner = j < first ? 0 : (j - first + 1) % p.parts;
        if (owner != part) continue;
        Unit<T> held[kUnits];
        const T* src = rows + (int64_t)j * kPageTokens * D;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const uint4* from = reinterpret_cast<const uint4*>(src + (u * kSideThreads + t) * 16);
#pragma unroll
            for (int e = 0; e < (int)sizeof(T); ++e) held[u].v[e] = from[e];
        }
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) held[u].top(m);
        m = side_max(Unit<T>::join(m), s_max[side], warp, lane);
        const bool odd = m >= Unit<T>::kFirstOdd;       // something is not finite (the same in the side)
        if (__syncthreads_or(odd)) {                    // the maximum again, of what is finite
            float f = 0.f;
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                float x[16];
                held[u].to_float(x);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (fabsf(x[e]) < INFINITY) f = fmaxf(f, fabsf(x[e]));
            }
            const uint32_t g2 = side_max(__float_as_uint(f), s_max[side], warp, lane);
            if (odd) m = sizeof(T) == 2 ? g2 >> 16 : g2;
            __syncthreads();
        }
        const float top = __uint_as_float(Unit<T>::bits(m));
        // 448 = 1.75 * 2^8: top = 1.f 2^k needs exponent k - 8, one more above 1.75
        const uint32_t bits = __float_as_uint(top);
        int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = e < kScaleExpMin ? kScaleExpMin : e;
        if (top == 0.f) e = 0;
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        const int64_t slot = ((int64_t)ids[j] * p.Hkv + g) * 2 + side;
        uint8_t* dst = layer.pages + slot * kPageTokens * D;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            float x[16];
            held[u].to_float(x);
            if (odd) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (!(fabsf(x[e]) < INFINITY)) x[e] = __int_as_float(0x7fffffff);
            }
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w[q] = (uint32_t)e4m3x2(x[4 * q] * inv, x[4 * q + 1] * inv) |
                       (uint32_t)e4m3x2(x[4 * q + 2] * inv, x[4 * q + 3] * inv) << 16;
            *reinterpret_cast<uint4*>(dst + (u * kSideThreads + t) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (t == 0) layer.scales[slot] = __uint_as_float((uint32_t)(127 + e) << 23);
    }
    if (part != 0) return;
    // The rows that stay, 64 at a time in ascending order: a chunk's destination lies below
    // every later chunk's source, and the chunk itself is read before it is written.
    const T* from = rows + (int64_t)n_b * kPageTokens * D;
    for (int64_t r0 = 0; r0 < rest; r0 += kPageTokens) {
        uint4 v[kMovePieces];
        const int64_t left = (rest - r0) * kRowPieces;
#pragma unroll
        for (int u = 0; u < kMovePieces; ++u) {
            const int x = u * kSideThreads + t;
            if (x < left) v[u] = reinterpret_cast<const uint4*>(from + r0 * D)[x];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kMovePieces; ++u) {
            const int x = u * kSideThreads + t;
            if (x < left) reinterpret_cast<uint4*>(rows + r0 * D)[x] = v[u];
        }
        __syncthreads();
    }
}

// One CTA per sequence.
__global__ void __launch_bounds__(32) kv_seal_advance_kernel(const SealPlan plan, int32_t* sealed_len,
                                                             int32_t* tail_len, unsigned int* err) {
    griddep_wait();
    const int b = blockIdx.x;
    const int n_b = seal_blocks(plan, b);
    if (threadIdx.x != 0) return;
    if (n_b < 0) {
        if (err) atomicOr(err, kErrBadInput);
        return;
    }
    sealed_len[b] += n_b * kPageTokens;
    tail_len[b] -= n_b * kPageTokens;
}

cudaLaunchConfig_t config(dim3 grid, int threads, cudaStream_t st, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = st;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace

cudaError_t launch_kv_seal(const SealParams& p0, int layers, int dtype, cudaStream_t st) {
    SealParams p = p0;
    // as many parts as one wave of CTAs holds: 33 blocks of 256 heads and layers, bf16, d = 128,
    // take 66.6 us with 2 parts (512 CTAs) and 77.7 with 3 (768, of which 608 run at once)
    const int64_t heads = (int64_t)p.plan.B * p.Hkv * layers;
    int64_t parts = (int64_t)sm_count() * (dtype == 1 ? kSealCtas<__nv_bfloat16> : kSealCtas<float>) / heads;
    const int64_t most = p.plan.cap / kPageTokens;
    if (parts > most) parts = most;
    p.parts = (int)(parts < 1 ? 1 : parts);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(dim3(p.parts, p.plan.B * p.Hkv, layers), kSealThreads, st, attr);
    if (dtype == 1)
        return p.d == 128 ? cudaLaunchKernelEx(&cfg, kv_seal_kernel<__nv_bfloat16, 128>, p)
                          : cudaLaunchKernelEx(&cfg, kv_seal_kernel<__nv_bfloat16, 64>, p);
    return p.d == 128 ? cudaLaunchKernelEx(&cfg, kv_seal_kernel<float, 128>, p)
                      : cudaLaunchKernelEx(&cfg, kv_seal_kernel<float, 64>, p);
}

cudaError_t launch_kv_seal_advance(const SealPlan& plan, int32_t* sealed_len, int32_t* tail_len,
                                   unsigned int* err, cudaStream_t st) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(dim3(plan.B, 1, 1), 32, st, attr);
    return cudaLaunchKernelEx(&cfg, kv_seal_advance_kernel, plan, sealed_len, tail_len, err);
}

}  // namespace rapid
