// C ABI of the latent cache: append, read back, commit, absorbed and expanded attention.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "latent.cuh"
#include "rapid.h"

namespace rapid {

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool cache_ok(int dtype) { return dtype == RAPID_DTYPE_BF16 || dtype == RAPID_CACHE_LATENT_Q8; }
bool capacity_ok(int64_t cap) { return cap >= 1 && cap <= RAPID_LATENT_MAX_ROWS; }
// element strides of bf16 rows that are read or written in 16-byte pieces
bool strides_ok(const int64_t* s, int n) {
    for (int i = 0; i < n; ++i)
        if (s[i] < 0 || s[i] > ((int64_t)1 << 38) || s[i] % 8 != 0) return false;
    return true;
}
rapid_status status_of(cudaError_t e) { return e == cudaSuccess ? RAPID_OK : RAPID_ECUDA; }

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct AttnPlan {
    int S, RB;
    size_t acc, ml, index;       // bytes of the workspace's parts
    size_t bytes() const { return acc + ml + 2 * index; }
};

AttnPlan plan_attn(int B, int H, int n_q, int64_t cap) {
    AttnPlan pl;
    const int R = H * n_q, nr = latent_attn_block_rows(R);
    pl.S = latent_attn_slots(B, R, cap);
    pl.RB = (R + nr - 1) / nr;
    const size_t rows = pl.S > B ? (size_t)pl.S * R : 0;      // one split each: no partials
    pl.acc = align_up(rows * kLatent * sizeof(float));
    pl.ml = align_up(rows * 2 * sizeof(float));
    pl.index = align_up((size_t)B * sizeof(int));
    return pl;
}

struct PrefillPlan {
    int ctas;
    size_t acc, ml, index;
    size_t bytes() const { return acc + ml + index; }
};

bool prefill_args_ok(int B, int n, int H, int64_t kv_rows) {
    if (B < 1 || B > 65535 || n < 1 || H < 1 || H > RAPID_LATENT_MAX_HEADS) return false;
    return (int64_t)B * n * H <= RAPID_LATENT_MAX_QUERIES && capacity_ok(kv_rows);
}

PrefillPlan plan_prefill(int B, int n, int H, int64_t kv_rows) {
    PrefillPlan pl;
    const size_t rows = latent_prefill_block_rows();
    pl.ctas = latent_prefill_ctas(B, n, H, kv_rows);
    pl.acc = align_up(2 * pl.ctas * rows * kLatentHead * sizeof(float));
    pl.ml = align_up(2 * pl.ctas * rows * 2 * sizeof(float));
    pl.index = pl.ctas ? align_up((B * ((n + rows - 1) / rows) + 1) * sizeof(int64_t)) : kAlign;
    return pl;
}

bool attn_args_ok(int B, int H, int n_q, int64_t cap, int cache_dtype) {
    if (B < 1 || B > 65535 || H < 1 || H > RAPID_LATENT_MAX_HEADS || !cache_ok(cache_dtype)) return false;
    if (n_q < 1 || n_q > RAPID_MAX_NQ || !capacity_ok(cap) || cap < n_q) return false;
    // tiles of 64 rows of all sequences are counted in 32 bits
    return (int64_t)B * H * n_q <= RAPID_LATENT_MAX_QUERIES && B * ((cap + 127) / 64) < ((int64_t)1 << 31);
}

}  // namespace
}  // namespace rapid

using namespace rapid;

extern "C" {

rapid_status rapid_latent_append(const void* kv, const int64_t* kv_strides, const void* q,
                                 const int64_t* q_strides, int B, int n, int H,
                                 const void* kv_weight, float eps, const float* inv_freq,
                                 uint32_t flags, const int32_t* prefix_len,
                                 const int32_t* row_offset, const int32_t* n_rows, void* q_out,
                                 void* cache, int cache_dtype, int64_t kv_capacity, void* stream) {
    if (!kv || !inv_freq || !prefix_len || !cache) return RAPID_EINVAL;
    if ((q == nullptr) != (q_out == nullptr)) return RAPID_EINVAL;
    if (B < 1 || n < 1 || (int64_t)B * n > ((int64_t)1 << 31)) return RAPID_EINVAL;
    if (q && (H < 1 || H > RAPID_LATENT_MAX_HEADS)) return RAPID_EINVAL;
    if (!cache_ok(cache_dtype) || !capacity_ok(kv_capacity)) return RAPID_EINVAL;
    if ((flags & ~(uint32_t)RAPID_ROPE_INTERLEAVED) != 0) return RAPID_EINVAL;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return RAPID_EINVAL;
    const void* rows16[] = {kv, q, q_out, kv_weight, cache};
    for (const void* x : rows16)
        if (!aligned(x, 16)) return RAPID_EINVAL;
    const void* words[] = {inv_freq, prefix_len, row_offset, n_rows};
    for (const void* x : words)
        if (!aligned(x, 4)) return RAPID_EINVAL;
    LatentAppendParams p{};
    const int64_t kv_packed[2] = {(int64_t)n * kLatentRow, kLatentRow};
    const int64_t* ks = kv_strides ? kv_strides : kv_packed;
    if (!strides_ok(ks, 2)) return RAPID_EINVAL;
    if (q) {
        const int64_t token = (int64_t)H * kLatentRope;
        const int64_t q_packed[6] = {n * token, token, kLatentRope, n * token, token, kLatentRope};
        const int64_t* qs = q_strides ? q_strides : q_packed;
        if (!strides_ok(qs, 6)) return RAPID_EINVAL;
        // rows of q_out that repeat or run into each other would be written at once
        const int64_t size[3] = {B, n, H};
        for (int i = 0; i < 3; ++i)
            if (size[i] > 1 && qs[3 + i] < kLatentRope) return RAPID_EINVAL;
        p.q_batch = qs[0]; p.q_token = qs[1]; p.q_head = qs[2];
        p.o_batch = qs[3]; p.o_token = qs[4]; p.o_head = qs[5];
        p.H = H;
    }
    p.kv = kv; p.q = q; p.q_out = q_out; p.weight = kv_weight; p.inv_freq = inv_freq;
    p.prefix_len = prefix_len; p.row_offset = row_offset; p.n_rows = n_rows;
    p.cache = static_cast<uint8_t*>(cache);
    p.err = device_error_word();
    p.kv_batch = ks[0]; p.kv_token = ks[1];
    p.cap = kv_capacity;
    p.B = B; p.n = n;
    p.interleaved = (flags & RAPID_ROPE_INTERLEAVED) ? 1 : 0;
    p.q8 = cache_dtype == RAPID_CACHE_LATENT_Q8;
    p.eps = eps;
    return status_of(launch_latent_append(p, static_cast<cudaStream_t>(stream)));
}

rapid_status rapid_latent_read(const void* cache, int cache_dtype, int B, int64_t kv_capacity, int n,
                               const int32_t* first, const int32_t* n_rows, void* rows, void* stream) {
    if (!cache || !rows || B < 1 || n < 1 || (int64_t)B * n > ((int64_t)1 << 31)) return RAPID_EINVAL;
    if (!cache_ok(cache_dtype) || !capacity_ok(kv_capacity)) return RAPID_EINVAL;
    if (!aligned(cache, 16) || !aligned(rows, 16) || !aligned(first, 4) || !aligned(n_rows, 4))
        return RAPID_EINVAL;
    LatentReadParams p{};
    p.cache = static_cast<const uint8_t*>(cache);
    p.first = first; p.n_rows = n_rows;
    p.rows = static_cast<uint8_t*>(rows);
    p.err = device_error_word();
    p.cap = kv_capacity;
    p.B = B; p.n = n;
    p.q8 = cache_dtype == RAPID_CACHE_LATENT_Q8;
    return status_of(launch_latent_read(p, static_cast<cudaStream_t>(stream)));
}

rapid_status rapid_latent_commit(void* const* caches, int layers, int cache_dtype, int B,
                                 int64_t kv_capacity, int n_q, const int32_t* prefix_len,
                                 const int32_t* path, const int32_t* n_accepted, void* stream) {
    if (!caches || !prefix_len || !path || !n_accepted) return RAPID_EINVAL;
    if (layers < 1 || layers > RAPID_COMMIT_MAX_LAYERS || B < 1 || !cache_ok(cache_dtype)) return RAPID_EINVAL;
    if (n_q < 1 || n_q > RAPID_MAX_NQ || !capacity_ok(kv_capacity)) return RAPID_EINVAL;
    if (!aligned(prefix_len, 4) || !aligned(path, 4) || !aligned(n_accepted, 4)) return RAPID_EINVAL;
    LatentCommitParams p{};
    for (int l = 0; l < layers; ++l) {
        if (!caches[l] || !aligned(caches[l], 16)) return RAPID_EINVAL;
        p.cache[l] = static_cast<uint8_t*>(caches[l]);
    }
    p.row_bytes = latent_row_bytes(cache_dtype == RAPID_CACHE_LATENT_Q8);
    // layers move their rows at the same time: a cache twice, or two that overlap, would be moved twice
    uintptr_t at[kLatentMaxLayers];
    for (int l = 0; l < layers; ++l) at[l] = reinterpret_cast<uintptr_t>(caches[l]);
    std::sort(at, at + layers);
    for (int l = 1; l < layers; ++l)
        if ((double)(at[l] - at[l - 1]) < (double)B * kv_capacity * p.row_bytes) return RAPID_EINVAL;
    p.prefix_len = prefix_len; p.path = path; p.n_acc = n_accepted;
    p.err = device_error_word();
    p.cap = kv_capacity;
    p.n_q = n_q;
    return status_of(launch_latent_commit(p, layers, B, static_cast<cudaStream_t>(stream)));
}

size_t rapid_latent_attn_workspace_size(int B, int H, int n_q, int64_t kv_capacity, int cache_dtype) {
    if (!attn_args_ok(B, H, n_q, kv_capacity, cache_dtype)) return 0;
    return plan_attn(B, H, n_q, kv_capacity).bytes();
}

rapid_status rapid_latent_attn(const void* Q, const void* cache, int cache_dtype, int B, int H, int n_q,
                               int64_t kv_capacity, const int32_t* prefix_len,
                               const uint8_t* spec_mask, float softmax_scale, void* O, float* LSE,
                               void* workspace, size_t workspace_bytes, void* stream) {
    if (!Q || !cache || !prefix_len || !O || !LSE || !workspace) return RAPID_EINVAL;
    if (!attn_args_ok(B, H, n_q, kv_capacity, cache_dtype)) return RAPID_EINVAL;
    const void* rows16[] = {Q, cache, O, workspace};
    for (const void* x : rows16)
        if (!aligned(x, 16)) return RAPID_EINVAL;
    if (!aligned(prefix_len, 4) || !aligned(LSE, 4) || !std::isfinite(softmax_scale)) return RAPID_EINVAL;
    const AttnPlan pl = plan_attn(B, H, n_q, kv_capacity);
    if (workspace_bytes < pl.bytes()) return RAPID_ENOMEM;
    LatentAttnParams p{};
    p.Q = Q; p.cache = static_cast<const uint8_t*>(cache);
    p.prefix_len = prefix_len; p.mask = spec_mask; p.O = O; p.LSE = LSE;
    p.err = device_error_word();
    p.cap = kv_capacity;
    p.B = B; p.H = H; p.n_q = n_q; p.S = pl.S; p.RB = pl.RB;
    char* ws = static_cast<char*>(workspace);
    p.part_acc = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + pl.acc);
    p.part_first = reinterpret_cast<int*>(ws + pl.acc + pl.ml);
    p.part_count = reinterpret_cast<int*>(ws + pl.acc + pl.ml + pl.index);
    p.q8 = cache_dtype == RAPID_CACHE_LATENT_Q8;
    p.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)(kLatentHead + kLatentRope))) * kLog2e;
    return status_of(launch_latent_attn(p, static_cast<cudaStream_t>(stream)));
}

size_t rapid_latent_prefill_attn_workspace_size(int B, int n, int H, int64_t kv_rows) {
    return prefill_args_ok(B, n, H, kv_rows) ? plan_prefill(B, n, H, kv_rows).bytes() : 0;
}

rapid_status rapid_latent_prefill_attn(const void* Q, const void* K, const void* V, const void* K_rope,
                                       const int64_t* strides, int B, int n, int H, int64_t kv_rows,
                                       const int32_t* prefix_len, const int32_t* n_rows,
                                       float softmax_scale, void* O, float* LSE, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    if (!Q || !K || !V || !K_rope || !prefix_len || !O || !LSE || !workspace) return RAPID_EINVAL;
    if (!prefill_args_ok(B, n, H, kv_rows)) return RAPID_EINVAL;
    const void* rows16[] = {Q, K, V, K_rope, O, workspace};
    for (const void* x : rows16)
        if (!aligned(x, 16)) return RAPID_EINVAL;
    if (!aligned(prefix_len, 4) || !aligned(n_rows, 4) || !aligned(LSE, 4)) return RAPID_EINVAL;
    if (!std::isfinite(softmax_scale)) return RAPID_EINVAL;
    const int64_t qk = kLatentHead + kLatentRope;
    const int64_t packed[11] = {n * H * qk, H * qk, qk,
                                kv_rows * H * kLatentHead, (int64_t)H * kLatentHead, kLatentHead,
                                kv_rows * H * kLatentHead, (int64_t)H * kLatentHead, kLatentHead,
                                kv_rows * kLatentRope, kLatentRope};
    const int64_t* s = strides ? strides : packed;
    if (!strides_ok(s, 11)) return RAPID_EINVAL;
    // rows are copied by their strides: a dimension that repeats a row has none
    const int64_t size[11] = {B, n, H, B, kv_rows, H, B, kv_rows, H, B, kv_rows};
    for (int i = 0; i < 11; ++i)
        if (size[i] > 1 && s[i] == 0) return RAPID_EINVAL;
    const PrefillPlan pl = plan_prefill(B, n, H, kv_rows);
    if (workspace_bytes < pl.bytes()) return RAPID_ENOMEM;
    LatentPrefillParams p{};
    char* ws = static_cast<char*>(workspace);
    p.part_acc = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + pl.acc);
    p.part_first = reinterpret_cast<int64_t*>(ws + pl.acc + pl.ml);
    p.ctas = pl.ctas;
    p.Q = Q; p.K = K; p.V = V; p.K_rope = K_rope;
    p.prefix_len = prefix_len; p.n_rows = n_rows; p.O = O; p.LSE = LSE;
    p.err = device_error_word();
    for (int i = 0; i < 3; ++i) { p.q_stride[i] = s[i]; p.k_stride[i] = s[3 + i]; p.v_stride[i] = s[6 + i]; }
    p.r_stride[0] = s[9]; p.r_stride[1] = s[10];
    p.kv_rows = kv_rows;
    p.B = B; p.n = n; p.H = H;
    p.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)qk)) * kLog2e;
    return status_of(launch_latent_prefill(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
