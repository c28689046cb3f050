// C ABI of the 8-bit cache: append with norm and rotation, sealing, attention.
#include <cmath>
#include <cstdint>

#include "attn_q8.cuh"
#include "common.cuh"
#include "kv_seal.cuh"
#include "qkv_append.cuh"
#include "rapid.h"

namespace rapid {

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int dtype) { return dtype == RAPID_DTYPE_F32 || dtype == RAPID_DTYPE_BF16; }

struct Q8Plan {
    int S;               // (sequence, split) slots per KV head
    size_t rows;         // partial rows
    size_t bytes;
};

bool attn_q8_args_ok(int B, int Hq, int Hkv, int d, int n_q, int64_t cap, int max_pages, int dtype) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return false;
    if ((int64_t)B * Hkv > 65535 || (d != 64 && d != 128)) return false;
    if (n_q < 1 || n_q > RAPID_MAX_NQ || !dtype_ok(dtype)) return false;
    if (cap < n_q || cap > ((int64_t)1 << 31)) return false;
    if (max_pages < 1 || max_pages > RAPID_Q8_MAX_PAGES) return false;
    // key tiles of all sequences are counted in 32 bits
    if ((int64_t)B * (max_pages + cap / kQ8SimtTile + 2) >= (int64_t)1 << 31) return false;
    return (int64_t)(Hq / Hkv) * n_q <= 4096;
}

Q8Plan plan_attn_q8(int B, int Hq, int Hkv, int d, int n_q, int dtype) {
    const int64_t R = (int64_t)(Hq / Hkv) * n_q;
    const int64_t sms = sm_count();
    int64_t S;
    if (dtype == RAPID_DTYPE_BF16) {
        // tensor cores: one CTA on every SM, and at least as many waves of them as give every
        // sequence a slot
        const int64_t per_slot = (int64_t)Hkv * q8_row_blocks((int)R);
        const int64_t waves = (B * per_slot + sms - 1) / sms;
        S = waves * sms / per_slot;
        // A second wave may hold few CTAs (20 sequences of 8 heads: 160 on 152 SMs).  More waves
        // of shorter splits then cost less: k splits of a sequence take w / k of its time, and
        // the start and end of a CTA, 1/32 of it (8 tiles of 256), w times.  20 sequences of 8
        // heads, 1 query, d = 128: 337 -> 248 us at 32K, 58 -> 53 us at 4K; 32 or 38 sequences
        // (nearly two full waves) stay with two.
        double least = waves * (1 + 1. / 32);
        for (int64_t w = waves + 1; waves > 1 && w <= waves + 2; ++w) {
            const int64_t slots = w * sms / per_slot;
            const double cost = w * ((double)B / (slots / B * B) + 1. / 32);
            if (cost < least) { least = cost; S = slots; }
        }
    } else {
        // CUDA cores: slots for two CTAs on every SM, which is what runs at once up to 32 rows; above,
        // one CTA fits (182 or 214 registers a thread) and the slots are two waves
        S = 2 * sms / (Hkv * ((R + kQ8SimtRows - 1) / kQ8SimtRows));
        if (S > 512) S = 512;
    }
    if (S < B) S = B;
    Q8Plan pl;
    pl.S = (int)S;
    pl.rows = (size_t)Hkv * S * R;
    pl.bytes = align_up(pl.rows * d * sizeof(float)) + align_up(pl.rows * 2 * sizeof(float)) +
               2 * align_up((size_t)B * Hkv * sizeof(int));
    return pl;
}

}  // namespace
}  // namespace rapid

using namespace rapid;

extern "C" {

rapid_status rapid_qkv_append(const void* q, const void* k, const void* v, const int64_t* strides,
                              int dtype, int B, int n, int Hq, int Hkv, int d,
                              const void* q_weight, const void* k_weight, float eps,
                              const float* inv_freq, int rot_dim, uint32_t flags,
                              const int32_t* prefix_len, const int32_t* pos_offset,
                              const int32_t* row_offset, const int32_t* n_rows, void* Q,
                              void* Kcache, void* Vcache, int64_t kv_capacity, void* stream) {
    if (!q || !k || !v || !prefix_len || !Q || !Kcache || !Vcache) return RAPID_EINVAL;
    if (B < 1 || n < 1 || Hq < 1 || Hkv < 1 || (d != 64 && d != 128) || !dtype_ok(dtype))
        return RAPID_EINVAL;
    if (Hq > 65535 || Hkv > 65535 || (int64_t)B * n > ((int64_t)1 << 31)) return RAPID_EINVAL;
    if (rot_dim < 0 || rot_dim > d || rot_dim % 16 != 0 || (rot_dim > 0 && !inv_freq))
        return RAPID_EINVAL;
    if ((flags & ~(uint32_t)RAPID_ROPE_INTERLEAVED) != 0) return RAPID_EINVAL;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return RAPID_EINVAL;
    if (kv_capacity < 1 || kv_capacity > ((int64_t)1 << 31)) return RAPID_EINVAL;
    const void* rows16[] = {q, k, v, Q, Kcache, Vcache, q_weight, k_weight};
    for (const void* x : rows16)
        if (x && !aligned(x, 16)) return RAPID_EINVAL;
    const void* words[] = {inv_freq, prefix_len, pos_offset, row_offset, n_rows};
    for (const void* x : words)
        if (x && !aligned(x, 4)) return RAPID_EINVAL;
    QkvAppendParams p{};
    const int64_t qs = (int64_t)Hq * d, ks = (int64_t)Hkv * d;
    const int64_t packed[6] = {n * qs, qs, n * ks, ks, n * ks, ks};
    const int64_t* s = strides ? strides : packed;
    for (int i = 0; i < 6; ++i)
        if (s[i] < 0 || s[i] * (dtype == RAPID_DTYPE_BF16 ? 2 : 4) % 16 != 0) return RAPID_EINVAL;
    p.q = q; p.k = k; p.v = v;
    p.q_batch = s[0]; p.q_token = s[1]; p.k_batch = s[2]; p.k_token = s[3];
    p.v_batch = s[4]; p.v_token = s[5];
    p.q_weight = q_weight; p.k_weight = k_weight; p.inv_freq = inv_freq;
    p.prefix_len = prefix_len; p.pos_offset = pos_offset; p.row_offset = row_offset;
    p.n_rows = n_rows; p.Q = Q; p.K = Kcache; p.V = Vcache;
    p.err = device_error_word();
    p.cap = kv_capacity;
    p.B = B; p.n = n; p.Hq = Hq; p.Hkv = Hkv; p.d = d; p.rot = rot_dim;
    p.interleaved = (flags & RAPID_ROPE_INTERLEAVED) ? 1 : 0;
    p.eps = eps;
    return launch_qkv_append(p, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? RAPID_OK
               : RAPID_ECUDA;
}

rapid_status rapid_kv_seal(void* const* K_layers, void* const* V_layers, void* const* page_layers,
                           float* const* scale_layers, int layers, int dtype, int B, int Hkv, int d,
                           int64_t tail_capacity, int keep_rows, int n_pages,
                           const int32_t* page_table, int max_pages, const int32_t* sealed_len,
                           const int32_t* tail_len, void* stream) {
    if (!K_layers || !V_layers || !page_layers || !scale_layers || !page_table || !sealed_len ||
        !tail_len)
        return RAPID_EINVAL;
    if (layers < 1 || layers > RAPID_COMMIT_MAX_LAYERS || !dtype_ok(dtype)) return RAPID_EINVAL;
    if (B < 1 || Hkv < 1 || (int64_t)B * Hkv > 65535 || (d != 64 && d != 128)) return RAPID_EINVAL;
    if (tail_capacity < 1 || tail_capacity > ((int64_t)1 << 31) || keep_rows < 0 || n_pages < 1)
        return RAPID_EINVAL;
    if (max_pages < 1 || max_pages > RAPID_Q8_MAX_PAGES) return RAPID_EINVAL;
    if (!aligned(page_table, 4) || !aligned(sealed_len, 4) || !aligned(tail_len, 4)) return RAPID_EINVAL;
    SealParams p{};
    for (int l = 0; l < layers; ++l) {
        if (!K_layers[l] || !V_layers[l] || !page_layers[l] || !scale_layers[l]) return RAPID_EINVAL;
        if (!aligned(K_layers[l], 16) || !aligned(V_layers[l], 16) || !aligned(page_layers[l], 16) ||
            !aligned(scale_layers[l], 4))
            return RAPID_EINVAL;
        p.layer[l].K = K_layers[l];
        p.layer[l].V = V_layers[l];
        p.layer[l].pages = static_cast<uint8_t*>(page_layers[l]);
        p.layer[l].scales = scale_layers[l];
    }
    p.plan = SealPlan{page_table, sealed_len, tail_len, tail_capacity, B, max_pages, n_pages, keep_rows};
    p.err = device_error_word();
    p.Hkv = Hkv;
    p.d = d;
    return launch_kv_seal(p, layers, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? RAPID_OK
               : RAPID_ECUDA;
}

rapid_status rapid_kv_seal_advance(int32_t* sealed_len, int32_t* tail_len, const int32_t* page_table,
                                   int B, int max_pages, int n_pages, int64_t tail_capacity,
                                   int keep_rows, void* stream) {
    if (!sealed_len || !tail_len || !page_table || B < 1 || n_pages < 1 || keep_rows < 0)
        return RAPID_EINVAL;
    if (max_pages < 1 || max_pages > RAPID_Q8_MAX_PAGES) return RAPID_EINVAL;
    if (tail_capacity < 1 || tail_capacity > ((int64_t)1 << 31)) return RAPID_EINVAL;
    if (!aligned(page_table, 4) || !aligned(sealed_len, 4) || !aligned(tail_len, 4)) return RAPID_EINVAL;
    const SealPlan plan{page_table, sealed_len, tail_len, tail_capacity, B, max_pages, n_pages, keep_rows};
    return launch_kv_seal_advance(plan, sealed_len, tail_len, device_error_word(),
                                  static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? RAPID_OK
               : RAPID_ECUDA;
}

size_t rapid_verify_attn_q8_workspace_size(int B, int Hq, int Hkv, int d, int n_q,
                                           int64_t tail_capacity, int max_pages, int dtype) {
    if (!attn_q8_args_ok(B, Hq, Hkv, d, n_q, tail_capacity, max_pages, dtype)) return 0;
    return plan_attn_q8(B, Hq, Hkv, d, n_q, dtype).bytes;
}

rapid_status rapid_verify_attn_q8(const void* Q, const void* K_tail, const void* V_tail,
                                  const void* pages, const float* scales, const int32_t* page_table,
                                  int dtype, int B, int Hq, int Hkv, int d, int n_q,
                                  int64_t tail_capacity, int n_pages, int max_pages,
                                  const int32_t* sealed_len, const int32_t* tail_len,
                                  const uint8_t* spec_mask, float softmax_scale, void* O, float* LSE,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    if (!Q || !K_tail || !V_tail || !pages || !scales || !page_table || !sealed_len || !tail_len ||
        !O || !LSE || !workspace)
        return RAPID_EINVAL;
    if (!attn_q8_args_ok(B, Hq, Hkv, d, n_q, tail_capacity, max_pages, dtype)) return RAPID_EINVAL;
    if (n_pages < 1 || (int64_t)n_pages * Hkv * 128 > 0x7fffffff) return RAPID_EINVAL;
    const void* rows16[] = {Q, K_tail, V_tail, pages, O, workspace};
    for (const void* x : rows16)
        if (!aligned(x, 16)) return RAPID_EINVAL;
    const void* words[] = {page_table, sealed_len, tail_len, LSE};
    for (const void* x : words)
        if (!aligned(x, 4)) return RAPID_EINVAL;
    if (!aligned(scales, 8)) return RAPID_EINVAL;
    if (!std::isfinite(softmax_scale)) return RAPID_EINVAL;
    const Q8Plan pl = plan_attn_q8(B, Hq, Hkv, d, n_q, dtype);
    if (workspace_bytes < pl.bytes) return RAPID_ENOMEM;

    AttnQ8Params p{};
    p.Q = Q; p.K = K_tail; p.V = V_tail;
    p.pages = static_cast<const uint8_t*>(pages);
    p.scales = scales; p.page_table = page_table; p.sealed_len = sealed_len; p.tail_len = tail_len;
    p.mask = spec_mask; p.O = O; p.LSE = LSE;
    p.err = device_error_word();
    p.cap = tail_capacity;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.d = d; p.n_q = n_q; p.G = Hq / Hkv; p.R = p.G * n_q;
    p.max_pages = max_pages; p.n_pages = n_pages; p.S = pl.S;
    p.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)d)) * kLog2e;
    char* ws = static_cast<char*>(workspace);
    p.part_acc = reinterpret_cast<float*>(ws);
    ws += align_up(pl.rows * d * sizeof(float));
    p.part_ml = reinterpret_cast<float*>(ws);
    ws += align_up(pl.rows * 2 * sizeof(float));
    p.part_first = reinterpret_cast<int*>(ws);
    ws += align_up((size_t)B * Hkv * sizeof(int));
    p.part_count = reinterpret_cast<int*>(ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == RAPID_DTYPE_BF16 ? launch_attn_q8_tc(p, st) : launch_attn_q8_simt(p, st);
    if (e != cudaSuccess) return RAPID_ECUDA;
    return launch_attn_q8_merge(p, dtype, st) == cudaSuccess ? RAPID_OK : RAPID_ECUDA;
}

}  // extern "C"
