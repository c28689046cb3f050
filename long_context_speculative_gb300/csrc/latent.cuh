// Latent caches: one row a token for all heads of a layer (a normed latent vector and a rotated
// key), the parameter blocks of their kernels and the launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rapid {

constexpr int kLatent = 512;                 // latent values of a row: the values of the absorbed form
constexpr int kLatentRope = 64;              // rotated values behind them
constexpr int kLatentRow = kLatent + kLatentRope;
constexpr int kLatentGroup = 128;            // e4m3 codes that share a scale
constexpr int kLatentGroups = kLatent / kLatentGroup;
// 8-bit row: 512 codes, 64 bf16, 4 floats
constexpr int kLatentQ8Rope = kLatent;
constexpr int kLatentQ8Scale = kLatent + 2 * kLatentRope;
constexpr int kLatentQ8Row = kLatentQ8Scale + 4 * kLatentGroups;
constexpr int kLatentHead = 128;             // plain key width and value width of an expanded head
constexpr int kLatentMaxLayers = 128;

inline int latent_row_bytes(bool q8) { return q8 ? kLatentQ8Row : 2 * kLatentRow; }

struct LatentAppendParams {
    const void* kv;              // rows of 576 bf16: latent, key to rotate
    const void* q;               // rows of 64 bf16, or nullptr
    void* q_out;
    const void* weight;          // [512] bf16 or nullptr
    const float* inv_freq;       // [32]
    const int32_t* prefix_len;   // [B]
    const int32_t* row_offset;   // [B, n] or nullptr
    const int32_t* n_rows;       // [B] or nullptr
    uint8_t* cache;
    unsigned int* err;
    int64_t kv_batch, kv_token;                      // element strides
    int64_t q_batch, q_token, q_head, o_batch, o_token, o_head;
    int64_t cap;
    int B, n, H, slices;         // slices: warps that share a token's query heads
    int interleaved, q8;
    float eps;
};

struct LatentReadParams {
    const uint8_t* cache;
    const int32_t* first;        // [B] or nullptr
    const int32_t* n_rows;       // [B] or nullptr
    uint8_t* rows;               // [B, n, 576] bf16
    unsigned int* err;
    int64_t cap;
    int B, n, q8;
};

struct LatentCommitParams {
    uint8_t* cache[kLatentMaxLayers];
    const int32_t* prefix_len;   // [B]
    const int32_t* path;         // [B, n_q]
    const int32_t* n_acc;        // [B]
    unsigned int* err;
    int64_t cap;
    int n_q, row_bytes;
};

struct LatentAttnParams {
    const void* Q;               // [B, H, n_q, 576] bf16
    const uint8_t* cache;
    const int32_t* prefix_len;   // [B]
    const uint8_t* mask;         // [B, n_q, n_q] or nullptr (chain)
    void* O;                     // [B, H, n_q, 512] bf16
    float* LSE;                  // [B, H, n_q]
    // Partials of sequences with several splits, by slot: un-normalised outputs [S, H n_q, 512]
    // and their (running maximum, sum) in the log2 domain; a sequence's splits are the slots
    // part_first[b] .. + part_count[b] - 1.
    float* part_acc;
    float* part_ml;
    int* part_first;
    int* part_count;
    unsigned int* err;
    int64_t cap;
    int B, H, n_q, q8;
    int S, RB;                   // slots (S == B: one split each), row blocks
    float scale_log2;            // softmax scale * log2(e)
};

struct LatentPrefillParams {
    const void *Q, *K, *V, *K_rope;
    const int32_t* prefix_len;   // [B]
    const int32_t* n_rows;       // [B] or nullptr
    void* O;                     // [B, n, H, 128] bf16
    float* LSE;                  // [B, H, n]
    unsigned int* err;
    int64_t q_stride[3], k_stride[3], v_stride[3], r_stride[2];   // batch, token, head (elements)
    // Parts of blocks of tokens (ctas > 0): un-normalised O [2 ctas, 32, 256, 4] and (running maximum, sum) in
    // the log2 domain; where the key tiles of each block [B, blocks] start in the line, and its length
    float* part_acc;
    float* part_ml;
    int64_t* part_first;
    int64_t kv_rows;
    int B, H, n, ctas;
    int group;                   // heads (of all sequences) whose blocks are taken longest first, ctas == 0
    float scale_log2;
};

cudaError_t launch_latent_append(LatentAppendParams p, cudaStream_t st);
cudaError_t launch_latent_read(const LatentReadParams& p, cudaStream_t st);
cudaError_t launch_latent_commit(const LatentCommitParams& p, int layers, int B, cudaStream_t st);
int latent_attn_block_rows(int R);                    // rows of a block for R = H n_q rows
int latent_attn_slots(int B, int R, int64_t cap);
cudaError_t launch_latent_attn(const LatentAttnParams& p, cudaStream_t st);
int latent_prefill_ctas(int B, int n, int H, int64_t kv_rows);
size_t latent_prefill_block_rows();                   // tokens of a block
cudaError_t launch_latent_prefill(LatentPrefillParams p, cudaStream_t st);

}  // namespace rapid
