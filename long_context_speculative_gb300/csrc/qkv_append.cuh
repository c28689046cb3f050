// Norm, rotation and append of a step's projection rows: parameter block and launcher.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rapid {

struct QkvAppendParams {
    const void* q;              // rows [B, n, Hq, d] at the strides below
    const void* k;              // rows [B, n, Hkv, d]
    const void* v;
    int64_t q_batch, q_token;   // strides in elements
    int64_t k_batch, k_token;
    int64_t v_batch, v_token;
    const void* q_weight;       // [d] or nullptr: no norm
    const void* k_weight;
    const float* inv_freq;      // [rot / 2]
    const int32_t* prefix_len;  // [B]
    const int32_t* pos_offset;  // [B] or nullptr
    const int32_t* row_offset;  // [B, n] or nullptr: row i sits at offset i
    const int32_t* n_rows;      // [B] or nullptr: n rows each
    void* Q;                    // [B, Hq, n, d]
    void* K;                    // [B, Hkv, cap, d]
    void* V;
    unsigned int* err;
    int64_t cap;
    int B, n, Hq, Hkv, d, rot;
    int interleaved;
    float eps;
    int slices;                 // warps that share the heads of one token
};

cudaError_t launch_qkv_append(QkvAppendParams p, int dtype, cudaStream_t st);

}  // namespace rapid
