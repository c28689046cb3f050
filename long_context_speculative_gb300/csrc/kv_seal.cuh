// Sealing of full tail blocks into 8-bit pages: parameter block, the per-sequence plan
// shared by its two kernels, and launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rapid {

constexpr int kPageTokens = 64;
constexpr int kSealMaxLayers = 128;
constexpr int kScaleExpMin = -64;   // smallest exponent of a block's scale

struct SealLayer {
    void* K;            // [B, Hkv, cap, d] tail caches
    void* V;
    uint8_t* pages;     // [n_pages, Hkv, 2, 64, d] e4m3
    float* scales;      // [n_pages, Hkv, 2]
};

struct SealPlan {
    const int32_t* page_table;   // [B, max_pages]
    const int32_t* sealed_len;   // [B]
    const int32_t* tail_len;     // [B]
    int64_t cap;
    int B, max_pages, n_pages, keep;
};

struct SealParams {
    SealLayer layer[kSealMaxLayers];
    SealPlan plan;
    unsigned int* err;
    int Hkv, d, parts;
};

cudaError_t launch_kv_seal(const SealParams& p, int layers, int dtype, cudaStream_t st);
cudaError_t launch_kv_seal_advance(const SealPlan& plan, int32_t* sealed_len, int32_t* tail_len,
                                   unsigned int* err, cudaStream_t st);

}  // namespace rapid
