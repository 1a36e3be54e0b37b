// rq_lora.h -- launchers of the adapter kernels (rq_lora.cu).
#pragma once

#include "rq_internal.h"

namespace rq {

struct LoraArgs {
    const uint16_t* x;                       // fp16 [M, K]
    const uint16_t* A;                       // fp16 [L, R, K]
    const uint16_t* B;                       // fp16 [L, N, R]
    const int32_t* ids;                      // [M]
    const int32_t* ranks;                    // [L] or NULL: R
    const float* scale;                      // [L] or NULL: 1
    const void* y;                           // [M, N]
    void* out;                               // [M, N]
    uint4* work;                             // many tokens only
    int* status;
    int64_t N;
    int M, K, R, L;
    bool relu_sq;
};

// Up to this many tokens each one is taken by itself (a cluster of CTAs); more
// are taken in tiles.
constexpr int kLoraTokens = 32;

cudaError_t launch_lora_tokens(const LoraArgs& a, bool half, cudaStream_t s);
cudaError_t launch_lora_tiles(const LoraArgs& a, bool half, cudaStream_t s);

}  // namespace rq
