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
    float* work;                             // [ksplit, M, R] (many tokens only)
    int* status;
    int64_t N;
    int M, K, R, L, ksplit;
    bool relu_sq;
};

// Up to this many tokens each one is taken by itself (a cluster of CTAs); more
// are taken in tiles.
constexpr int kLoraTokens = 32;

// K splits of the tiled form: [ksplit, M, R] partial sums in the workspace.
int lora_ksplit(int64_t M, int64_t K);

cudaError_t launch_lora_tokens(const LoraArgs& a, bool half, cudaStream_t s);
cudaError_t launch_lora_tiles(const LoraArgs& a, bool half, cudaStream_t s);

}  // namespace rq
