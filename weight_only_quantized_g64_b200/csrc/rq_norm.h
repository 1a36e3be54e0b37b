// rq_norm.h -- launcher of the norm / gate / residual kernel (rq_norm.cu).
#pragma once

#include "rq_internal.h"

namespace rq {

struct NormArgs {
    const void *y, *add, *gate, *h;          // [M, D] of one type; y, add and gate with row strides
    void* h_out;                             // [M, D] of that type, or NULL
    void* x;                                 // fp16 [M, D], or NULL
    const float *post_weight, *post_bias, *pre_weight, *pre_bias, *alpha;   // [D] or NULL
    int64_t ld_y, ld_add, ld_gate, M;
    int D, post, post_group, pre, gate_act;  // post_group 0: the whole row
    float eps_post, eps_pre, inv_row, inv_group;     // 1 / D, 1 / post_group
};

cudaError_t launch_norm_residual(const NormArgs& a, bool half, cudaStream_t s);

}  // namespace rq
