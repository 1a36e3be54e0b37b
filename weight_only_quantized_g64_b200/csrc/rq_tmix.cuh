// rq_tmix.cuh -- what the kernels of the time-mix recurrence share: packed
// fp32 arithmetic, the decay, element loads, the sequence table.
//
// Per head, with a 64 x 64 fp32 state S (rows i: value, columns j: key),
//   w_t = exp(-e^{-1/2} sigmoid(d_t))
//   S_t = S_{t-1} diag(w_t) + (S_{t-1} a_t) b_t^T + v_t k_t^T,   y_t = S_t r_t.
// Every row of S evolves by itself: its update needs the row, the five key
// vectors of the token and one value v_i.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "rq_internal.h"
#include "rq_once.h"
#include "rq_pairs.cuh"

namespace rq {

constexpr int kHead = 64;                    // channels of a head
constexpr int kTmixChunk = 16;               // tokens between two stored states (training)
constexpr float kDecay = 0.60653065971263342f;   // e^{-1/2}
constexpr float kLn2 = 0.69314718055994531f;

struct TmixArgs {
    const void* in[6];                       // r, d, k, v, a, b: [T, H, 64], rows ld elements apart
    const void* dy;                          // backward: [T, H, 64]
    void* out[6];                            // forward: y; backward: dr, dd, dk, dv, da, db
    const float* state_in;                   // [*, H, 64, 64] or NULL
    float* state_out;                        // [*, H, 64, 64] or NULL
    const int32_t* slots;                    // [S] state of each sequence, or NULL: its own index
    const int32_t* seq_start;                // [S + 1]
    float* ckpt;                             // forward states before each chunk, or NULL
    float* gckpt;                            // backward: gradient of the state after each chunk
    int* status;
    int64_t T, ld, n_slots;
    int S, H;
};

// ---------------------------------------------------------------- elements --
// Eight consecutive elements, 16-byte aligned (fp16: one load, fp32: two).
struct Raw8 {
    uint4 u[2];
};
template <typename T>
__device__ __forceinline__ Raw8 load8(const T* p) {
    Raw8 r;
    r.u[0] = __ldg(reinterpret_cast<const uint4*>(p));
    if constexpr (sizeof(T) == 4) r.u[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    return r;
}
template <typename T>
__device__ __forceinline__ void cvt8(const Raw8& r, float* f) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4*>(&r.u[0]);
        const float4 b = *reinterpret_cast<const float4*>(&r.u[1]);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        const __half2* h = reinterpret_cast<const __half2*>(&r.u[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(h[i]);
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}
template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
    if constexpr (sizeof(T) == 4) return __ldg(reinterpret_cast<const float4*>(p));
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = v;
    } else {
        const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                  *reinterpret_cast<const uint32_t*>(&b));
    }
}
template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    if constexpr (sizeof(T) == 4) return v;
    else return __half2float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
    if constexpr (sizeof(T) == 4) return v;
    else return __float2half_rn(v);
}

// ------------------------------------------------------------------- decay --
// sigmoid(d), relative error at most (|d| + 6) 2^-24 below 0 and 2^-21 above (the
// hardware's 2^x and 1/x are good to 2^-22 and 2^-23, d log2(e) is rounded once):
// it scales log w, which is small where that grows.  Below -87.3, where it would be
// under 2^-126, it is 0.
__device__ __forceinline__ float exp2_approx(float x) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    return e;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float exp_minus(float d) { return exp2_approx(d * -1.4426950408889634f); }
__device__ __forceinline__ float decay_gate(float d) { return rcp_approx(1.f + exp_minus(d)); }
// Its derivative, s (1 - s).  From 0 on 1 - s is e^-d s, as the difference would lose
// its bits (9e-3 of it at d = 12, all from 17 on); below, e^-d may be infinite.
__device__ __forceinline__ float decay_gate_slope(float d) {
    const float e = exp_minus(d), s = rcp_approx(1.f + e);
    return s * (d >= 0.f ? e * s : 1.f - s);
}
__device__ __forceinline__ float log2_decay(float d) { return -kDecay / kLn2 * decay_gate(d); }
// e^x - 1 for -ln 2 <= x <= 0 by its series x (1 + x/2! + x^2/3! + ...): nine terms
// leave less than 0.7^9 / 10! < 2^-26 of it.
__device__ __forceinline__ float expm1_near(float x) {
    float p = 1.f / 362880.f;
    p = fmaf(p, x, 1.f / 40320.f);
    p = fmaf(p, x, 1.f / 5040.f);
    p = fmaf(p, x, 1.f / 720.f);
    p = fmaf(p, x, 1.f / 120.f);
    p = fmaf(p, x, 1.f / 24.f);
    p = fmaf(p, x, 1.f / 6.f);
    p = fmaf(p, x, 0.5f);
    p = fmaf(p, x, 1.f);
    return x * p;
}
// w - 1: the update w S = S + (w - 1) S then rounds S once, and a decay near 1
// keeps its distance from 1 over thousands of steps (w itself, rounded to 24
// bits, would be off by up to 2^-25 in every step, in the same direction).
__device__ __forceinline__ float decay_m1(float d) { return expm1_near(-kDecay * decay_gate(d)); }

// --------------------------------------------------------------- sequences --
// Tokens [lo, hi) of sequence i; false (and a status) for offsets that are
// not 0 <= lo <= hi <= T.
__device__ __forceinline__ bool sequence_of(const TmixArgs& p, int i, int& lo, int& hi) {
    lo = p.seq_start[i];
    hi = p.seq_start[i + 1];
    if (lo >= 0 && hi >= lo && hi <= p.T) return true;
    if (p.status != nullptr && threadIdx.x == 0) atomicMax(p.status, RQ_ERR_RANGE);
    return false;
}
// State of sequence i, -1 for none (a negative slot, or one out of range,
// which also sets the status).
__device__ __forceinline__ int64_t state_of(const TmixArgs& p, int i) {
    if (p.slots == nullptr) return i;
    const int s = p.slots[i];
    if (s < p.n_slots) return s < 0 ? -1 : s;
    if (p.status != nullptr && threadIdx.x == 0) atomicMax(p.status, RQ_ERR_RANGE);
    return -1;
}
// First stored state of a sequence: sequences of len tokens have
// ceil(len / chunk) of them, and lo / chunk + i leaves room for each.
__device__ __forceinline__ int64_t ckpt_base(int lo, int i) { return lo / kTmixChunk + i; }

// The scan in pairs of tokens (few heads); launch_tmix_scan chooses.
cudaError_t launch_tmix_pairs(const TmixArgs& a, bool half, bool reverse, cudaStream_t s);
cudaError_t launch_tmix_scan(const TmixArgs& a, bool half, bool reverse, cudaStream_t s);
cudaError_t launch_tmix_step(const TmixArgs& a, bool half, cudaStream_t s);
cudaError_t launch_tmix_chunks_bwd(const TmixArgs& a, bool half, cudaStream_t s);

}  // namespace rq
