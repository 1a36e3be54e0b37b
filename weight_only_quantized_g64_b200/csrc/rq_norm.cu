// rq_norm.cu -- the step between two projections: norm of a block's output,
// gate, residual with its scale, and the norm that the next projection reads.
//
//   u = (Norm_post(y) + add) * act(gate);   h' = h + alpha u;   x = Norm_pre(h')
//
// One CTA per row; a thread holds V pieces of 8 channels in registers, so each
// tensor is read once and each result written once: bound by those bytes.
// Mean and squared deviation come from one reduction: every thread forms them
// over its own values (two passes over registers) and pairs are joined by
//   delta = m2 - m1;  m = m1 + delta n2/(n1+n2);  M2 = M2_1 + M2_2 + delta^2 n1 n2/(n1+n2),
// which loses nothing when the mean is large against the deviation.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rq_norm.h"

namespace rq {
namespace {

struct Moments {
    float n, mean, m2;
};
__device__ __forceinline__ Moments join(Moments a, Moments b) {
    const float n = a.n + b.n;
    const float f = n > 0.f ? b.n / n : 0.f, d = b.mean - a.mean;
    return {n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * (a.n * f)};
}
__device__ __forceinline__ Moments join_xor(Moments a, int mask) {
    return join(a, {__shfl_xor_sync(0xffffffffu, a.n, mask), __shfl_xor_sync(0xffffffffu, a.mean, mask),
                    __shfl_xor_sync(0xffffffffu, a.m2, mask)});
}

template <typename T>
__device__ __forceinline__ void load8(const void* base, int64_t at, float* f) {
    const T* p = static_cast<const T*>(base) + at;
    if constexpr (sizeof(T) == 4) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
        const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(h[i]);
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}
template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t at, const float* f) {
    T* p = static_cast<T*>(base) + at;
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        uint4 u;
        __half2* h = reinterpret_cast<__half2*>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<uint4*>(p) = u;
    }
}

// The mean (0 for the rms norm) and 1 / sqrt(mean square + eps) of the
// values that `width` consecutive lanes (a power of two) or, width 0, the
// whole CTA hold.  v: V pieces of 8 values, the first `pieces` of them real.
template <int V>
__device__ __forceinline__ void stats(const float (*v)[8], int pieces, bool layer, int width, float eps,
                                      Moments* shared, float& mean, float& rstd) {
    Moments a = {8.f * pieces, 0.f, 0.f};
    if (layer) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += i < pieces ? v[i][j] : 0.f;
        a.mean = pieces > 0 ? s / a.n : 0.f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = v[i][j] - a.mean;
            a.m2 = i < pieces ? fmaf(d, d, a.m2) : a.m2;
        }
    // rms: every mean is 0, and joining leaves the sum of squares
    const int steps = width ? width : 32;
    for (int m = 1; m < steps; m <<= 1) a = join_xor(a, m);
    if (!width && blockDim.x > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) shared[warp] = a;
        __syncthreads();
        a = lane < warps ? shared[lane] : Moments{0.f, 0.f, 0.f};
        for (int m = 1; m < warps; m <<= 1) a = join_xor(a, m);
        a = {__shfl_sync(0xffffffffu, a.n, 0), __shfl_sync(0xffffffffu, a.mean, 0), __shfl_sync(0xffffffffu, a.m2, 0)};
    }
    mean = a.mean;
    rstd = rsqrtf(a.m2 / a.n + eps);
}

template <int V>
__device__ __forceinline__ void apply(float (*v)[8], int pieces, const NormArgs& p, bool post, int threads, float mean,
                                      float rstd) {
    const float* w = post ? p.post_weight : p.pre_weight;
    const float* b = post ? p.post_bias : p.pre_bias;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i >= pieces) break;
        const int c = (threadIdx.x + i * threads) * 8;
        float wv[8], bv[8];
        if (w != nullptr) load8<float>(w, c, wv);
        if (b != nullptr) load8<float>(b, c, bv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float f = (v[i][j] - mean) * rstd;
            if (w != nullptr) f *= wv[j];
            if (b != nullptr) f += bv[j];
            v[i][j] = f;
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(V == 1 ? 512 : 1024) norm_residual_kernel(const NormArgs p) {
    __shared__ Moments shared[2][32];
    const int64_t row = blockIdx.x;
    const int threads = blockDim.x, all = p.D / 8;
    // pieces threadIdx.x + i * threads < D / 8
    int pieces = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) pieces += static_cast<int>(threadIdx.x) + i * threads < all;
    float u[V][8];
    // one piece per thread: everything is in flight at once; with more, the
    // other rows of the SM hide the second group of loads (registers would not
    // hold it)
    constexpr bool EARLY = V == 1;
    float a[8], g[8], h[8];
    const auto others = [&](int c) {
        if (p.add != nullptr) load8<T>(p.add, row * p.ld_add + c, a);
        if (p.gate != nullptr) load8<T>(p.gate, row * p.ld_gate + c, g);
        if (p.h != nullptr) load8<T>(p.h, row * p.D + c, h);
    };
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (threadIdx.x + i * threads) * 8;
        if (i < pieces) load8<T>(p.y, row * p.ld_y + c, u[i]);
    }
    if (EARLY && pieces > 0) others(threadIdx.x * 8);
    if (p.post != RQ_NORM_NONE) {
        float mean, rstd;
        const bool layer = p.post == RQ_NORM_LAYER;
        if (p.post_group == 0) {
            stats<V>(u, pieces, layer, 0, p.eps_post, shared[0], mean, rstd);
            apply<V>(u, pieces, p, true, threads, mean, rstd);
        } else {                             // a group is 8 width channels of one piece row
            const int width = p.post_group / 8;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                stats<1>(&u[i], i < pieces, layer, width, p.eps_post, nullptr, mean, rstd);
                if (i < pieces) {
                    const int c = (threadIdx.x + i * threads) * 8;
                    float wv[8], bv[8];
                    if (p.post_weight != nullptr) load8<float>(p.post_weight, c, wv);
                    if (p.post_bias != nullptr) load8<float>(p.post_bias, c, bv);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float f = (u[i][j] - mean) * rstd;
                        if (p.post_weight != nullptr) f *= wv[j];
                        if (p.post_bias != nullptr) f += bv[j];
                        u[i][j] = f;
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i >= pieces) break;
        const int c = (threadIdx.x + i * threads) * 8;
        float al[8];
        if (!EARLY) others(c);
        if (p.alpha != nullptr) load8<float>(p.alpha, c, al);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float f = u[i][j];
            if (p.add != nullptr) f += a[j];
            if (p.gate != nullptr) {
                const float x = g[j];
                f *= p.gate_act == RQ_GATE_IDENTITY ? x : (p.gate_act == RQ_GATE_SILU ? x : 1.f) / (1.f + expf(-x));
            }
            if (p.alpha != nullptr) f *= al[j];
            if (p.h != nullptr) f += h[j];
            u[i][j] = f;
        }
        if (p.h_out != nullptr) store8<T>(p.h_out, row * p.D + c, u[i]);
    }
    if (p.x == nullptr) return;
    if (p.pre != RQ_NORM_NONE) {
        float mean, rstd;
        stats<V>(u, pieces, p.pre == RQ_NORM_LAYER, 0, p.eps_pre, shared[1], mean, rstd);
        apply<V>(u, pieces, p, false, threads, mean, rstd);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < pieces) store8<__half>(p.x, row * p.D + (threadIdx.x + i * threads) * 8, u[i]);
}

template <typename T>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
    const int pieces = a.D / 8;
    const auto threads = [&](int v) { return ((pieces + v - 1) / v + 31) / 32 * 32; };
    const unsigned rows = static_cast<unsigned>(a.M);
    if (pieces <= 512) norm_residual_kernel<T, 1><<<rows, threads(1), 0, s>>>(a);
    else norm_residual_kernel<T, 2><<<rows, threads(2), 0, s>>>(a);
    return cudaGetLastError();
}

bool mis(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

}  // namespace

cudaError_t launch_norm_residual(const NormArgs& a, bool half, cudaStream_t s) {
    return half ? launch<__half>(a, s) : launch<float>(a, s);
}

}  // namespace rq

using namespace rq;

extern "C" rq_status rq_norm_residual(const void* y, int64_t ld_y, int64_t M, int64_t D, int dtype, int post,
                                      int64_t post_group, const float* post_weight, const float* post_bias,
                                      float eps_post, const void* add, int64_t ld_add, const void* gate,
                                      int64_t ld_gate, int gate_act, const void* h, const float* alpha, int pre,
                                      const float* pre_weight, const float* pre_bias, float eps_pre, void* h_out,
                                      uint16_t* x, rq_stream_t stream) {
    if (dtype != RQ_OUT_F32 && dtype != RQ_OUT_F16) return RQ_ERR_RANGE;
    if (post < RQ_NORM_NONE || post > RQ_NORM_RMS || pre < RQ_NORM_NONE || pre > RQ_NORM_RMS) return RQ_ERR_RANGE;
    if (gate_act < RQ_GATE_IDENTITY || gate_act > RQ_GATE_SILU) return RQ_ERR_RANGE;
    if (!(eps_post >= 0.f) || !(eps_pre >= 0.f)) return RQ_ERR_RANGE;
    if (M < 1 || M >= (int64_t{1} << 31) || D < 64 || D % 64 != 0 || D > 16384) return RQ_ERR_SHAPE;
    if (post_group != 0 && post_group != D && (post_group < 8 || post_group > 256 || (post_group & (post_group - 1)) != 0 ||
                            D % post_group != 0))
        return RQ_ERR_SHAPE;
    const int64_t strides[3] = {ld_y, add != nullptr ? ld_add : D, gate != nullptr ? ld_gate : D};
    for (int64_t ld : strides)
        if (ld < D || ld % 8 != 0 || ld >= (int64_t{1} << 32)) return RQ_ERR_SHAPE;
    if (y == nullptr || (h_out == nullptr && x == nullptr)) return RQ_ERR_NULL;
    const void* all[] = {y, post_weight, post_bias, add, gate, h, alpha, pre_weight, pre_bias, h_out, x};
    for (const void* q : all)
        if (mis(q, 16)) return RQ_ERR_ALIGN;
    NormArgs a = {};
    a.y = y;
    a.add = add;
    a.gate = gate;
    a.h = h;
    a.h_out = h_out;
    a.x = x;
    a.post_weight = post_weight;
    a.post_bias = post_bias;
    a.pre_weight = pre_weight;
    a.pre_bias = pre_bias;
    a.alpha = alpha;
    a.ld_y = ld_y;
    a.ld_add = ld_add;
    a.ld_gate = ld_gate;
    a.M = M;
    a.D = static_cast<int>(D);
    a.post = post;
    a.post_group = post_group == D ? 0 : static_cast<int>(post_group);
    a.pre = pre;
    a.gate_act = gate_act;
    a.eps_post = eps_post;
    a.eps_pre = eps_pre;
    const cudaError_t e =
        launch_norm_residual(a, dtype == RQ_OUT_F16, reinterpret_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) return RQ_OK;
    record_cuda_error(e);
    return RQ_ERR_CUDA;
}
