// rq_norm.cu -- the step between two projections: norm of a block's output,
// gate, residual with its scale, and the norm that the next projection reads.
//
//   u = (Norm_post(y) + add) * act(gate);   h' = h + alpha u;   x = Norm_pre(h')
//
// A CTA takes a row at a time; a thread holds V pieces of 8 channels in
// registers, so each tensor is read once and each result written once: bound by
// those bytes.  Rows of up to 4096 channels are taken by CTAs that stay and
// bring the next rows' pieces into shared memory meanwhile (a thread waits for
// its own pieces only); longer rows, whose ring would not fit, are loaded as
// they come, a CTA each.
// Mean and squared deviation come from one reduction: every thread forms them
// over its own values (two passes over registers) and pairs are joined by
//   delta = m2 - m1;  m = m1 + delta n2/(n1+n2);  M2 = M2_1 + M2_2 + delta^2 n1 n2/(n1+n2),
// which loses nothing when the mean is large against the deviation.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <algorithm>

#include "rq_norm.h"
#include "rq_once.h"
#include "rq_pairs.cuh"

namespace rq {
namespace {

struct Moments {
    float n, mean, m2;
};
__device__ __forceinline__ Moments join(Moments a, Moments b) {
    const float n = a.n + b.n;
    const float f = b.n > 0.f ? __fdividef(b.n, n) : 0.f, d = b.mean - a.mean;
    return {n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * (a.n * f)};
}
__device__ __forceinline__ Moments join_xor(Moments a, int mask) {
    return join(a, {__shfl_xor_sync(0xffffffffu, a.n, mask), __shfl_xor_sync(0xffffffffu, a.mean, mask),
                    __shfl_xor_sync(0xffffffffu, a.m2, mask)});
}

// Eight neighbouring channels, as four pairs.
struct Piece {
    uint64_t v[4];
};
__device__ __forceinline__ uint64_t both(float f) { return pack2(f, f); }
template <typename T>
__device__ __forceinline__ Piece expand(uint4 a, uint4 b) {
    Piece r;
    if constexpr (sizeof(T) == 4) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&a), y = *reinterpret_cast<const ulonglong2*>(&b);
        r.v[0] = x.x; r.v[1] = x.y;
        r.v[2] = y.x; r.v[3] = y.y;
    } else {
        const __half2* h = reinterpret_cast<const __half2*>(&a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(h[i]);
            r.v[i] = pack2(f.x, f.y);
        }
    }
    return r;
}
template <typename T>
__device__ __forceinline__ Piece load(const void* base, int64_t at) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const T*>(base) + at);
    return expand<T>(__ldg(p), sizeof(T) == 4 ? __ldg(p + 1) : make_uint4(0u, 0u, 0u, 0u));
}
template <typename T>
__device__ __forceinline__ void store(void* base, int64_t at, const Piece& u) {
    T* p = static_cast<T*>(base) + at;
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(u.v[0], u.v[1]);
        reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(u.v[2], u.v[3]);
    } else {
        uint4 w;
        __half2* h = reinterpret_cast<__half2*>(&w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(u.v[i]);
            h[i] = __floats2half2_rn(f.x, f.y);
        }
        *reinterpret_cast<uint4*>(p) = w;
    }
}
__device__ __forceinline__ void times(Piece& u, const Piece& f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u.v[i] = mul2(u.v[i], f.v[i]);
}
__device__ __forceinline__ void plus(Piece& u, const Piece& f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u.v[i] = add2(u.v[i], f.v[i]);
}
__device__ __forceinline__ float sum(uint64_t p) {
    const float2 f = unpack2(p);
    return f.x + f.y;
}

constexpr int MAX_WARPS = 32;

// The mean (0 for the rms norm) and 1 / sqrt(mean square + eps) of the 1 / inv_n
// values that `width` consecutive lanes (a power of two) or, width 0, the whole
// CTA hold.  v: V pieces, the first `pieces` of them real, the others zeros.
template <int V>
__device__ __forceinline__ void stats(const Piece* v, int pieces, bool layer, int width, float eps, float inv_n,
                                      Moments* shared, float& mean, float& rstd) {
    Moments a = {8.f * pieces, 0.f, 0.f};
    if (layer && pieces > 0) {
        uint64_t s = add2(add2(v[0].v[0], v[0].v[1]), add2(v[0].v[2], v[0].v[3]));
#pragma unroll
        for (int i = 1; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s = add2(s, v[i].v[j]);
        a.mean = V == 1 ? sum(s) * 0.125f : __fdividef(sum(s), a.n);
    }
    if (pieces > 0) {
        const uint64_t away = both(-a.mean);
        uint64_t s = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (V == 1 || i < pieces) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t d = layer ? add2(v[i].v[j], away) : v[i].v[j];
                    s = fma2(d, d, s);
                }
            }
        a.m2 = sum(s);
    }
    if (width) {
        for (int m = 1; m < width; m <<= 1) {
            if (layer) a = join_xor(a, m);
            else a.m2 += __shfl_xor_sync(0xffffffffu, a.m2, m);
        }
    } else {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (layer) {
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) a = join_xor(a, m);
            if (lane == 0) shared[warp] = a;
        } else {
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) a.m2 += __shfl_xor_sync(0xffffffffu, a.m2, m);
            if (lane == 0) shared[warp].m2 = a.m2;
        }
        __syncthreads();
        // the first 16 lanes (a CTA of 1024 threads: all) join the warps' parts, whatever their number
        if (layer) {
            a = lane < warps ? shared[lane] : Moments{0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 1; m < 16; m <<= 1) a = join_xor(a, m);
            if (warps > 16) a = join_xor(a, 16);
            a.mean = __shfl_sync(0xffffffffu, a.mean, 0);
        } else {
            a.m2 = lane < warps ? shared[lane].m2 : 0.f;
#pragma unroll
            for (int m = 1; m < 16; m <<= 1) a.m2 += __shfl_xor_sync(0xffffffffu, a.m2, m);
            if (warps > 16) a.m2 += __shfl_xor_sync(0xffffffffu, a.m2, 16);
        }
        a.m2 = __shfl_sync(0xffffffffu, a.m2, 0);
    }
    mean = a.mean;
    rstd = rsqrtf(a.m2 * inv_n + eps);
}

__device__ __forceinline__ void apply(Piece& v, const NormArgs& p, bool post, int c, float mean, float rstd) {
    const float* w = post ? p.post_weight : p.pre_weight;
    const float* b = post ? p.post_bias : p.pre_bias;
    if ((post ? p.post : p.pre) == RQ_NORM_LAYER) {
        const uint64_t away = both(-mean);
#pragma unroll
        for (int j = 0; j < 4; ++j) v.v[j] = add2(v.v[j], away);
    }
    const uint64_t r = both(rstd);
#pragma unroll
    for (int j = 0; j < 4; ++j) v.v[j] = mul2(v.v[j], r);
    if (w != nullptr) times(v, load<float>(w, c));
    if (b != nullptr) plus(v, load<float>(b, c));
}

template <int V>
__device__ __forceinline__ void normed(Piece* u, int pieces, const NormArgs& p, bool post, int threads,
                                       Moments* shared) {
    const int kind = post ? p.post : p.pre;
    if (kind == RQ_NORM_NONE) return;
    const bool layer = kind == RQ_NORM_LAYER;
    const float eps = post ? p.eps_post : p.eps_pre;
    float mean, rstd;
    if (!post || p.post_group == 0) {
        stats<V>(u, pieces, layer, 0, eps, p.inv_row, shared, mean, rstd);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < pieces) apply(u[i], p, post, (threadIdx.x + i * threads) * 8, mean, rstd);
    } else {                                 // post_group / 8 neighbouring threads hold a group
#pragma unroll
        for (int i = 0; i < V; ++i) {
            stats<1>(&u[i], i < pieces, layer, p.post_group / 8, eps, p.inv_group, nullptr, mean, rstd);
            if (i < pieces) apply(u[i], p, post, (threadIdx.x + i * threads) * 8, mean, rstd);
        }
    }
}

// Relative error below 2^-20: the hardware's 2^x and 1/x are good to 2^-22 and
// 2^-23, and x log2(e) is rounded once.
__device__ __forceinline__ uint64_t sigmoid2(uint64_t x) {
    float2 t = unpack2(mul2(x, both(-1.4426950408889634f)));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t.y));
    t = unpack2(add2(pack2(t.x, t.y), both(1.f)));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(t.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(t.y));
    return pack2(t.x, t.y);
}

// u = (u + add) * act(gate), h' = h + alpha u of the piece at channel c; take() gives
// the next of the tensors that are there.
template <typename Take>
__device__ __forceinline__ void combine(Piece& u, const NormArgs& p, int c, Take&& take) {
    if (p.add != nullptr) plus(u, take(p.add, p.ld_add));
    if (p.gate != nullptr) {
        const Piece g = take(p.gate, p.ld_gate);
        if (p.gate_act != RQ_GATE_SIGMOID) times(u, g);
        if (p.gate_act != RQ_GATE_IDENTITY) {
#pragma unroll
            for (int j = 0; j < 4; ++j) u.v[j] = mul2(u.v[j], sigmoid2(g.v[j]));
        }
    }
    if (p.alpha != nullptr) times(u, load<float>(p.alpha, c));
    if (p.h != nullptr) plus(u, take(p.h, p.D));
}

__device__ __forceinline__ void cp16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}

// Rows of up to 4096 channels: row blockIdx.x, + gridDim.x, ...; one piece per thread.
constexpr int RING = 3;                      // rows on their way, the current one among them
template <typename T>
__global__ void __launch_bounds__(512, 2) norm_rows_kernel(const NormArgs p) {
    constexpr int PB = 8 * sizeof(T);        // bytes of a piece
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ Moments shared[2][2][MAX_WARPS];      // of alternate rows: one norm alone has one barrier a row
    const int threads = blockDim.x, tid = threadIdx.x, c = tid * 8;
    const bool in = c < p.D;
    const int tensors = 1 + (p.add != nullptr) + (p.gate != nullptr) + (p.h != nullptr);
    const int tensor_bytes = threads * PB, row_bytes = tensors * tensor_bytes;
    unsigned char* mine = ring + tid * PB;
    // where this thread's pieces of the next row to be fetched lie
    const auto start = [&](const void* base, int64_t ld) {
        return static_cast<const char*>(base) + (blockIdx.x * ld + c) * static_cast<int64_t>(sizeof(T));
    };
    const char *py = start(p.y, p.ld_y), *pa = start(p.add, p.ld_add), *pg = start(p.gate, p.ld_gate),
               *ph = start(p.h, p.D);
    const int64_t step = gridDim.x * static_cast<int64_t>(sizeof(T));
    const auto fetch = [&](int64_t row, int slot) {
        if (row < p.M && in) {
            unsigned char* to = mine + slot * row_bytes;
            const auto one = [&](const char*& from, int64_t ld) {
#pragma unroll
                for (int i = 0; i < PB; i += 16) cp16(to + i, from + i);
                to += tensor_bytes;
                from += ld * step;
            };
            one(py, p.ld_y);
            if (p.add != nullptr) one(pa, p.ld_add);
            if (p.gate != nullptr) one(pg, p.ld_gate);
            if (p.h != nullptr) one(ph, p.D);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) fetch(blockIdx.x + static_cast<int64_t>(i) * gridDim.x, i);
    int slot = 0, parity = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        fetch(row + static_cast<int64_t>(RING - 1) * gridDim.x, slot == 0 ? RING - 1 : slot - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
        Piece u[1] = {};
        const unsigned char* from = mine + slot * row_bytes;
        const auto take = [&](const void*, int64_t) {
            const uint4* q = reinterpret_cast<const uint4*>(from);
            from += tensor_bytes;
            return expand<T>(q[0], sizeof(T) == 4 ? q[1] : make_uint4(0u, 0u, 0u, 0u));
        };
        if (in) u[0] = take(nullptr, 0);
        normed<1>(u, in, p, true, threads, shared[parity][0]);
        if (in) {
            combine(u[0], p, c, take);
            if (p.h_out != nullptr) store<T>(p.h_out, row * p.D + c, u[0]);
        }
        if (p.x != nullptr) {
            normed<1>(u, in, p, false, threads, shared[parity][1]);
            if (in) store<__half>(p.x, row * p.D + c, u[0]);
        }
        slot = slot == RING - 1 ? 0 : slot + 1;
        parity ^= 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Longer rows: a CTA each, V pieces per thread.
template <typename T, int V>
__global__ void __launch_bounds__(1024) norm_row_kernel(const NormArgs p) {
    __shared__ Moments shared[2][MAX_WARPS];
    const int64_t row = blockIdx.x;
    const int threads = blockDim.x, all = p.D / 8;
    int pieces = 0;                          // threadIdx.x + i * threads < D / 8
#pragma unroll
    for (int i = 0; i < V; ++i) pieces += static_cast<int>(threadIdx.x) + i * threads < all;
    Piece u[V] = {};
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < pieces) u[i] = load<T>(p.y, row * p.ld_y + (threadIdx.x + i * threads) * 8);
    normed<V>(u, pieces, p, true, threads, shared[0]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i >= pieces) break;
        const int c = (threadIdx.x + i * threads) * 8;
        combine(u[i], p, c, [&](const void* base, int64_t ld) { return load<T>(base, row * ld + c); });
        if (p.h_out != nullptr) store<T>(p.h_out, row * p.D + c, u[i]);
    }
    if (p.x == nullptr) return;
    normed<V>(u, pieces, p, false, threads, shared[1]);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < pieces) store<__half>(p.x, row * p.D + (threadIdx.x + i * threads) * 8, u[i]);
}

template <typename T>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
    const int pieces = a.D / 8;
    if (pieces <= 512) {
        const int threads = (pieces + 31) / 32 * 32;
        const int tensors = 1 + (a.add != nullptr) + (a.gate != nullptr) + (a.h != nullptr);
        const int smem = RING * tensors * threads * 8 * static_cast<int>(sizeof(T));   // at most 192 KB
        const cudaError_t e = allow_smem<norm_rows_kernel<T>>(RING * 4 * 512 * 8 * static_cast<int>(sizeof(T)));
        if (e != cudaSuccess) return e;
        // CTAs that an SM holds: 1024 threads at 64 registers, and their rings
        const int per_sm = std::max(1, std::min(1024 / threads, (220 << 10) / (smem + 2048)));
        const int64_t grid = std::min<int64_t>(a.M, static_cast<int64_t>(num_sms()) * per_sm);
        norm_rows_kernel<T><<<static_cast<unsigned>(grid), threads, smem, s>>>(a);
        return cudaGetLastError();
    }
    norm_row_kernel<T, 2><<<static_cast<unsigned>(a.M), ((pieces + 1) / 2 + 31) / 32 * 32, 0, s>>>(a);
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
    a.inv_row = 1.f / static_cast<float>(D);
    a.inv_group = post_group > 0 ? 1.f / static_cast<float>(post_group) : 0.f;
    const cudaError_t e =
        launch_norm_residual(a, dtype == RQ_OUT_F16, reinterpret_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) return RQ_OK;
    record_cuda_error(e);
    return RQ_ERR_CUDA;
}
