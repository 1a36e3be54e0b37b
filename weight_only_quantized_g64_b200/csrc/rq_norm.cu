// rq_norm.cu -- the step between two projections: norm of a block's output,
// gate, residual with its scale, and the norm that the next projection reads.
//
//   u = (Norm_post(y) + add) * act(gate);   h' = h + alpha u;   x = Norm_pre(h')
//
// A thread holds pieces of 8 channels in registers, so each tensor is read once
// and each result written once.  Rows of up to 4096 channels are taken by CTAs that
// stay, one row or two at a time, a piece of each per thread, and that bring the
// next rows' pieces into shared memory meanwhile (a thread waits for its own
// pieces only); longer rows, whose ring would not fit, are loaded as they come, a
// CTA each.  4096 rows of 4096 fp16 channels with both norms, gate and residual:
// 36.7 us, 4.6 TB/s.  The bytes would take 26; no unit is at its limit (58 % of the
// issue slots), the CTA waits twice a pair of rows at its norms' barriers (one row at
// a time, twice as often: 42.7 us).
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

// The same of parts of n values each: n doubles, and nothing is divided.
__device__ __forceinline__ Moments join_equal(Moments a, int mask) {
    const float d = __shfl_xor_sync(0xffffffffu, a.mean, mask) - a.mean;
    return {a.n + a.n, fmaf(d, 0.5f, a.mean), fmaf(d * d, 0.5f * a.n, a.m2 + __shfl_xor_sync(0xffffffffu, a.m2, mask))};
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

constexpr int MAX_WARPS = 16;

// For R rows of which a thread holds V pieces each (the first `pieces` real, the
// others zeros): the mean (0 for the rms norm) and 1 / sqrt(mean square + eps) of
// the 1 / inv_n values of a row that `width` consecutive lanes (a power of two)
// or, width 0, the whole CTA hold.
template <int R, int V, bool LAYER>
__device__ __forceinline__ void stats(const Piece (&v)[R][V], int pieces, int width, float eps, float inv_n,
                                      Moments (*shared)[MAX_WARPS], float (&mean)[R], float (&rstd)[R]) {
    Moments a[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        a[r] = {8.f * pieces, 0.f, 0.f};
        if (LAYER) {
            uint64_t s = add2(add2(v[r][0].v[0], v[r][0].v[1]), add2(v[r][0].v[2], v[r][0].v[3]));
#pragma unroll
            for (int i = 1; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s = add2(s, v[r][i].v[j]);
            a[r].mean = V == 1 ? sum(s) * 0.125f : pieces > 0 ? __fdividef(sum(s), a[r].n) : 0.f;
        }
        const uint64_t away = both(-a[r].mean);
        uint64_t s = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (V == 1 || i < pieces) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t d = LAYER ? add2(v[r][i].v[j], away) : v[r][i].v[j];
                    s = fma2(d, d, s);
                }
            }
        a[r].m2 = sum(s);
    }
    // lanes that hold equally many values: those of a group, and of a full warp with V = 1 (2049 x 2048, heads of 64:
    // 8.0 us without that case, 7.2 with it)
    const auto join_lanes = [&](int m, bool equal) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (LAYER) a[r] = equal ? join_equal(a[r], m) : join_xor(a[r], m);
            else a[r].m2 += __shfl_xor_sync(0xffffffffu, a[r].m2, m);
        }
    };
    if (width) {
        for (int m = 1; m < width; m <<= 1) join_lanes(m, true);
    } else {
        const bool equal = V == 1 && __all_sync(0xffffffffu, pieces);
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) join_lanes(m, equal);
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (LAYER) shared[r][warp] = a[r];
                else shared[r][warp].m2 = a[r].m2;
            }
        }
        __syncthreads();
        // 16 lanes join the warps' parts, whatever their number (at most 16)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int w = lane & 15;
            if (LAYER) a[r] = w < warps ? shared[r][w] : Moments{0.f, 0.f, 0.f};
            else a[r].m2 = w < warps ? shared[r][w].m2 : 0.f;
        }
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) join_lanes(m, false);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        mean[r] = a[r].mean;
        rstd[r] = rsqrtf(fmaf(a[r].m2, inv_n, eps));
    }
}

// v = (v - mean) * rstd * weight + bias
template <int R, int V, bool LAYER>
__device__ __forceinline__ void normed_as(Piece (&u)[R][V], int pieces, int group, float eps, float inv_n,
                                          const float* weight, const float* bias, Moments (*shared)[MAX_WARPS]) {
    float mean[R], rstd[R];
    const int threads = blockDim.x;
    const auto apply = [&](Piece& v, float m, float s) {
        if (LAYER) {
            const uint64_t away = both(-m);
#pragma unroll
            for (int j = 0; j < 4; ++j) v.v[j] = add2(v.v[j], away);
        }
        const uint64_t r = both(s);
#pragma unroll
        for (int j = 0; j < 4; ++j) v.v[j] = mul2(v.v[j], r);
    };
    if (group == 0) stats<R, V, LAYER>(u, pieces, 0, eps, inv_n, shared, mean, rstd);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (group != 0) {                    // group / 8 neighbouring threads hold a group
            Piece one[R][1];
#pragma unroll
            for (int r = 0; r < R; ++r) one[r][0] = u[r][i];
            stats<R, 1, LAYER>(one, i < pieces, group / 8, eps, inv_n, nullptr, mean, rstd);
        }
        if (i >= pieces) continue;
        const int c = (threadIdx.x + i * threads) * 8;
#pragma unroll
        for (int r = 0; r < R; ++r) apply(u[r][i], mean[r], rstd[r]);
        if (weight != nullptr) {
            const Piece w = load<float>(weight, c);
#pragma unroll
            for (int r = 0; r < R; ++r) times(u[r][i], w);
        }
        if (bias != nullptr) {
            const Piece b = load<float>(bias, c);
#pragma unroll
            for (int r = 0; r < R; ++r) plus(u[r][i], b);
        }
    }
}

template <int R, int V>
__device__ __forceinline__ void normed(Piece (&u)[R][V], int pieces, const NormArgs& p, bool post,
                                       Moments (*shared)[MAX_WARPS]) {
    const int kind = post ? p.post : p.pre;
    if (kind == RQ_NORM_NONE) return;
    const int group = post ? p.post_group : 0;
    const float eps = post ? p.eps_post : p.eps_pre, inv_n = group ? p.inv_group : p.inv_row;
    const float* w = post ? p.post_weight : p.pre_weight;
    const float* b = post ? p.post_bias : p.pre_bias;
    if (kind == RQ_NORM_LAYER) normed_as<R, V, true>(u, pieces, group, eps, inv_n, w, b, shared);
    else normed_as<R, V, false>(u, pieces, group, eps, inv_n, w, b, shared);
}

// Relative error at most (|x| + 6) 2^-24 below 0, and 2^-21 above: the hardware's
// 2^x and 1/x are good to 2^-22 and 2^-23, and x log2(e) is rounded once.  Below
// -87.3, where it would be under 2^-126, it is 0.
__device__ __forceinline__ uint64_t sigmoid2(uint64_t x) {
    float2 t = unpack2(mul2(x, both(-1.4426950408889634f)));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t.y));
    t = unpack2(add2(pack2(t.x, t.y), both(1.f)));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(t.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(t.y));
    return pack2(t.x, t.y);
}

// u = (u + add) * act(gate), h' = h + alpha u of the pieces of R rows at channel c;
// take(r) gives the next of the tensors that are there.
template <int R, typename Take>
__device__ __forceinline__ void combine(Piece* (&u)[R], const NormArgs& p, int c, Take&& take) {
    if (p.add != nullptr) {
#pragma unroll
        for (int r = 0; r < R; ++r) plus(*u[r], take(r, p.add, p.ld_add));
    }
    if (p.gate != nullptr) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            Piece g = take(r, p.gate, p.ld_gate);
            if (p.gate_act != RQ_GATE_IDENTITY) {        // act(gate) first: u * gate alone might not be finite
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t s = sigmoid2(g.v[j]);
                    g.v[j] = p.gate_act == RQ_GATE_SIGMOID ? s : mul2(g.v[j], s);
                }
            }
            times(*u[r], g);
        }
    }
    if (p.alpha != nullptr) {
        const Piece f = load<float>(p.alpha, c);
#pragma unroll
        for (int r = 0; r < R; ++r) times(*u[r], f);
    }
    if (p.h != nullptr) {
#pragma unroll
        for (int r = 0; r < R; ++r) plus(*u[r], take(r, p.h, p.D));
    }
}

__device__ __forceinline__ void cp16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}

// Rows of up to 4096 channels: R rows at a time, one piece of each per thread,
// the next R (with R = 1 the next two) on their way.  Two rows at a time share
// the loads of the weights, the tests of what is there and the barriers.
template <typename T, int R>
__global__ void __launch_bounds__(512, 2) norm_rows_kernel(const NormArgs p) {
    constexpr int PB = 8 * sizeof(T);        // bytes of a piece
    constexpr int RING = R == 1 ? 3 : 2;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ Moments shared[2][2][R][MAX_WARPS];   // of alternate rows: one norm alone has one barrier a row
    const int threads = blockDim.x, tid = threadIdx.x, c = tid * 8;
    const bool in = c < p.D;
    const int tensors = 1 + (p.add != nullptr) + (p.gate != nullptr) + (p.h != nullptr);
    const int piece_step = threads * PB;
    unsigned char* mine = ring + tid * PB;
    const auto fetch = [&](int64_t row, int slot) {          // R rows from this one on
        if (in) {
            unsigned char* to = mine + slot * tensors * R * piece_step;
            const auto one = [&](const void* base, int64_t ld) {
                const char* from = static_cast<const char*>(base) + (row * ld + c) * static_cast<int64_t>(sizeof(T));
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (row + r < p.M) {
#pragma unroll
                        for (int j = 0; j < PB; j += 16) cp16(to + j, from + j);
                    }
                    to += piece_step;
                    from += ld * static_cast<int64_t>(sizeof(T));
                }
            };
            one(p.y, p.ld_y);
            if (p.add != nullptr) one(p.add, p.ld_add);
            if (p.gate != nullptr) one(p.gate, p.ld_gate);
            if (p.h != nullptr) one(p.h, p.D);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int64_t stride = static_cast<int64_t>(gridDim.x) * R;
    int64_t row = static_cast<int64_t>(blockIdx.x) * R;
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) fetch(row + i * stride, i);
    int slot = 0, parity = 0;
    for (; row < p.M; row += stride) {
        fetch(row + (RING - 1) * stride, slot == 0 ? RING - 1 : slot - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
        Piece u[R][1] = {};
        const unsigned char* const from = mine + slot * tensors * R * piece_step;
        const auto take = [&](int place) {
            const uint4* q = reinterpret_cast<const uint4*>(from + place * piece_step);
            return expand<T>(q[0], sizeof(T) == 4 ? q[1] : make_uint4(0u, 0u, 0u, 0u));
        };
        if (in) {
#pragma unroll
            for (int r = 0; r < R; ++r) u[r][0] = take(r);   // (a row behind the last: whatever the slot holds)
        }
        normed<R, 1>(u, in, p, true, shared[parity][0]);
        if (in) {
            int place = R;
            Piece* rows[R];
#pragma unroll
            for (int r = 0; r < R; ++r) rows[r] = &u[r][0];
            combine<R>(rows, p, c, [&](int, const void*, int64_t) { return take(place++); });
            if (p.h_out != nullptr) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (row + r < p.M) store<T>(p.h_out, (row + r) * p.D + c, u[r][0]);
            }
        }
        if (p.x != nullptr) {
            normed<R, 1>(u, in, p, false, shared[parity][1]);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (in && row + r < p.M) store<__half>(p.x, (row + r) * p.D + c, u[r][0]);
        }
        slot = slot == RING - 1 ? 0 : slot + 1;
        parity ^= 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Longer rows: a CTA each, V pieces per thread.
template <typename T, int V>
__global__ void __launch_bounds__(512) norm_row_kernel(const NormArgs p) {
    __shared__ Moments shared[2][1][MAX_WARPS];
    const int64_t row = blockIdx.x;
    const int threads = blockDim.x, all = p.D / 8;
    int pieces = 0;                          // threadIdx.x + i * threads < D / 8
#pragma unroll
    for (int i = 0; i < V; ++i) pieces += static_cast<int>(threadIdx.x) + i * threads < all;
    Piece u[1][V] = {};
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < pieces) u[0][i] = load<T>(p.y, row * p.ld_y + (threadIdx.x + i * threads) * 8);
    normed<1, V>(u, pieces, p, true, shared[0]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i >= pieces) break;
        const int c = (threadIdx.x + i * threads) * 8;
        Piece* rows[1] = {&u[0][i]};
        // (not as read-only data: h may be h_out)
        combine<1>(rows, p, c, [&](int, const void* base, int64_t ld) {
            const uint4* from = reinterpret_cast<const uint4*>(static_cast<const T*>(base) + row * ld + c);
            return expand<T>(from[0], sizeof(T) == 4 ? from[1] : make_uint4(0u, 0u, 0u, 0u));
        });
        if (p.h_out != nullptr) store<T>(p.h_out, row * p.D + c, u[0][i]);
    }
    if (p.x == nullptr) return;
    normed<1, V>(u, pieces, p, false, shared[1]);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < pieces) store<__half>(p.x, row * p.D + (threadIdx.x + i * threads) * 8, u[0][i]);
}

template <typename T, int R>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t s) {
    constexpr int RING = R == 1 ? 3 : 2;
    const int threads = (a.D / 8 + 31) / 32 * 32;
    const int tensors = 1 + (a.add != nullptr) + (a.gate != nullptr) + (a.h != nullptr);
    const int row_bytes = threads * 8 * static_cast<int>(sizeof(T));
    const int smem = RING * R * tensors * row_bytes;
    if (smem > (200 << 10)) return launch_rows<T, 1>(a, s);              // two fp32 rows of four tensors
    const cudaError_t e = allow_smem<norm_rows_kernel<T, R>>(200 << 10);
    if (e != cudaSuccess) return e;
    const int per_sm = std::max(1, std::min(std::min(1024 / threads, 32), (220 << 10) / (smem + (3 << 10))));
    const int64_t grid = std::min<int64_t>((a.M + R - 1) / R, static_cast<int64_t>(num_sms()) * per_sm);
    norm_rows_kernel<T, R><<<static_cast<unsigned>(grid), threads, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
    const int pieces = a.D / 8;
    // One row at a time while an SM has at most 8192 channels of all rows, as two
    // then leave SMs without work (fp16, two norms, gate and residual, us one / two:
    // 148 rows of 4096 3.8 / 4.4, 444 7.8 / 7.0, 4096 42.7 / 34.7; 592 rows of 2048
    // 5.1 / 5.3, 1184 8.4 / 6.6; 2048 rows of 512 4.7 / 4.9, 4096 7.5 / 6.2).
    if (pieces <= 512) return a.M * a.D <= int64_t{8192} * num_sms() ? launch_rows<T, 1>(a, s) : launch_rows<T, 2>(a, s);
    norm_row_kernel<T, 4><<<static_cast<unsigned>(a.M), ((pieces + 3) / 4 + 31) / 32 * 32, 0, s>>>(a);
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
