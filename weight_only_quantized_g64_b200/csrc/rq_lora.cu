// rq_lora.cu -- low-rank adapters of many requests beside one product:
//   out[m] = epi(y[m] + s_a B_a (A_a x[m])),   a = ids[m].
//
// Products with B run on the warp-level tensor cores with each fp32 sum t split
// into two fp16 parts, t = 2^-e (hi + lo), scaled per token so that the largest
// lies near 2^14: 22 bits of it enter the product, whose terms are exact.  All
// operands go into the MMAs as they come from memory, 16 bytes of a row per
// lane: the order of the summed index does not matter as long as both operands
// follow it.
//
// Few tokens (decode): one launch, a cluster of 8 CTAs per token.  Each takes an
// eighth of K for A x (plain fp32 sums), sends its R sums to all eight, and
// after one cluster barrier takes an eighth of the outputs; hi and lo are two of
// the eight columns of an MMA over 16 rows of B, the first of which are on their
// way before the cluster meets.  Bound by latency: two dependent reads of memory
// and a barrier; 32 tokens beside 16384 x 4096, R = 32: 13.0 us, 3.4 TB/s.
//
// Many tokens (prefill): two launches.  A CTA per 16 tokens (and some of their
// adapters) splits K over its warps for A x, 640 KB through its L1 (the bound: 64
// bytes of every row and load), and leaves hi and lo of t in the order of the
// MMA's registers; then every warp of a second launch takes 16 tokens x 64 outputs
// without shared memory or barriers, its y and B on their way before the first
// launch has ended.  Tokens of several adapters in a warp's 16 are taken in turn, and each
// keeps its own sum.  2048 tokens beside 4096 x 4096, R = 64: 32 us.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cfloat>
#include <climits>

#include "rq_lora.h"
#include "rq_once.h"
#include "rq_ptx.cuh"

namespace rq {
namespace {

namespace cg = cooperative_groups;

// The adapter of a token: -1 for none (and, with the status, for one that does not exist).
__device__ __forceinline__ int adapter_of(const LoraArgs& p, int m) {
    const int a = p.ids[m];
    if (a < p.L) return a < 0 ? -1 : a;
    if (p.status != nullptr) atomicMax(p.status, RQ_ERR_RANGE);
    return -1;
}
__device__ __forceinline__ int rank_of(const LoraArgs& p, int a) {
    return p.ranks == nullptr ? p.R : min(max(p.ranks[a], 0), p.R);
}
__device__ __forceinline__ float finish(float v, bool relu_sq) {
    if (!relu_sq) return v;
    const float f = v < 0.f ? 0.f : v;       // keeps NaN
    return f * f;
}
template <typename T>
__device__ __forceinline__ float get(const void* p, int64_t i) {
    if constexpr (sizeof(T) == 4) return static_cast<const float*>(p)[i];
    else return __half2float(static_cast<const __half*>(p)[i]);
}
template <typename T>
__device__ __forceinline__ void put(void* p, int64_t i, float v) {
    if constexpr (sizeof(T) == 4) static_cast<float*>(p)[i] = v;
    else static_cast<__half*>(p)[i] = __float2half_rn(v);
}
__device__ __forceinline__ float dot8(const uint4& a, const float* b, float c) {
    const __half2* h = reinterpret_cast<const __half2*>(&a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        c = fmaf(f.x, b[2 * i], c);
        c = fmaf(f.y, b[2 * i + 1], c);
    }
    return c;
}

// The power of two 2^e that brings a largest magnitude into [2^14, 2^15).
__device__ __forceinline__ int scale_of(float top) {
    const int ex = static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127;
    return top > 0.f ? min(14 - ex, 100) : 0;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
// The first or the second fp16 part of f; an infinite one has no rest.
__device__ __forceinline__ __half split(float f, int part) {
    const __half h = __float2half_rn(f);
    if (part == 0) return h;
    return __float2half_rn(fabsf(f) <= 65504.f ? f - __half2float(h) : 0.f);
}
__device__ __forceinline__ void mma(float c[4], const uint32_t a[4], const uint32_t b[2]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// The order of the ranks in the MMAs with B, R <= 8 PR: register j of a row holds, in lane (g, q), this rank and the
// next: 2 ranks of 8, 4 of 16 in a lane, or 8 (16 bytes) of every 32.
template <int PR>
__device__ __forceinline__ int rank_at(int q, int j) {
    return PR == 1 ? 2 * q + 8 * j : PR == 2 ? 4 * q + 2 * j : 8 * q + 8 * (j & ~3) + 2 * (j & 3);
}
// Those registers of one row of B (from: the row at rank_at(q, 0)), zeros where it is not live or behind the rank.
template <int PR>
__device__ __forceinline__ void row_of_b(const uint16_t* from, bool live, int rank0, int rank, uint32_t* r) {
    if constexpr (PR == 1) r[0] = live && rank0 < rank ? __ldg(reinterpret_cast<const uint32_t*>(from)) : 0u;
    if constexpr (PR == 2) {
        const uint2 v = live && rank0 < rank ? __ldg(reinterpret_cast<const uint2*>(from)) : make_uint2(0u, 0u);
        r[0] = v.x;
        r[1] = v.y;
    }
    if constexpr (PR >= 4) {
#pragma unroll
        for (int j = 0; j < PR; j += 4) {    // 32 ranks further every 4 registers
            const uint4 v = live && rank0 + 8 * j < rank ? __ldg(reinterpret_cast<const uint4*>(from + 8 * j))
                                                         : make_uint4(0u, 0u, 0u, 0u);
            r[j] = v.x;
            r[j + 1] = v.y;
            r[j + 2] = v.z;
            r[j + 3] = v.w;
        }
    }
}
// Ranks behind the adapter's own are not its: what B holds there does not count.
__device__ __forceinline__ uint32_t keep_of(int r, int rank) {
    return r + 1 < rank ? 0xffffffffu : r < rank ? 0xffffu : 0u;
}

// ------------------------------------------------------------- few tokens --
constexpr int CS = 8;                        // CTAs of a token
constexpr int TT = 256;                      // threads

// PR: pieces of 8 ranks (R <= 8 PR); a row of B is read by PR lanes.
template <typename T, int PR>
__global__ void __cluster_dims__(CS, 1, 1) __launch_bounds__(TT) lora_token_kernel(const LoraArgs p) {
    __shared__ float part[CS][PR * 8];
    __shared__ float ts[PR * 8];
    cg::cluster_group cluster = cg::this_cluster();
    const int m = blockIdx.x / CS, me = blockIdx.x % CS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int a = adapter_of(p, m);
    const int64_t n0 = p.N * me / CS, n1 = p.N * (me + 1) / CS;
    const int64_t yrow = static_cast<int64_t>(m) * p.N;
    if (a < 0) {                             // the whole cluster takes this way
        for (int64_t n = n0 + threadIdx.x; n < n1; n += TT)
            put<T>(p.out, yrow + n, finish(get<T>(p.y, yrow + n), p.relu_sq));
        return;
    }
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");

    // A x over this CTA's part of K; warp w takes ranks w, w + 8, ...
    const int rank = rank_of(p, a);
    const int pieces = p.K / 8, p0 = static_cast<int64_t>(pieces) * me / CS,
              p1 = static_cast<int64_t>(pieces) * (me + 1) / CS;
    const uint4* xp = reinterpret_cast<const uint4*>(p.x) + static_cast<int64_t>(m) * pieces;
    const uint4* ap = reinterpret_cast<const uint4*>(p.A) + static_cast<int64_t>(a) * p.R * pieces;
    float acc[PR];
#pragma unroll
    for (int r = 0; r < PR; ++r) acc[r] = 0.f;
#pragma unroll 2
    for (int i = p0 + lane; i < p1; i += 32) {
        uint4 w[PR];
        const uint4 xv = __ldg(xp + i);
#pragma unroll
        for (int r = 0; r < PR; ++r)
            w[r] = warp + 8 * r < rank ? __ldg(ap + static_cast<int64_t>(warp + 8 * r) * pieces + i)
                                       : make_uint4(0u, 0u, 0u, 0u);
        float xf[8];
        const __half2* h = reinterpret_cast<const __half2*>(&xv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(h[j]);
            xf[2 * j] = f.x;
            xf[2 * j + 1] = f.y;
        }
#pragma unroll
        for (int r = 0; r < PR; ++r) acc[r] = dot8(w[r], xf, acc[r]);
    }

    // the first rows of B and y, while the sums are joined.  A warp takes 32 outputs at a time: two MMAs of 16 rows;
    // lane (g, q) supplies rows g and g + 8 of each, and for the ranks that its registers hold the same of t
    constexpr int NR = PR;
    constexpr int AHEAD = PR <= 2 ? 4 : PR == 4 ? 3 : 1;         // (4 for R = 32 leaves an SM one CTA: 28 us for 13.5)
    const int g = lane >> 2, q = lane & 3;
    const int rank0 = rank_at<PR>(q, 0);
    const uint16_t* bp = p.B + static_cast<int64_t>(a) * p.N * p.R + rank0;
    const bool ragged = rank < 8 * PR;
    struct Rows {
        uint32_t r[4][NR];                   // rows g, g + 8, g + 16, g + 24
        float y;                             // of output `lane`
    };
    const auto rows_at = [&](int64_t n, Rows& w) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = n + 8 * i + g;
            row_of_b<PR>(bp + row * p.R, row < n1, rank0, rank, w.r[i]);
        }
        w.y = n + lane < n1 ? get<T>(p.y, yrow + n + lane) : 0.f;
    };
    constexpr int STEP = TT;                 // outputs that the CTA takes at a time
    const int64_t first = n0 + 32 * warp;
    Rows w[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) rows_at(first + i * STEP, w[i]);
#pragma unroll
    for (int r = 0; r < PR; ++r)
#pragma unroll
        for (int o = 16; o; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
    asm volatile("barrier.cluster.wait;" ::: "memory");   // every CTA of the cluster runs
    if (lane < CS) {
        float* there = cluster.map_shared_rank(&part[me][0], lane);
#pragma unroll
        for (int r = 0; r < PR; ++r) there[warp + 8 * r] = warp + 8 * r < rank ? acc[r] : 0.f;
    }
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (threadIdx.x < PR * 8) {
        float t = 0.f;
#pragma unroll
        for (int c = 0; c < CS; ++c) t += part[c][threadIdx.x];
        ts[threadIdx.x] = p.scale == nullptr ? t : t * p.scale[a];
    }
    __syncthreads();
    float top = 0.f;
#pragma unroll 8
    for (int r = 0; r < PR * 8; ++r) {
        const float mag = fabsf(ts[r]);
        top = mag <= FLT_MAX ? fmaxf(top, mag) : top;            // infinities and NaN pass as they are
    }
    const int e = scale_of(top);
    const float up = pow2(e), back = pow2(-e);
    uint32_t tf[NR], keep[NR];               // column 0 of the product: hi, column 1: lo
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        const int r = rank_at<PR>(q, j);
        __half2 v = __floats2half2_rn(0.f, 0.f);
        if (g < 2) v = __halves2half2(split(ts[r] * up, g), split(ts[r + 1] * up, g));
        tf[j] = *reinterpret_cast<const uint32_t*>(&v);
        keep[j] = keep_of(r, rank);
    }
    const auto finish_rows = [&](int64_t n, Rows& w) {
        float v[4];
#pragma unroll
        for (int pair = 0; pair < 2; ++pair) {
            uint32_t(&lo)[NR] = w.r[2 * pair];
            uint32_t(&hi)[NR] = w.r[2 * pair + 1];
            if (ragged) {
#pragma unroll
                for (int j = 0; j < NR; ++j) {
                    lo[j] &= keep[j];
                    hi[j] &= keep[j];
                }
            }
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NR; j += 2) {
                const uint32_t fa[4] = {lo[j], hi[j], NR > 1 ? lo[NR > 1 ? j + 1 : j] : 0u,
                                        NR > 1 ? hi[NR > 1 ? j + 1 : j] : 0u};
                const uint32_t fb[2] = {tf[j], NR > 1 ? tf[NR > 1 ? j + 1 : j] : 0u};
                mma(c, fa, fb);
            }
            v[2 * pair] = c[0] + c[1];       // right in the lanes with q = 0
            v[2 * pair + 1] = c[2] + c[3];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], (lane & 7) * 4);
        const float s = lane < 8 ? v[0] : lane < 16 ? v[1] : lane < 24 ? v[2] : v[3];
        if (n + lane < n1) put<T>(p.out, yrow + n + lane, finish(fmaf(s, back, w.y), p.relu_sq));
    };
    for (int64_t n = first; n < n1; n += AHEAD * STEP) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (n + i * STEP < n1) {
                finish_rows(n + i * STEP, w[i]);
                rows_at(n + (AHEAD + i) * STEP, w[i]);
            }
        }
    }
}

template <typename T, int PR>
cudaError_t launch_tokens(const LoraArgs& a, cudaStream_t s) {
    lora_token_kernel<T, PR><<<a.M * CS, TT, 0, s>>>(a);
    return cudaGetLastError();
}

// ------------------------------------------------------------ many tokens --
constexpr int TM = 16;                       // tokens of a tile
constexpr int SW = 16;                       // warps that split K

// The smallest adapter of 16 tokens above `after` (INT_MAX: none); id: of token lane % 16.
__device__ __forceinline__ int next_adapter(int id, int after) {
    return __reduce_min_sync(0xffffffffu, id > after ? id : INT_MAX);
}

// Four consecutive outputs, `left` of them inside the row; WIDE: 4 | N.
template <typename T, bool WIDE>
__device__ __forceinline__ void get4(const void* p, int64_t at, int64_t left, float f[4]) {
    if constexpr (WIDE) {
        if (left <= 0) return;
        if constexpr (sizeof(T) == 4) {
            const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
            f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __half*>(p) + at);
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
            f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = j < left ? get<T>(p, at + j) : 0.f;
    }
}
template <typename T, bool WIDE>
__device__ __forceinline__ void put4(void* p, int64_t at, int64_t left, const float f[4]) {
    if constexpr (WIDE) {
        if (left <= 0) return;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(f[0], f[1], f[2], f[3]);
        } else {
            const __half2 a = __floats2half2_rn(f[0], f[1]), b = __floats2half2_rn(f[2], f[3]);
            *reinterpret_cast<uint2*>(static_cast<__half*>(p) + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left) put<T>(p, at + j, f[j]);
    }
}

// The workspace: per tile of 16 tokens and MMA step the four registers of every lane, hi then lo; then 2^-e of
// every token.
template <int PR>
constexpr int mma_steps() { return PR < 4 ? 1 : PR / 2; }

// PR: pieces of 8 ranks (R <= 8 PR)
template <int PR>
__global__ void __launch_bounds__(SW * 32) lora_sums_kernel(const LoraArgs p) {
    constexpr int LDP = PR * 8 + 1;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    float (*part)[TM][LDP] = reinterpret_cast<float (*)[TM][LDP]>(smem_raw);      // [SW]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the second launch's y and B
    const int m0 = blockIdx.x * TM;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int row = lane & 15;
    const int id = m0 + row < p.M ? adapter_of(p, m0 + row) : -1;
    const int id_of[2] = {__shfl_sync(0xffffffffu, id, g), __shfl_sync(0xffffffffu, id, g + 8)};

    // this warp's part of K, in steps of 32: lane (g, q) holds k 8 q + 0..7 of rows g (and g + 8)
    const int steps = (p.K + 31) / 32;
    const int s0 = static_cast<int64_t>(steps) * warp / SW, s1 = static_cast<int64_t>(steps) * (warp + 1) / SW;
    const int64_t xrow[2] = {static_cast<int64_t>(min(m0 + g, p.M - 1)) * p.K, static_cast<int64_t>(min(m0 + g + 8, p.M - 1)) * p.K};
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    int slot = blockIdx.y;                   // adapters until the next that is this CTA's
    bool mine = false;                       // token `row` has one of them
    for (int a = next_adapter(id, -1); a != INT_MAX; a = next_adapter(id, a)) {
        if (slot-- != 0) continue;
        slot = gridDim.y - 1;
        mine = mine || id == a;
        const uint16_t* A = p.A + (static_cast<int64_t>(a) * p.R + g) * p.K;
        float acc[PR][4];
#pragma unroll
        for (int n = 0; n < PR; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[n][j] = 0.f;
        struct Step {
            uint4 x[2], w[PR];
        };
        // every address lies inside (k and the ranks are cut off), so all loads of a step are in flight at once
        const auto read = [&](int step, Step& f) {
            const int k = min(step * 32 + 8 * q, p.K - 8);
#pragma unroll
            for (int i = 0; i < 2; ++i) f.x[i] = __ldg(reinterpret_cast<const uint4*>(p.x + xrow[i] + k));
#pragma unroll
            for (int n = 0; n < PR; ++n)
                f.w[n] = __ldg(reinterpret_cast<const uint4*>(A + static_cast<int64_t>(8 * n < p.R ? 8 * n : 0) * p.K + k));
        };
        const auto take = [&](int step, Step& f) {
            if (step * 32 + 8 * q >= p.K) {  // behind the end: neither operand counts
                f.x[0] = f.x[1] = none;
#pragma unroll
                for (int n = 0; n < PR; ++n) f.w[n] = none;
            }
            const uint32_t f0[4] = {f.x[0].x, f.x[1].x, f.x[0].y, f.x[1].y}, f1[4] = {f.x[0].z, f.x[1].z, f.x[0].w, f.x[1].w};
#pragma unroll
            for (int n = 0; n < PR; ++n) {
                const uint32_t b0[2] = {f.w[n].x, f.w[n].y}, b1[2] = {f.w[n].z, f.w[n].w};
                mma(acc[n], f0, b0);
                mma(acc[n], f1, b1);
            }
        };
        // steps in flight of a warp; with 16 warps one is enough when it is 160 bytes a lane (8192 tokens, R = 32: four 61
        // us, two 56; 2048 tokens, R = 64: two 32.9, one 32.0)
        constexpr int DEEP = PR <= 2 ? 4 : PR == 4 ? 2 : 1;
        Step ring[DEEP];
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
            if (s0 + i < s1) read(s0 + i, ring[i]);
        for (int step = s0; step < s1; step += DEEP) {
#pragma unroll
            for (int i = 0; i < DEEP; ++i) {
                if (step + i >= s1) break;
                take(step + i, ring[i]);
                if (step + i + DEEP < s1) read(step + i + DEEP, ring[i]);
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (id_of[half] != a) continue;
#pragma unroll
            for (int n = 0; n < PR; ++n) {
                part[warp][g + 8 * half][8 * n + 2 * q] = acc[n][2 * half];
                part[warp][g + 8 * half][8 * n + 2 * q + 1] = acc[n][2 * half + 1];
            }
        }
    }
    const uint32_t tokens = __ballot_sync(0xffffffffu, mine);    // (the same in every warp)
    if (tokens == 0) return;
    __syncthreads();
    // one warp per token: t in part[0], its scale
    if (tokens >> warp & 1) {
        const int a = __shfl_sync(0xffffffffu, id, warp);
        const int rank = rank_of(p, a);
        const float s = p.scale != nullptr ? p.scale[a] : 1.f;
        float top = 0.f;
        for (int r = lane; r < PR * 8; r += 32) {
            float t = 0.f;
            if (r < rank) {
#pragma unroll
                for (int w = 0; w < SW; ++w) t += part[w][warp][r];
                t *= s;
            }
            part[0][warp][r] = t;
            const float mag = fabsf(t);
            top = mag <= FLT_MAX ? fmaxf(top, mag) : top;        // infinities and NaN pass as they are
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int e = scale_of(top);
        __syncwarp();
        for (int r = lane; r < PR * 8; r += 32) part[0][warp][r] *= pow2(e);
        if (lane == 0)
            reinterpret_cast<float*>(p.work + static_cast<int64_t>(gridDim.x) * mma_steps<PR>() * 64)[m0 + warp] = pow2(-e);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < mma_steps<PR>() * 64; i += SW * 32) {
        const int l = i & 31, lo = (i >> 5) & 1, step = i >> 6, gg = l >> 2, qq = l & 3;
        uint4* const to = p.work + (static_cast<int64_t>(blockIdx.x) * mma_steps<PR>() + step) * 64 + lo * 32 + l;
        uint32_t f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {        // registers: rows gg, gg + 8 of the first two ranks, then of the next
            const int r = rank_at<PR>(qq, 2 * step + (j >> 1)), t = gg + 8 * (j & 1);
            const __half2 v = r < PR * 8 ? __halves2half2(split(part[0][t][r], lo), split(part[0][t][r + 1], lo))
                                         : __floats2half2_rn(0.f, 0.f);
            f[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
        const bool low = tokens >> gg & 1, high = tokens >> (gg + 8) & 1;
        if (low && high) {
            *to = make_uint4(f[0], f[1], f[2], f[3]);
        } else if (low) {                    // (the other token is another CTA's, or has no adapter)
            to->x = f[0];
            to->z = f[2];
        } else if (high) {
            to->y = f[1];
            to->w = f[3];
        }
    }
}

// out = epi(y + t B^T): a warp takes 16 tokens x 64 outputs.  A lane's columns in a pair of 8-column products are four
// neighbours: column c of product i stands for output 16 (i / 2) + 4 (c / 2) + 2 (i % 2) + c % 2.
constexpr int EW = 8;                        // warps of a CTA: 4 tiles of tokens x 2 of outputs, which share B and t in L1
template <typename T, int PR, bool WIDE>
__global__ void __launch_bounds__(EW * 32, 2) lora_outputs_kernel(const LoraArgs p) {
    constexpr int NR = PR, STEPS = mma_steps<PR>();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int tiles = (p.M + TM - 1) / TM, tile = blockIdx.y * 4 + (warp & 3), m0 = tile * TM;
    if (tile >= tiles) return;
    const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * 2 + (warp >> 2)) * 64;
    if (n0 >= p.N) return;
    const int id = m0 + (lane & 15) < p.M ? adapter_of(p, m0 + (lane & 15)) : -1;
    const int id_of[2] = {__shfl_sync(0xffffffffu, id, g), __shfl_sync(0xffffffffu, id, g + 8)};
    const int64_t rows[2] = {m0 + g, m0 + g + 8};
    float acc[4][2][4];                      // [16 outputs][row half][neighbour]: y, then the sum
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int64_t n = n0 + 16 * i + 4 * q;
            if (rows[half] < p.M) get4<T, WIDE>(p.y, rows[half] * p.N + n, p.N - n, acc[i][half]);
        }
    bool waited = false;
    for (int a = next_adapter(id, -1); a != INT_MAX; a = next_adapter(id, a)) {
        const int rank = rank_of(p, a), rank0 = rank_at<PR>(q, 0);
        const uint16_t* B = p.B + (static_cast<int64_t>(a) * p.N + n0) * p.R + rank0;
        const bool ragged = rank < 8 * PR;
        constexpr bool HOLD = PR <= 8;       // t stays in registers; else it is read for every 16 outputs
        uint4 held[HOLD ? STEPS : 1][2];
        const uint4* work = p.work + static_cast<int64_t>(tile) * STEPS * 64 + lane;
        constexpr int AHEAD = PR <= 8 ? 1 : 0;   // the rows of the next 16 outputs are on their way (if registers hold them)
        uint32_t b[1 + AHEAD][2][NR];
        const auto fetch = [&](int i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = 16 * i + 4 * (g >> 1) + 2 * h + (g & 1);
                row_of_b<PR>(B + static_cast<int64_t>(n) * p.R, n0 + n < p.N, rank0, rank, b[i & AHEAD][h]);
            }
        };
        if (AHEAD) fetch(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {        // 16 outputs
            if (i + AHEAD < 4) fetch(i + AHEAD);
            if (!waited) {                   // y and the first rows of B are on their way; t comes from the launch before
                asm volatile("griddepcontrol.wait;" ::: "memory");
                waited = true;
            }
            if (HOLD && i == 0) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    held[HOLD ? s : 0][0] = work[s * 64];
                    held[HOLD ? s : 0][1] = work[s * 64 + 32];
                }
            }
            if (ragged) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < NR; ++j) b[i & AHEAD][h][j] &= keep_of(rank_at<PR>(q, j), rank);
            }
            float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const uint4 hi = HOLD ? held[HOLD ? s : 0][0] : work[s * 64], lo = HOLD ? held[HOLD ? s : 0][1] : work[s * 64 + 32];
                const uint32_t fh[4] = {hi.x, hi.y, hi.z, hi.w}, fl[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t fb[2] = {b[i & AHEAD][h][2 * s < NR ? 2 * s : 0], NR > 1 ? b[i & AHEAD][h][2 * s + 1 < NR ? 2 * s + 1 : 0] : 0u};
                    mma(c[h], fl, fb);
                    mma(c[h], fh, fb);
                }
            }
            const float* back = reinterpret_cast<const float*>(p.work + static_cast<int64_t>(tiles) * STEPS * 64);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (id_of[half] != a) continue;
                const float f = back[rows[half]];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float& o = acc[i][half][2 * h + j];
                        o = fmaf(c[h][2 * half + j], f, o);
                    }
            }
        }
    }
    // no CTA ends before the first launch has (its workspace is then free for the next call)
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int64_t n = n0 + 16 * i + 4 * q;
            if (rows[half] >= p.M) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][half][j] = finish(acc[i][half][j], p.relu_sq);
            put4<T, WIDE>(p.out, rows[half] * p.N + n, p.N - n, acc[i][half]);
        }
}

template <typename T, int PR>
cudaError_t launch_tiles(const LoraArgs& a, cudaStream_t s) {
    constexpr int smem = SW * TM * (PR * 8 + 1) * 4;
    cudaError_t e = allow_smem<lora_sums_kernel<PR>>(smem);
    if (e != cudaSuccess) return e;
    const int tiles = (a.M + TM - 1) / TM;
    // A tile's adapters are dealt over up to 16 CTAs, as far as two CTAs an SM go: where one request ends and the next
    // begins the two are then not summed one after the other (2048 tokens of 6 requests, R = 64: 32.0 us, by one CTA
    // 37.9; 40 tokens of as many requests, R = 16, 4096 x 4096: 16.0, by one 45).  Without a use for them the others cost
    // their start (8192 tokens of one request beside 2048 x 2048: four CTAs a tile 8 us more).
    const int share = std::max(1, std::min(std::min(a.L, TM), 2 * num_sms() / tiles));
    lora_sums_kernel<PR><<<dim3(tiles, share), SW * 32, smem, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.N + 127) / 128), (tiles + 3) / 4);
    cfg.blockDim = dim3(EW * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.N % 4 == 0 ? cudaLaunchKernelEx(&cfg, lora_outputs_kernel<T, PR, true>, a)
                        : cudaLaunchKernelEx(&cfg, lora_outputs_kernel<T, PR, false>, a);
}

template <typename T>
cudaError_t tokens(const LoraArgs& a, cudaStream_t s) {
    return a.R <= 8    ? launch_tokens<T, 1>(a, s)
           : a.R <= 16 ? launch_tokens<T, 2>(a, s)
           : a.R <= 32 ? launch_tokens<T, 4>(a, s)
           : a.R <= 64 ? launch_tokens<T, 8>(a, s)
                       : launch_tokens<T, 16>(a, s);
}
template <typename T>
cudaError_t tiles(const LoraArgs& a, cudaStream_t s) {
    return a.R <= 8    ? launch_tiles<T, 1>(a, s)
           : a.R <= 16 ? launch_tiles<T, 2>(a, s)
           : a.R <= 32 ? launch_tiles<T, 4>(a, s)
           : a.R <= 64 ? launch_tiles<T, 8>(a, s)
                       : launch_tiles<T, 16>(a, s);
}

bool mis(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

rq_status check_sizes(int64_t M, int64_t K, int64_t N, int64_t L, int64_t R) {
    if (M < 1 || M > 64 * 65535 || K < 8 || K % 8 != 0 || K > (1 << 30)) return RQ_ERR_SHAPE;
    if (N < 1 || N > (int64_t{1} << 31) - 1 || L < 1 || L > (1 << 30)) return RQ_ERR_SHAPE;
    if (R < 8 || R % 8 != 0 || R > RQ_MAX_LORA_RANK) return RQ_ERR_SHAPE;
    return RQ_OK;
}

}  // namespace

cudaError_t launch_lora_tokens(const LoraArgs& a, bool half, cudaStream_t s) {
    return half ? tokens<__half>(a, s) : tokens<float>(a, s);
}
cudaError_t launch_lora_tiles(const LoraArgs& a, bool half, cudaStream_t s) {
    return half ? tiles<__half>(a, s) : tiles<float>(a, s);
}

}  // namespace rq

using namespace rq;

extern "C" {

size_t rq_lora_work_bytes(int64_t M, int64_t R) {
    if (check_sizes(M, 8, 1, 1, R) != RQ_OK || M <= kLoraTokens) return 0;
    const int64_t tiles = (M + TM - 1) / TM, steps = R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8;
    return static_cast<size_t>(tiles * (steps * 64 * sizeof(uint4) + TM * sizeof(float)));
}

rq_status rq_lora_add(const uint16_t* x, int64_t M, int64_t K, const uint16_t* A, const uint16_t* B, int64_t L,
                      int64_t R, const int32_t* ids, const int32_t* ranks, const float* scale, const void* y,
                      void* out, int64_t N, int dtype, int epilogue, void* work, int* dev_status,
                      rq_stream_t stream) {
    if (dtype != RQ_OUT_F32 && dtype != RQ_OUT_F16) return RQ_ERR_RANGE;
    if (epilogue != RQ_EPI_NONE && epilogue != RQ_EPI_RELU_SQ) return RQ_ERR_RANGE;
    const rq_status st = check_sizes(M, K, N, L, R);
    if (st != RQ_OK) return st;
    if (x == nullptr || A == nullptr || B == nullptr || ids == nullptr || y == nullptr || out == nullptr)
        return RQ_ERR_NULL;
    if (work == nullptr && M > kLoraTokens) return RQ_ERR_NULL;
    if (mis(x, 16) || mis(A, 16) || mis(B, 16) || mis(y, 16) || mis(out, 16) || mis(work, 16) || mis(ids, 4) ||
        mis(ranks, 4) || mis(scale, 4) || mis(dev_status, 4))
        return RQ_ERR_ALIGN;
    LoraArgs a = {};
    a.x = x;
    a.A = A;
    a.B = B;
    a.ids = ids;
    a.ranks = ranks;
    a.scale = scale;
    a.y = y;
    a.out = out;
    a.work = static_cast<uint4*>(work);
    a.status = dev_status;
    a.N = N;
    a.M = static_cast<int>(M);
    a.K = static_cast<int>(K);
    a.R = static_cast<int>(R);
    a.L = static_cast<int>(L);
    a.relu_sq = epilogue == RQ_EPI_RELU_SQ;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool half = dtype == RQ_OUT_F16;
    const cudaError_t e = M <= kLoraTokens ? launch_lora_tokens(a, half, s) : launch_lora_tiles(a, half, s);
    if (e == cudaSuccess) return RQ_OK;
    record_cuda_error(e);
    return RQ_ERR_CUDA;
}

}  // extern "C"
