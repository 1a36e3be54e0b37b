// rq_lora.cu -- low-rank adapters of many requests beside one product:
//   out[m] = epi(y[m] + s_a B_a (A_a x[m])),   a = ids[m].
//
// Few tokens (decode): a cluster of 8 CTAs per token, one launch.  Each CTA
// forms A x over an eighth of K, sends its R sums to all eight, and after one
// cluster barrier adds them in rank order and takes an eighth of the outputs;
// its first rows of B are already on their way then.  Bound by latency: two
// dependent reads of memory and a barrier.
//
// Many tokens (prefill): tiles of 64 tokens on the warp-level tensor cores,
// two launches (A x split over K into the workspace, then B).  The products of
// the first are exact in fp32; the second splits each fp32 sum t into two fp16
// parts, t = 2^-e (hi + lo) with |t| 2^e scaled near 2^14 per token, so 22 bits
// of t enter the product.  Bound by the bytes of x, y and out.  A tile whose
// tokens use several adapters takes them in turn and keeps each token's own.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cfloat>
#include <climits>

#include "rq_lora.h"
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

// ------------------------------------------------------------- few tokens --
constexpr int CS = 8;                        // CTAs of a token
constexpr int TT = 256;                      // threads

// PR: pieces of 8 ranks (R <= 8 PR); a row of B is read by PR lanes.
template <typename T, int PR>
__global__ void __launch_bounds__(TT) lora_token_kernel(const LoraArgs p) {
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

    // the first rows of B and y, while the sums are joined
    constexpr int ROWS = TT / PR, AHEAD = 4;
    const int piece = threadIdx.x % PR;
    const uint4* bp = reinterpret_cast<const uint4*>(p.B) + static_cast<int64_t>(a) * p.N * (p.R / 8) + piece;
    const int64_t first = n0 + threadIdx.x / PR;
    const auto row_of_b = [&](int64_t n) {
        return n < n1 && piece * 8 < rank ? __ldg(bp + n * (p.R / 8)) : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 bv[AHEAD];
    float yv[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
        bv[i] = row_of_b(first + i * ROWS);
        yv[i] = piece == 0 && first + i * ROWS < n1 ? get<T>(p.y, yrow + first + i * ROWS) : 0.f;
    }
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
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = ts[piece * 8 + j];
    // ranks behind the adapter's own are not its: neither their sums nor their columns of B count
    const int tail = rank - piece * 8;
    const auto row_sum = [&](uint4 b) {
        if (tail > 0 && tail < 8) {
            __half* h = reinterpret_cast<__half*>(&b);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j >= tail) h[j] = __float2half_rn(0.f);
        }
        float s = tail > 0 ? dot8(b, t, 0.f) : 0.f;
#pragma unroll
        for (int o = 1; o < PR; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
        const float s = row_sum(bv[i]);
        const int64_t n = first + i * ROWS;
        if (piece == 0 && n < n1) put<T>(p.out, yrow + n, finish(yv[i] + s, p.relu_sq));
    }
    for (int64_t base = n0 + AHEAD * ROWS; base < n1; base += AHEAD * ROWS) {
        const int64_t at = base + threadIdx.x / PR;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            bv[i] = row_of_b(at + i * ROWS);
            yv[i] = piece == 0 && at + i * ROWS < n1 ? get<T>(p.y, yrow + at + i * ROWS) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const float s = row_sum(bv[i]);
            const int64_t n = at + i * ROWS;
            if (piece == 0 && n < n1) put<T>(p.out, yrow + n, finish(yv[i] + s, p.relu_sq));
        }
    }
}

template <typename T, int PR>
cudaError_t launch_tokens(const LoraArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.M * CS);
    cfg.blockDim = dim3(TT);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_token_kernel<T, PR>, a);
}

// ------------------------------------------------------------ many tokens --
constexpr int TM = 64;                       // tokens of a tile
constexpr int KT = 64;                       // k of a stage
constexpr int NT = 128;                      // outputs of a tile
constexpr int LDK = KT + 8;                  // halves; 16-byte pieces of 8 rows meet no bank twice

__device__ __forceinline__ void cp16(void* dst, const void* src, bool live) {
    const int n = live ? 16 : 0;             // 0: the destination is filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t r[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}
__device__ __forceinline__ void ldsm2(uint32_t r[2], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(smem_u32(p)));
}
__device__ __forceinline__ void mma(float c[4], const uint32_t a[4], const uint32_t b[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// The smallest adapter of the tile above `after` (INT_MAX: none); all threads.
__device__ __forceinline__ int next_adapter(const int* ids, int after) {
    const int lane = threadIdx.x & 31;
    int best = INT_MAX;
#pragma unroll
    for (int i = lane; i < TM; i += 32) best = ids[i] > after ? min(best, ids[i]) : best;
    return __reduce_min_sync(0xffffffffu, best);
}

// t[split][m][r] = sum over the split's k of x[m, k] A[r, k]
template <int RT>                            // tiles of 8 ranks (R <= 8 RT)
__global__ void __launch_bounds__(128) lora_shrink_kernel(const LoraArgs p) {
    constexpr int STAGES = 3;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __half (*xs)[TM][LDK] = reinterpret_cast<__half (*)[TM][LDK]>(smem_raw);
    __half (*as)[RT * 8][LDK] = reinterpret_cast<__half (*)[RT * 8][LDK]>(smem_raw + sizeof(__half) * STAGES * TM * LDK);
    __shared__ int ids[TM];
    const int m0 = blockIdx.x * TM, split = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < TM) ids[threadIdx.x] = m0 + threadIdx.x < p.M ? adapter_of(p, m0 + threadIdx.x) : -1;
    __syncthreads();
    const int steps = (p.K + KT - 1) / KT;
    const int s0 = static_cast<int64_t>(steps) * split / p.ksplit, s1 = static_cast<int64_t>(steps) * (split + 1) / p.ksplit;
    const __half* X = reinterpret_cast<const __half*>(p.x);
    const __half* Ab = reinterpret_cast<const __half*>(p.A);

    for (int a = next_adapter(ids, -1); a != INT_MAX; a = next_adapter(ids, a)) {
        const __half* A = Ab + static_cast<int64_t>(a) * p.R * p.K;
        const auto stage = [&](int step) {
            if (step < s1) {
                const int k0 = step * KT, b = step % STAGES;
                for (int i = threadIdx.x; i < TM * (KT / 8); i += 128) {
                    const int r = i >> 3, c = (i & 7) * 8;
                    const bool live = m0 + r < p.M && k0 + c < p.K;
                    cp16(&xs[b][r][c], live ? X + static_cast<int64_t>(m0 + r) * p.K + k0 + c : X, live);
                }
                for (int i = threadIdx.x; i < RT * 8 * (KT / 8); i += 128) {
                    const int r = i >> 3, c = (i & 7) * 8;
                    const bool live = r < p.R && k0 + c < p.K;
                    cp16(&as[b][r][c], live ? A + static_cast<int64_t>(r) * p.K + k0 + c : A, live);
                }
            }
            cp_commit();
        };
        const bool mine = __any_sync(0xffffffffu, ids[warp * 16 + (lane & 15)] == a);
        float acc[RT][4];
#pragma unroll
        for (int n = 0; n < RT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[n][j] = 0.f;
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) stage(s0 + i);
        for (int step = s0; step < s1; ++step) {
            cp_wait<STAGES - 2>();
            __syncthreads();
            stage(step + STAGES - 1);
            const int b = step % STAGES;
            if (mine) {
#pragma unroll
                for (int k = 0; k < KT; k += 16) {
                    uint32_t fx[4];
                    ldsm4(fx, &xs[b][warp * 16 + (lane & 15)][k + (lane >> 4) * 8]);
#pragma unroll
                    for (int n = 0; n < RT; ++n) {
                        uint32_t fa[2];
                        ldsm2(fa, &as[b][n * 8 + (lane & 7)][k + ((lane >> 3) & 1) * 8]);
                        mma(acc[n], fx, fa);
                    }
                }
            }
        }
        cp_wait<0>();
        __syncthreads();                     // the stages are free for the next adapter
        if (!mine) continue;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = warp * 16 + half * 8 + (lane >> 2);
            if (ids[r] != a) continue;
            float* t = p.work + (static_cast<int64_t>(split) * p.M + m0 + r) * p.R + 2 * (lane & 3);
#pragma unroll
            for (int n = 0; n < RT; ++n)
                if (n * 8 < p.R) *reinterpret_cast<float2*>(t + n * 8) = make_float2(acc[n][2 * half], acc[n][2 * half + 1]);
        }
    }
}

// out = epi(y + scale t B^T)
template <typename T, int RK>                // steps of 16 ranks (R <= 16 RK)
__global__ void __launch_bounds__(256) lora_expand_kernel(const LoraArgs p) {
    constexpr int LDR = RK * 16 + 8;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __half (*hi)[LDR] = reinterpret_cast<__half (*)[LDR]>(smem_raw);
    __half (*lo)[LDR] = hi + TM;
    __half (*bs)[LDR] = lo + TM;
    __shared__ int ids[TM];
    __shared__ float back[TM];               // 2^-e of each token
    const int m0 = blockIdx.y * TM;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * NT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < TM) ids[threadIdx.x] = m0 + threadIdx.x < p.M ? adapter_of(p, m0 + threadIdx.x) : -1;
    __syncthreads();

    // this thread's outputs: rows mw + g and mw + g + 8, columns nw + 8 i + 2 q + 0..1
    const int mw = (warp & 3) * 16, g = lane >> 2, q = lane & 3;
    const int64_t nw = n0 + (warp >> 2) * 64;
    const bool pairs = (p.N & 1) == 0;
    float acc[8][4], yv[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int m = m0 + mw + g + 8 * half;
            const int64_t n = nw + 8 * i + 2 * q, at = static_cast<int64_t>(m) * p.N + n;
            acc[i][2 * half] = acc[i][2 * half + 1] = 0.f;
            yv[i][2 * half] = yv[i][2 * half + 1] = 0.f;
            if (m >= p.M || n >= p.N) continue;
            if (pairs) {
                float2 f;
                if constexpr (sizeof(T) == 4) f = *reinterpret_cast<const float2*>(static_cast<const float*>(p.y) + at);
                else f = __half22float2(*reinterpret_cast<const __half2*>(static_cast<const __half*>(p.y) + at));
                yv[i][2 * half] = f.x;
                yv[i][2 * half + 1] = f.y;
            } else {
                yv[i][2 * half] = get<T>(p.y, at);
                if (n + 1 < p.N) yv[i][2 * half + 1] = get<T>(p.y, at + 1);
            }
        }

    // t of each token, in two fp16 parts; four threads a token
    {
        const int r = threadIdx.x >> 2, c0 = threadIdx.x & 3, a = ids[r];
        const int rank = a >= 0 ? rank_of(p, a) : 0;
        const float s = a >= 0 && p.scale != nullptr ? p.scale[a] : 1.f;
        float t[RK * 4], top = 0.f;
#pragma unroll
        for (int i = 0; i < RK * 4; ++i) {
            const int c = c0 + 4 * i;
            float f = 0.f;
            if (c < rank)
                for (int k = 0; k < p.ksplit; ++k) f += p.work[(static_cast<int64_t>(k) * p.M + m0 + r) * p.R + c];
            t[i] = c < rank ? f * s : 0.f;
            const float mag = fabsf(t[i]);
            top = mag <= FLT_MAX ? fmaxf(top, mag) : top;    // infinities and NaN pass as they are
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the power of two that brings the largest |t| into [2^14, 2^15)
        const int ex = static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127;
        const int e = top > 0.f ? min(14 - ex, 100) : 0;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        if (c0 == 0) back[r] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < RK * 4; ++i) {
            const float f = t[i] * up;
            const __half h = __float2half_rn(f);
            const float rest = f - __half2float(h);
            hi[r][c0 + 4 * i] = h;
            lo[r][c0 + 4 * i] = __float2half_rn(fabsf(f) <= 65504.f ? rest : 0.f);   // an infinite t has no rest
        }
    }

    for (int a = next_adapter(ids, -1); a != INT_MAX; a = next_adapter(ids, a)) {
        const int rank = rank_of(p, a);
        const __half* B = reinterpret_cast<const __half*>(p.B) + static_cast<int64_t>(a) * p.N * p.R;
        for (int i = threadIdx.x; i < NT * RK * 2; i += 256) {
            const int r = i / (RK * 2), c = (i % (RK * 2)) * 8;
            const bool live = n0 + r < p.N && c < rank;
            cp16(&bs[r][c], live ? B + (n0 + r) * p.R + c : B, live);
        }
        cp_commit();
        cp_wait<0>();
        __syncthreads();
        if (rank & 7) {                      // columns behind the rank share its last piece: not the adapter's
            const int c = rank + threadIdx.x / NT;
            for (int cc = c; cc < (rank | 7) + 1; cc += 2) bs[threadIdx.x % NT][cc] = __float2half_rn(0.f);
            __syncthreads();
        }
        if (__any_sync(0xffffffffu, ids[mw + (lane & 15)] == a)) {
            const bool own0 = ids[mw + g] == a, own1 = ids[mw + g + 8] == a;
            uint32_t fh[RK][4], fl[RK][4];
#pragma unroll
            for (int k = 0; k < RK; ++k) {
                ldsm4(fh[k], &hi[mw + (lane & 15)][k * 16 + (lane >> 4) * 8]);
                ldsm4(fl[k], &lo[mw + (lane & 15)][k * 16 + (lane >> 4) * 8]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < RK; ++k) {
                    uint32_t fb[2];
                    ldsm2(fb, &bs[(warp >> 2) * 64 + i * 8 + (lane & 7)][k * 16 + ((lane >> 3) & 1) * 8]);
                    mma(c, fl[k], fb);
                    mma(c, fh[k], fb);
                }
                acc[i][0] = own0 ? c[0] : acc[i][0];
                acc[i][1] = own0 ? c[1] : acc[i][1];
                acc[i][2] = own1 ? c[2] : acc[i][2];
                acc[i][3] = own1 ? c[3] : acc[i][3];
            }
        }
        __syncthreads();
    }

#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = mw + g + 8 * half, m = m0 + r;
        if (m >= p.M) continue;
        const bool has = ids[r] >= 0;
        const float b = has ? back[r] : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t n = nw + 8 * i + 2 * q, at = static_cast<int64_t>(m) * p.N + n;
            if (n >= p.N) continue;
            float f0 = yv[i][2 * half], f1 = yv[i][2 * half + 1];
            if (has) {
                f0 = fmaf(acc[i][2 * half], b, f0);
                f1 = fmaf(acc[i][2 * half + 1], b, f1);
            }
            f0 = finish(f0, p.relu_sq);
            f1 = finish(f1, p.relu_sq);
            if (pairs) {
                if constexpr (sizeof(T) == 4) *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at) = make_float2(f0, f1);
                else *reinterpret_cast<__half2*>(static_cast<__half*>(p.out) + at) = __floats2half2_rn(f0, f1);
            } else {
                put<T>(p.out, at, f0);
                if (n + 1 < p.N) put<T>(p.out, at + 1, f1);
            }
        }
    }
}

template <int RT>
cudaError_t launch_shrink(const LoraArgs& a, cudaStream_t s) {
    constexpr int smem = 3 * (TM + RT * 8) * LDK * 2;
    const cudaError_t e = cudaFuncSetAttribute(lora_shrink_kernel<RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    lora_shrink_kernel<RT><<<dim3((a.M + TM - 1) / TM, a.ksplit), 128, smem, s>>>(a);
    return cudaGetLastError();
}
template <typename T, int RK>
cudaError_t launch_expand(const LoraArgs& a, cudaStream_t s) {
    constexpr int smem = (2 * TM + NT) * (RK * 16 + 8) * 2;
    const cudaError_t e = cudaFuncSetAttribute(lora_expand_kernel<T, RK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    lora_expand_kernel<T, RK><<<dim3(static_cast<unsigned>((a.N + NT - 1) / NT), (a.M + TM - 1) / TM), 256, smem, s>>>(a);
    return cudaGetLastError();
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
    const cudaError_t e = a.R <= 8    ? launch_shrink<1>(a, s)
                          : a.R <= 16 ? launch_shrink<2>(a, s)
                          : a.R <= 32 ? launch_shrink<4>(a, s)
                          : a.R <= 64 ? launch_shrink<8>(a, s)
                                      : launch_shrink<16>(a, s);
    if (e != cudaSuccess) return e;
    return a.R <= 16   ? launch_expand<T, 1>(a, s)
           : a.R <= 32 ? launch_expand<T, 2>(a, s)
           : a.R <= 64 ? launch_expand<T, 4>(a, s)
                       : launch_expand<T, 8>(a, s);
}

bool mis(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

rq_status check_sizes(int64_t M, int64_t K, int64_t N, int64_t L, int64_t R) {
    if (M < 1 || M > 64 * 65535 || K < 8 || K % 8 != 0 || K > (1 << 30)) return RQ_ERR_SHAPE;
    if (N < 1 || N > (int64_t{1} << 31) - 1 || L < 1 || L > (1 << 30)) return RQ_ERR_SHAPE;
    if (R < 8 || R % 8 != 0 || R > RQ_MAX_LORA_RANK) return RQ_ERR_SHAPE;
    return RQ_OK;
}

}  // namespace

// Enough CTAs for two per SM, each with at least four stages of k.
int lora_ksplit(int64_t M, int64_t K) {
    const int64_t tiles = (M + TM - 1) / TM, steps = (K + KT - 1) / KT;
    int64_t s = (2 * 148 + tiles - 1) / tiles;
    if (s > steps / 4) s = steps / 4;
    return static_cast<int>(s < 1 ? 1 : s > 32 ? 32 : s);
}

cudaError_t launch_lora_tokens(const LoraArgs& a, bool half, cudaStream_t s) {
    return half ? tokens<__half>(a, s) : tokens<float>(a, s);
}
cudaError_t launch_lora_tiles(const LoraArgs& a, bool half, cudaStream_t s) {
    return half ? tiles<__half>(a, s) : tiles<float>(a, s);
}

}  // namespace rq

using namespace rq;

extern "C" {

size_t rq_lora_work_bytes(int64_t M, int64_t K, int64_t R) {
    if (check_sizes(M, K, 1, 1, R) != RQ_OK || M <= kLoraTokens) return 0;
    return static_cast<size_t>(lora_ksplit(M, K)) * M * R * sizeof(float);
}

rq_status rq_lora_add(const uint16_t* x, int64_t M, int64_t K, const uint16_t* A, const uint16_t* B, int64_t L,
                      int64_t R, const int32_t* ids, const int32_t* ranks, const float* scale, const void* y,
                      void* out, int64_t N, int dtype, int epilogue, float* work, int* dev_status,
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
    a.work = work;
    a.status = dev_status;
    a.N = N;
    a.M = static_cast<int>(M);
    a.K = static_cast<int>(K);
    a.R = static_cast<int>(R);
    a.L = static_cast<int>(L);
    a.ksplit = lora_ksplit(M, K);
    a.relu_sq = epilogue == RQ_EPI_RELU_SQ;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool half = dtype == RQ_OUT_F16;
    const cudaError_t e = M <= kLoraTokens ? launch_lora_tokens(a, half, s) : launch_lora_tiles(a, half, s);
    if (e == cudaSuccess) return RQ_OK;
    record_cuda_error(e);
    return RQ_ERR_CUDA;
}

}  // extern "C"
