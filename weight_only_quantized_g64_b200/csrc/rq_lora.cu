// rq_lora.cu -- low-rank adapters of many requests beside one product:
//   out[m] = epi(y[m] + s_a B_a (A_a x[m])),   a = ids[m].
//
// One launch either way: a cluster of CTAs splits K for A x, exchanges the R
// sums of each token through distributed shared memory, and splits N for B.
//
// Few tokens (decode): a cluster of 8 per token, plain fp32 sums.  Its part of
// B (one contiguous piece) is sent for into L2 at the start, and its first rows
// into registers before the cluster meets.  Bound by latency: two dependent
// reads of memory and a barrier.
//
// Many tokens (prefill): a cluster per 64 tokens on the warp-level tensor
// cores.  The products of A x are exact in fp32; for B each fp32 sum t is split
// into two fp16 parts, t = 2^-e (hi + lo), scaled per token so that the largest
// lies near 2^14, so 22 bits of it enter the product.  Bound by the bytes of x,
// y and out.  A tile whose tokens use several adapters takes them in turn and
// keeps each token's own.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
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
    if (threadIdx.x == 0 && n1 > n0) {
        const char* from = reinterpret_cast<const char*>(p.B + (static_cast<int64_t>(a) * p.N + n0) * p.R);
        const uint32_t size = static_cast<uint32_t>(min((n1 - n0) * p.R * 2, int64_t{1} << 20));
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(size) : "memory");
    }

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
constexpr int STAGES = 3;

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

// Four consecutive outputs of row m from column n on; `wide`: 4 | N.
template <typename T>
__device__ __forceinline__ void get4(const void* p, int64_t at, int64_t left, bool wide, float f[4]) {
    if (wide && left >= 4) {
        if constexpr (sizeof(T) == 4) {
            const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
            f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __half*>(p) + at);
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
            f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = j < left ? get<T>(p, at + j) : 0.f;
}
template <typename T>
__device__ __forceinline__ void put4(void* p, int64_t at, int64_t left, bool wide, const float f[4]) {
    if (wide && left >= 4) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(f[0], f[1], f[2], f[3]);
        } else {
            const __half2 a = __floats2half2_rn(f[0], f[1]), b = __floats2half2_rn(f[2], f[3]);
            *reinterpret_cast<uint2*>(static_cast<__half*>(p) + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < left) put<T>(p, at + j, f[j]);
}

// RT: tiles of 8 ranks (R <= 8 RT)
template <int RT>
struct TileSmem {
    static constexpr int RK = RT < 2 ? 1 : RT / 2;       // steps of 16 ranks
    static constexpr int LDR = RK * 16 + 8;
    static constexpr int LDP = RT * 8 + 4;
    union {
        struct {
            __half x[STAGES][TM][LDK], a[STAGES][RT * 8][LDK];
        } in;
        __half b[2][NT][LDR];
    };
    __half hi[TM][LDR], lo[TM][LDR];
    float part[TM][LDP];
    float back[TM];                          // 2^-e of each token
    int ids[TM];
};

template <typename T, int RT>
__global__ void __launch_bounds__(256, RT <= 8 ? 2 : 1) lora_tile_kernel(const LoraArgs p) {
    using Smem = TileSmem<RT>;
    constexpr int RK = Smem::RK;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), me = cluster.block_rank();
    const int m0 = blockIdx.x / ctas * TM;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    if (tid < TM) sm.ids[tid] = m0 + tid < p.M ? adapter_of(p, m0 + tid) : -1;
    __syncthreads();

    // ---- part[m][r] = sum over this CTA's k of x[m, k] A[r, k]; a warp takes 16 tokens and half of each stage
    const int steps = (p.K + KT - 1) / KT;
    const int s0 = static_cast<int64_t>(steps) * me / ctas, s1 = static_cast<int64_t>(steps) * (me + 1) / ctas;
    const int mw = (warp & 3) * 16, kh = warp >> 2, g = lane >> 2, q = lane & 3;
    const __half* X = reinterpret_cast<const __half*>(p.x);
    for (int a = next_adapter(sm.ids, -1); a != INT_MAX; a = next_adapter(sm.ids, a)) {
        const __half* A = reinterpret_cast<const __half*>(p.A) + static_cast<int64_t>(a) * p.R * p.K;
        const auto stage = [&](int step) {
            if (step < s1) {
                const int k0 = step * KT, b = (step - s0) % STAGES;
#pragma unroll
                for (int i = tid; i < TM * (KT / 8); i += 256) {
                    const int r = i >> 3, c = (i & 7) * 8;
                    const bool live = m0 + r < p.M && k0 + c < p.K;
                    cp16(&sm.in.x[b][r][c], live ? X + static_cast<int64_t>(m0 + r) * p.K + k0 + c : X, live);
                }
                for (int i = tid; i < RT * 8 * (KT / 8); i += 256) {
                    const int r = i >> 3, c = (i & 7) * 8;
                    const bool live = r < p.R && k0 + c < p.K;
                    cp16(&sm.in.a[b][r][c], live ? A + static_cast<int64_t>(r) * p.K + k0 + c : A, live);
                }
            }
            cp_commit();
        };
        const bool mine = __any_sync(0xffffffffu, sm.ids[mw + (lane & 15)] == a);
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
            const int b = (step - s0) % STAGES;
            if (mine) {
#pragma unroll
                for (int k = kh * 32; k < kh * 32 + 32; k += 16) {
                    uint32_t fx[4];
                    ldsm4(fx, &sm.in.x[b][mw + (lane & 15)][k + (lane >> 4) * 8]);
#pragma unroll
                    for (int n = 0; n < RT; ++n) {
                        uint32_t fa[2];
                        ldsm2(fa, &sm.in.a[b][n * 8 + (lane & 7)][k + ((lane >> 3) & 1) * 8]);
                        mma(acc[n], fx, fa);
                    }
                }
            }
        }
        cp_wait<0>();
        // the two halves of the stages are added through shared memory: part is the second's, then the sum
        const bool own[2] = {sm.ids[mw + g] == a, sm.ids[mw + g + 8] == a};
#pragma unroll
        for (int turn = 1; turn >= 0; --turn) {
            if (kh == turn && mine) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!own[half]) continue;
#pragma unroll
                    for (int n = 0; n < RT; ++n) {
                        float2* at = reinterpret_cast<float2*>(&sm.part[mw + g + 8 * half][n * 8 + 2 * q]);
                        float2 v = make_float2(acc[n][2 * half], acc[n][2 * half + 1]);
                        if (turn == 0) {
                            const float2 o = *at;
                            v = make_float2(v.x + o.x, v.y + o.y);
                        }
                        *at = v;
                    }
                }
            }
            __syncthreads();                 // and the stages are free for the next adapter
        }
    }

    // ---- B of the first tile on its way, then the cluster's sums
    const int tiles = static_cast<int>((p.N + NT - 1) / NT);
    const auto fetch = [&](int tile, int a, int buf) {
        const int rank = rank_of(p, a);
        const __half* B = reinterpret_cast<const __half*>(p.B) + static_cast<int64_t>(a) * p.N * p.R;
        const int64_t n0 = static_cast<int64_t>(tile) * NT;
#pragma unroll 4
        for (int i = tid; i < NT * RK * 2; i += 256) {
            const int r = i / (RK * 2), c = (i % (RK * 2)) * 8;
            const bool live = n0 + r < p.N && c < rank;
            cp16(&sm.b[buf][r][c], live ? B + (n0 + r) * p.R + c : B, live);
        }
        cp_commit();
    };
    const int first = next_adapter(sm.ids, -1);
    if (first != INT_MAX && me < tiles) fetch(me, first, 0);
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    {                                        // four threads a token
        const int r = tid >> 2, c0 = (tid & 3) * 4, a = sm.ids[r];
        const int rank = a >= 0 ? rank_of(p, a) : 0;
        const float s = a >= 0 && p.scale != nullptr ? p.scale[a] : 1.f;
        float t[RK][4], top = 0.f;
#pragma unroll
        for (int i = 0; i < RK; ++i) {
            const int c = c0 + 16 * i;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < rank) {
                for (int k = 0; k < ctas; ++k) {
                    const float4 v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&sm.part[r][c], k));
                    f.x += v.x; f.y += v.y; f.z += v.z; f.w += v.w;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                t[i][j] = c + j < rank ? (&f.x)[j] * s : 0.f;
                const float mag = fabsf(t[i][j]);
                top = mag <= FLT_MAX ? fmaxf(top, mag) : top;    // infinities and NaN pass as they are
            }
        }
        // no CTA leaves before the others have read its sums
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the power of two that brings the largest |t| into [2^14, 2^15)
        const int ex = static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127;
        const int e = top > 0.f ? min(14 - ex, 100) : 0;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        if ((tid & 3) == 0) sm.back[r] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < RK; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float f = t[i][j] * up;
                const __half h = __float2half_rn(f);
                sm.hi[r][c0 + 16 * i + j] = h;
                // an infinite t has no rest
                sm.lo[r][c0 + 16 * i + j] = __float2half_rn(fabsf(f) <= 65504.f ? f - __half2float(h) : 0.f);
            }
    }
    __syncthreads();

    // ---- out = epi(y + t B^T); warp: 16 tokens x 64 outputs of a tile.  A thread's columns of a pair of 8-column
    // products are four neighbours: product column c of product i stands for output 16 (i / 2) + 4 (c / 2) + 2 (i % 2)
    // + c % 2.
    const bool wide = (p.N & 3) == 0;
    const int64_t rows[2] = {m0 + mw + g, m0 + mw + g + 8};
    const float back[2] = {sm.ids[mw + g] >= 0 ? sm.back[mw + g] : 0.f,
                           sm.ids[mw + g + 8] >= 0 ? sm.back[mw + g + 8] : 0.f};
    int buf = 0;
    for (int tile = me; tile < tiles; tile += ctas) {
        const int64_t nw = static_cast<int64_t>(tile) * NT + (warp >> 2) * 64 + 4 * q;
        float acc[4][2][4];                  // [16 outputs][row half][neighbour]: y, then the sum
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half)
                if (rows[half] < p.M)
                    get4<T>(p.y, rows[half] * p.N + nw + 16 * i, p.N - nw - 16 * i, wide, acc[i][half]);
        for (int a = first; a != INT_MAX;) {
            const int after = next_adapter(sm.ids, a);
            if (after != INT_MAX) fetch(tile, after, buf ^ 1);
            else if (tile + ctas < tiles) fetch(tile + ctas, first, buf ^ 1);
            else cp_commit();
            cp_wait<1>();
            __syncthreads();
            const int rank = rank_of(p, a);
            if (rank & 7) {                  // columns behind the rank share its last piece: not the adapter's
                for (int c = rank + tid / NT; c < (rank | 7) + 1; c += 2) sm.b[buf][tid % NT][c] = __float2half_rn(0.f);
                __syncthreads();
            }
            if (__any_sync(0xffffffffu, sm.ids[mw + (lane & 15)] == a)) {
                float c[8][4];
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
#pragma unroll
                for (int k = 0; k < RK; ++k) {
                    uint32_t fh[4], fl[4];
                    ldsm4(fh, &sm.hi[mw + (lane & 15)][k * 16 + (lane >> 4) * 8]);
                    ldsm4(fl, &sm.lo[mw + (lane & 15)][k * 16 + (lane >> 4) * 8]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int col = lane & 7;
                        uint32_t fb[2];
                        ldsm2(fb, &sm.b[buf][(warp >> 2) * 64 + 16 * (i >> 1) + 4 * (col >> 1) + 2 * (i & 1) + (col & 1)]
                                        [k * 16 + ((lane >> 3) & 1) * 8]);
                        mma(c[i], fl, fb);
                        mma(c[i], fh, fb);
                    }
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (sm.ids[mw + g + 8 * half] != a) continue;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float& f = acc[i >> 1][half][2 * (i & 1) + j];
                            f = fmaf(c[i][2 * half + j], back[half], f);
                        }
                }
            }
            __syncthreads();
            buf ^= 1;
            a = after;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (rows[half] >= p.M) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][half][j] = finish(acc[i][half][j], p.relu_sq);
                put4<T>(p.out, rows[half] * p.N + nw + 16 * i, p.N - nw - 16 * i, wide, acc[i][half]);
            }
    }
    cp_wait<0>();
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

template <typename T, int RT>
cudaError_t launch_tiles(const LoraArgs& a, cudaStream_t s) {
    constexpr int smem = sizeof(TileSmem<RT>);
    cudaError_t e = allow_smem<lora_tile_kernel<T, RT>>(smem);
    if (e != cudaSuccess) return e;
    const int tiles = (a.M + TM - 1) / TM;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles * CS);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_tile_kernel<T, RT>, a);
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
    if (M < 1 || M >= (1 << 24) || K < 8 || K % 8 != 0 || K > (1 << 30)) return RQ_ERR_SHAPE;
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

rq_status rq_lora_add(const uint16_t* x, int64_t M, int64_t K, const uint16_t* A, const uint16_t* B, int64_t L,
                      int64_t R, const int32_t* ids, const int32_t* ranks, const float* scale, const void* y,
                      void* out, int64_t N, int dtype, int epilogue, int* dev_status, rq_stream_t stream) {
    if (dtype != RQ_OUT_F32 && dtype != RQ_OUT_F16) return RQ_ERR_RANGE;
    if (epilogue != RQ_EPI_NONE && epilogue != RQ_EPI_RELU_SQ) return RQ_ERR_RANGE;
    const rq_status st = check_sizes(M, K, N, L, R);
    if (st != RQ_OK) return st;
    if (x == nullptr || A == nullptr || B == nullptr || ids == nullptr || y == nullptr || out == nullptr)
        return RQ_ERR_NULL;
    if (mis(x, 16) || mis(A, 16) || mis(B, 16) || mis(y, 16) || mis(out, 16) || mis(ids, 4) ||
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
