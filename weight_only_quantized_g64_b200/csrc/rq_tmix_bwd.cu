// rq_tmix_bwd.cu -- gradients of the time-mix recurrence, chunk by chunk.
//
// With the state before a chunk (S0, stored by the forward pass) and the
// gradient of the state behind it (G, stored by the backward walk of
// rq_tmix.cu) every chunk of C = 16 tokens stands alone.  Inside it the decay
// is divided out: W_t = prod_{s <= t} w_s, and with
//   R_t = W_t r_t,  A_t = W_{t-1} a_t,  B_t = b_t / W_t,  K_t = k_t / W_t
// the recurrence of S / W has no decay.  (w >= exp(-e^{-1/2}) > 0.545, so
// 1 / W <= 1.7e4 over a chunk.)  With L keeping t >= s and M keeping t > s of
// a 16 x 16 matrix, u_t = S_{t-1} a_t and e_t = G_t b_t as rows of U and E:
//   (1 - M(A B^T)) U = A S0^T + M(A K^T) V
//   (1 - M(A B^T))^T E = L(R B^T)^T dY + B G^T            (G times W_last)
//   dV = L(R K^T)^T dY + M(A K^T)^T E + K G^T
//   dR = dY S0 + L(dY U^T) B + L(dY V^T) K
//   dA = E S0 + M(E U^T) B + M(E V^T) K
//   dB = U G + L(dY U^T)^T R + M(E U^T)^T A
//   dK = V G + L(dY V^T)^T R + M(E V^T)^T A
// and the decay's gradient is a sum over the later tokens of the chunk,
//   dlogw_s = sum_{t >= s} (R dR - K dK - B dB)_t + sum_{t > s} (A dA)_t + Z,
//   Z = sum_i (S0 + U^T B + V^T K) G            (the state behind the chunk).
// About 50 000 fp32 FMA per token and head, all from shared memory.
#include "rq_tmix.cuh"

namespace rq {
namespace {

constexpr int C = kTmixChunk;
constexpr int LD = kHead + 4;                // row stride: 8 rows' 16-byte pieces meet no bank twice
constexpr int LM = C + 4;
#ifndef VAR_U
#define VAR_U 1
#endif
constexpr int U = VAR_U;
constexpr int THREADS = 256;

struct Smem {
    float R[C][LD], A[C][LD], B[C][LD], K[C][LD], V[C][LD], dY[C][LD], U[C][LD], E[C][LD], W[C][LD];
    float S0[kHead][LD], G[kHead][LD];
    float ab[C][LM], ak[C][LM], rb[C][LM], rk[C][LM], yu[C][LM], yv[C][LM], eu[C][LM], ev[C][LM];
    float z[kHead];
};

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

// A thread's 4 x 4 tile of a [16, 64] result: rows 4 tg + 0..3; columns
// 4 cg + 0..3 (tile "wide") or, where both operands lie along the sum,
// cg + 8 n (tile "tall": rows of the second operand, without bank conflicts).
struct Tile {
    float v[4][4];
};
struct Lane {
    int tg, cg, half;
    __device__ __forceinline__ int row(int m) const { return 4 * tg + m; }
    __device__ __forceinline__ int wide() const { return 32 * half + 4 * cg; }
    __device__ __forceinline__ int tall(int n) const { return 32 * half + cg + 8 * n; }
};

// X [16, 64] times Y [64, 64]^T, tall
__device__ __forceinline__ void mul_nt(Tile& a, const Lane& l, const float (*X)[LD], const float (*Y)[LD]) {
#pragma unroll U
    for (int k = 0; k < kHead; k += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = ld4(&X[l.row(m)][k]);
#pragma unroll
        for (int n = 0; n < 4; ++n) y[n] = ld4(&Y[l.tall(n)][k]);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n) a.v[m][n] = dot4(x[m], y[n], a.v[m][n]);
    }
}
// one row of the second operand times four factors, wide
__device__ __forceinline__ void rank1(Tile& a, const float f[4], float4 y) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        a.v[m][0] = fmaf(f[m], y.x, a.v[m][0]);
        a.v[m][1] = fmaf(f[m], y.y, a.v[m][1]);
        a.v[m][2] = fmaf(f[m], y.z, a.v[m][2]);
        a.v[m][3] = fmaf(f[m], y.w, a.v[m][3]);
    }
}
// X [16, N] times Y [N, 64], wide; X has row stride LX
template <int N, int LX>
__device__ __forceinline__ void mul_nn(Tile& a, const Lane& l, const float (*X)[LX], const float (*Y)[LD]) {
#pragma unroll U
    for (int k = 0; k < N; k += 4) {
        float4 x[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = ld4(&X[l.row(m)][k]);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const float f[4] = {(&x[0].x)[kk], (&x[1].x)[kk], (&x[2].x)[kk], (&x[3].x)[kk]};
            rank1(a, f, ld4(&Y[k + kk][l.wide()]));
        }
    }
}
// M [16, 16]^T times Y [16, 64], wide
__device__ __forceinline__ void mul_tn(Tile& a, const Lane& l, const float (*M)[LM], const float (*Y)[LD]) {
#pragma unroll U
    for (int k = 0; k < C; ++k) {
        const float4 x = ld4(&M[k][4 * l.tg]);
        const float f[4] = {x.x, x.y, x.z, x.w};
        rank1(a, f, ld4(&Y[k][l.wide()]));
    }
}
// the same, tall
__device__ __forceinline__ void mul_tn_tall(Tile& a, const Lane& l, const float (*M)[LM], const float (*Y)[LD]) {
#pragma unroll U
    for (int k = 0; k < C; ++k) {
        const float4 x = ld4(&M[k][4 * l.tg]);
        const float f[4] = {x.x, x.y, x.z, x.w};
        rank1(a, f, make_float4(Y[k][l.tall(0)], Y[k][l.tall(1)], Y[k][l.tall(2)], Y[k][l.tall(3)]));
    }
}
__device__ __forceinline__ void mul_nn_tall(Tile& a, const Lane& l, const float (*M)[LM], const float (*Y)[LD]) {
#pragma unroll U
    for (int k = 0; k < C; ++k) {
        const float f[4] = {M[l.row(0)][k], M[l.row(1)][k], M[l.row(2)][k], M[l.row(3)][k]};
        rank1(a, f, make_float4(Y[k][l.tall(0)], Y[k][l.tall(1)], Y[k][l.tall(2)], Y[k][l.tall(3)]));
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 2) tmix_chunk_bwd_kernel(const TmixArgs p) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int tid = threadIdx.x;
    const int h = blockIdx.x % p.H, place = blockIdx.x / p.H;

    // the sequence whose stored states hold this place: the last one whose first is not behind it
    int a = 0, b = p.S - 1;
    while (a < b) {
        const int m = (a + b + 1) >> 1;
        if (ckpt_base(p.seq_start[m], m) <= place) a = m;
        else b = m - 1;
    }
    int lo, hi;
    if (!sequence_of(p, a, lo, hi)) return;
    const int64_t first = ckpt_base(lo, a);
    if (place < first || place - first >= (hi - lo + C - 1) / C) return;
    const int64_t t0 = lo + (place - first) * C;
    const int nt = static_cast<int>(min(static_cast<int64_t>(C), hi - t0));

    // ---- load
    const int64_t state = (static_cast<int64_t>(place) * p.H + h) * kHead * kHead;
    for (int i = tid; i < kHead * kHead / 4; i += THREADS) {
        const int r = i >> 4, c = (i & 15) * 4;
        *reinterpret_cast<float4*>(&sm.S0[r][c]) = ld4(p.ckpt + state + 4 * i);
        *reinterpret_cast<float4*>(&sm.G[r][c]) = ld4(p.gckpt + state + 4 * i);
    }
    const int et = tid >> 4, ec = (tid & 15) * 4;        // this thread's 4 elements of every [16, 64] array
    const int64_t in_at = (t0 + et) * p.ld + static_cast<int64_t>(h) * kHead + ec;
    const int64_t out_at = ((t0 + et) * p.H + h) * kHead + ec;
    const bool in = et < nt;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto get = [&](int i) { return in ? load4(static_cast<const T*>(p.in[i]) + in_at) : zero; };
    const float4 xr = get(0), xd = get(1), xk = get(2), xv = get(3), xa = get(4), xb = get(5);
    const float4 xy = in ? load4(static_cast<const T*>(p.dy) + out_at) : zero;
    *reinterpret_cast<float4*>(&sm.V[et][ec]) = xv;
    *reinterpret_cast<float4*>(&sm.dY[et][ec]) = xy;
    *reinterpret_cast<float4*>(&sm.W[et][ec]) =
        in ? make_float4(decay_m1(xd.x), decay_m1(xd.y), decay_m1(xd.z), decay_m1(xd.w)) : zero;
    __syncthreads();
    if (tid < kHead) {                                   // W_t
        float w = 1.f;
#pragma unroll
        for (int t = 0; t < C; ++t) {
            w = fmaf(w, sm.W[t][tid], w);
            sm.W[t][tid] = w;
        }
    }
    __syncthreads();
    const auto mul = [](float4 x, float4 y) { return make_float4(x.x * y.x, x.y * y.y, x.z * y.z, x.w * y.w); };
    {
        const float4 w = ld4(&sm.W[et][ec]);
        const float4 wp = et ? ld4(&sm.W[et - 1][ec]) : make_float4(1.f, 1.f, 1.f, 1.f);
        const float4 iw = make_float4(1.f / w.x, 1.f / w.y, 1.f / w.z, 1.f / w.w);
        *reinterpret_cast<float4*>(&sm.R[et][ec]) = mul(xr, w);
        *reinterpret_cast<float4*>(&sm.A[et][ec]) = mul(xa, wp);
        *reinterpret_cast<float4*>(&sm.B[et][ec]) = mul(xb, iw);
        *reinterpret_cast<float4*>(&sm.K[et][ec]) = mul(xk, iw);
        for (int i = tid; i < kHead * kHead / 4; i += THREADS) {
            const int r = i >> 4, c = (i & 15) * 4;
            float4* g = reinterpret_cast<float4*>(&sm.G[r][c]);
            *g = mul(*g, ld4(&sm.W[C - 1][c]));
        }
    }
    __syncthreads();

    // ---- the 16 x 16 products that need no solution
    const int mt = tid >> 4, ms = tid & 15;
    {
        float ab = 0.f, ak = 0.f, rb = 0.f, rk = 0.f, yv = 0.f;
#pragma unroll U
        for (int k = 0; k < kHead; k += 4) {
            const float4 A = ld4(&sm.A[mt][k]), R = ld4(&sm.R[mt][k]), Y = ld4(&sm.dY[mt][k]);
            const float4 B = ld4(&sm.B[ms][k]), K = ld4(&sm.K[ms][k]), V = ld4(&sm.V[ms][k]);
            ab = dot4(A, B, ab);
            ak = dot4(A, K, ak);
            rb = dot4(R, B, rb);
            rk = dot4(R, K, rk);
            yv = dot4(Y, V, yv);
        }
        sm.ab[mt][ms] = mt > ms ? ab : 0.f;
        sm.ak[mt][ms] = mt > ms ? ak : 0.f;
        sm.rb[mt][ms] = mt >= ms ? rb : 0.f;
        sm.rk[mt][ms] = mt >= ms ? rk : 0.f;
        sm.yv[mt][ms] = mt >= ms ? yv : 0.f;
    }
    __syncthreads();

    // ---- right-hand sides; each pair of warps takes one [16, 64] result
    const int warp = tid >> 5, lane = tid & 31, pair = warp >> 1;
    const Lane l = {lane >> 3, lane & 7, warp & 1};
    Tile acc;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) acc.v[m][n] = 0.f;
    if (pair == 0) {
        mul_nt(acc, l, sm.A, sm.S0);
        mul_nn_tall(acc, l, sm.ak, sm.V);
    } else if (pair == 1) {
        mul_nt(acc, l, sm.B, sm.G);
        mul_tn_tall(acc, l, sm.rb, sm.dY);
    } else if (pair == 2) {
        mul_nt(acc, l, sm.K, sm.G);
        mul_tn_tall(acc, l, sm.rk, sm.dY);
    } else {
        mul_nn<kHead, LD>(acc, l, sm.dY, sm.S0);
    }
    if (pair < 2) {
        float (*dst)[LD] = pair ? sm.E : sm.U;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n) dst[l.row(m)][l.tall(n)] = acc.v[m][n];
    }
    __syncthreads();

    // ---- triangular solutions, one column per thread
    if (tid < kHead) {
        float u[C];
#pragma unroll
        for (int t = 0; t < C; ++t) u[t] = sm.U[t][tid];
#pragma unroll
        for (int t = 1; t < C; ++t)
#pragma unroll
            for (int s = 0; s < t; ++s) u[t] = fmaf(sm.ab[t][s], u[s], u[t]);
#pragma unroll
        for (int t = 1; t < C; ++t) sm.U[t][tid] = u[t];
    } else if (tid < 2 * kHead) {
        float e[C];
#pragma unroll
        for (int t = 0; t < C; ++t) e[t] = sm.E[t][tid - kHead];
#pragma unroll
        for (int s = C - 2; s >= 0; --s)
#pragma unroll
            for (int t = s + 1; t < C; ++t) e[s] = fmaf(sm.ab[t][s], e[t], e[s]);
#pragma unroll
        for (int t = 0; t < C - 1; ++t) sm.E[t][tid - kHead] = e[t];
    }
    __syncthreads();
    {
        float yu = 0.f, eu = 0.f, ev = 0.f;
#pragma unroll U
        for (int k = 0; k < kHead; k += 4) {
            const float4 Y = ld4(&sm.dY[mt][k]), E = ld4(&sm.E[mt][k]);
            const float4 U = ld4(&sm.U[ms][k]), V = ld4(&sm.V[ms][k]);
            yu = dot4(Y, U, yu);
            eu = dot4(E, U, eu);
            ev = dot4(E, V, ev);
        }
        sm.yu[mt][ms] = mt >= ms ? yu : 0.f;
        sm.eu[mt][ms] = mt > ms ? eu : 0.f;
        sm.ev[mt][ms] = mt > ms ? ev : 0.f;
    }
    __syncthreads();

    // ---- gradients.  decay[]: what each product adds to the decay's gradient, per token and channel
    T* const out[6] = {static_cast<T*>(p.out[0]), static_cast<T*>(p.out[1]), static_cast<T*>(p.out[2]),
                       static_cast<T*>(p.out[3]), static_cast<T*>(p.out[4]), static_cast<T*>(p.out[5])};
    const auto at = [&](int t) { return ((t0 + t) * p.H + h) * kHead; };
    if (pair == 2) {                                     // dV: add M(A K^T)^T E to the held sum
        mul_tn_tall(acc, l, sm.ak, sm.E);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (l.row(m) < nt) out[3][at(l.row(m)) + l.tall(n)] = from_f32<T>(acc.v[m][n]);
    }
    if (pair < 3) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n) acc.v[m][n] = 0.f;
    }
    float zpart[4] = {0.f, 0.f, 0.f, 0.f};               // sum over this thread's rows of (B or K) times (U G or V G)
    if (pair == 0) {                                     // dA
        mul_nn<kHead, LD>(acc, l, sm.E, sm.S0);
        mul_nn<C, LM>(acc, l, sm.eu, sm.B);
        mul_nn<C, LM>(acc, l, sm.ev, sm.K);
    } else if (pair == 1) {                              // dB
        mul_nn<kHead, LD>(acc, l, sm.U, sm.G);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n) zpart[n] = fmaf(acc.v[m][n], sm.B[l.row(m)][l.wide() + n], zpart[n]);
        mul_tn(acc, l, sm.yu, sm.R);
        mul_tn(acc, l, sm.eu, sm.A);
    } else if (pair == 2) {                              // dK
        mul_nn<kHead, LD>(acc, l, sm.V, sm.G);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n) zpart[n] = fmaf(acc.v[m][n], sm.K[l.row(m)][l.wide() + n], zpart[n]);
        mul_tn(acc, l, sm.yv, sm.R);
        mul_tn(acc, l, sm.ev, sm.A);
    } else {                                             // dR
        mul_nn<C, LM>(acc, l, sm.yu, sm.B);
        mul_nn<C, LM>(acc, l, sm.yv, sm.K);
        float z = 0.f;
        const int j = tid - 6 * 32;                      // 64 threads, one channel each
#pragma unroll 4
        for (int i = 0; i < kHead; ++i) z = fmaf(sm.S0[i][j], sm.G[i][j], z);
        sm.z[j] = z;
    }
    // the four row groups of a warp add their parts of Z in a fixed order
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        zpart[n] += __shfl_xor_sync(0xffffffffu, zpart[n], 8);
        zpart[n] += __shfl_xor_sync(0xffffffffu, zpart[n], 16);
    }
    float4 own[4];                                       // this product's operand rows, before they are overwritten
    {
        const float (*X)[LD] = pair == 0 ? sm.A : pair == 1 ? sm.B : pair == 2 ? sm.K : sm.R;
#pragma unroll
        for (int m = 0; m < 4; ++m) own[m] = ld4(&X[l.row(m)][l.wide()]);
    }
    __syncthreads();                                     // U, E, S0 and G are free from here
    float (*dl)[LD] = &sm.S0[16 * pair];                 // four [16, 64] arrays in the place of S0
    {
        T* o = out[pair == 0 ? 4 : pair == 1 ? 5 : pair == 2 ? 2 : 0];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int t = l.row(m);
            const float4 g = make_float4(acc.v[m][0], acc.v[m][1], acc.v[m][2], acc.v[m][3]);
            *reinterpret_cast<float4*>(&dl[t][l.wide()]) = mul(own[m], g);
            float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
            if (pair != 0) w = ld4(&sm.W[t][l.wide()]);
            else if (t > 0) w = ld4(&sm.W[t - 1][l.wide()]);
            if (pair == 1 || pair == 2) w = make_float4(1.f / w.x, 1.f / w.y, 1.f / w.z, 1.f / w.w);
            if (t < nt) store4(o + at(t) + l.wide(), mul(g, w));
        }
        if ((pair == 1 || pair == 2) && l.tg == 0)
            *reinterpret_cast<float4*>(&sm.G[pair][l.wide()]) = make_float4(zpart[0], zpart[1], zpart[2], zpart[3]);
    }
    __syncthreads();
    if (tid < kHead) {
        const float (*dA)[LD] = &sm.S0[0], (*dB)[LD] = &sm.S0[16], (*dK)[LD] = &sm.S0[32], (*dR)[LD] = &sm.S0[48];
        float sum = sm.z[tid] + sm.G[1][tid] + sm.G[2][tid];
#pragma unroll
        for (int t = C - 1; t >= 0; --t) {
            sum += (dR[t][tid] - dK[t][tid]) - dB[t][tid];
            if (t + 1 < C) sum += dA[t + 1][tid];
            sm.E[t][tid] = sum;
        }
    }
    __syncthreads();
    if (in) {
        const float4 g = ld4(&sm.E[et][ec]);
        const auto dd = [](float dlogw, float d) {
            const float s = decay_gate(d);
            return dlogw * (-kDecay * s * (1.f - s));
        };
        store4(out[1] + out_at, make_float4(dd(g.x, xd.x), dd(g.y, xd.y), dd(g.z, xd.z), dd(g.w, xd.w)));
    }
}

template <typename T>
cudaError_t launch(const TmixArgs& a, cudaStream_t s) {
    const cudaError_t e = allow_smem<tmix_chunk_bwd_kernel<T>>(sizeof(Smem));
    if (e != cudaSuccess) return e;
    const int64_t places = a.T / C + a.S;
    tmix_chunk_bwd_kernel<T><<<static_cast<unsigned>(places * a.H), THREADS, sizeof(Smem), s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tmix_chunks_bwd(const TmixArgs& a, bool half, cudaStream_t s) {
    return half ? launch<__half>(a, s) : launch<float>(a, s);
}

}  // namespace rq
