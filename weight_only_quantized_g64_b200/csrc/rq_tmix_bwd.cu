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
// About 800 000 multiplications per chunk and head, on the tensor cores
// (rq_tf32.cuh): 2300 MMAs of 8 cycles over the four of an SM bound it.  With
// plain FMAs the kernel was bound by shared-memory reads at 4 x 4 results per
// thread: 322 us where this takes 197 (2048 tokens, 32 heads, fp16).
// The loops over the summed index are not unrolled: the code of all products is
// what the instruction cache holds least of (steps of 2 together 205 us, all 268).
// A value that is not finite may spoil the gradients of its chunk of 16 tokens.
#include "rq_tf32.cuh"
#include "rq_tmix.cuh"

namespace rq {
namespace {

constexpr int C = kTmixChunk;
constexpr int LD = kHead + 8;                // rows 8 banks apart: the pairs that eight lanes of a column group read
constexpr int LM = C + 8;
constexpr int THREADS = 256;
static_assert(LD % 4 == 0 && LM % 4 == 0);   // 16-byte accesses: every row is a multiple of 16 bytes

struct alignas(16) Smem {
    float R[C][LD], A[C][LD], B[C][LD], K[C][LD], V[C][LD], dY[C][LD], U[C][LD], E[C][LD], W[C][LD];
    float S0[kHead][LD], G[kHead][LD];
    float ab[C][LM], ak[C][LM], rb[C][LM], rk[C][LM], yu[C][LM], yv[C][LM], eu[C][LM], ev[C][LM];
    float z[3][kHead];                       // the parts of Z: S0, U^T B, V^T K
};

__device__ __forceinline__ void cp16(float* dst, const float* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// Half of a [16, 64] result per warp: four products of 8 columns, c[n] the
// columns 32 half + 8 n.
using Half = Sums<4>;
struct Lane {
    int g, q, first;                         // first: 32 half
};
// c += X Y^T, X [16, 64], Y [64, 64]
__device__ __forceinline__ void times_rows(Half& c, const Lane& l, const float (*X)[LD], const float (*Y)[LD]) {
#pragma unroll 1
    for (int k = 0; k < kHead; k += 8) {
        float4 b[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) b[n] = along(&Y[l.first + 8 * n + l.g][k + 2 * l.q]);
        products(c, rows_at(X, l.g, k + 2 * l.q), b);
    }
}
// c += X Y, X [16, N] (or, TRANSPOSED, of X [N, 16] the columns), Y [N, 64]
template <int N, bool TRANSPOSED, int LX>
__device__ __forceinline__ void times(Half& c, const Lane& l, const float (*X)[LX], const float (*Y)[LD]) {
#pragma unroll 1
    for (int k = 0; k < N; k += 8) {
        float4 b[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) b[n] = down(&Y[k + 2 * l.q][l.first + 8 * n + l.g], LD);
        products(c, TRANSPOSED ? columns_at(X, l.g, k + 2 * l.q) : rows_at(X, l.g, k + 2 * l.q), b);
    }
}
// m = X Y^T, both [16, 64], what lies above the diagonal (or on it, STRICT) zero
__device__ __forceinline__ void square(float (*m)[LM], const Lane& l, const float (*X)[LD], const float (*Y)[LD],
                                       bool strict) {
    Sums<2> c;                               // two column halves
    c.clear();
#pragma unroll 1
    for (int k = 0; k < kHead; k += 8) {
        const int at = k + 2 * l.q;
        const float4 b[2] = {along(&Y[l.g][at]), along(&Y[8 + l.g][at])};
        products(c, rows_at(X, l.g, at), b);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = l.g + 8 * (j >> 1), s = 8 * n + 2 * l.q + (j & 1);
            m[t][s] = t > s || (t == s && !strict) ? c.at(n, j) : 0.f;
        }
}
__device__ __forceinline__ void put(const Half& c, const Lane& l, float (*to)[LD]) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const int k = l.first + 8 * n + 2 * l.q;
        *reinterpret_cast<float2*>(&to[l.g][k]) = make_float2(c.at(n, 0), c.at(n, 1));
        *reinterpret_cast<float2*>(&to[l.g + 8][k]) = make_float2(c.at(n, 2), c.at(n, 3));
    }
}
// sum over the 16 tokens of c times X, into z
__device__ __forceinline__ void weigh(const Half& c, const Lane& l, const float (*X)[LD], float* z) {
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = l.first + 8 * n + 2 * l.q + j;
            float s = fmaf(c.at(n, j), X[l.g][k], c.at(n, j + 2) * X[l.g + 8][k]);
            s += __shfl_xor_sync(0xffffffffu, s, 4);
            s += __shfl_xor_sync(0xffffffffu, s, 8);
            s += __shfl_xor_sync(0xffffffffu, s, 16);
            if (l.g == 0) z[k] = s;
        }
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 2) tmix_chunk_bwd_kernel(const TmixArgs p) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int tid = threadIdx.x;
    const int h = blockIdx.x % p.H, place = blockIdx.x / p.H;

    // the stored states (every place has memory, whether a chunk uses it or not), on their way while the rest is found
    const int64_t state = (static_cast<int64_t>(place) * p.H + h) * kHead * kHead;
    for (int i = tid; i < kHead * kHead / 4; i += THREADS) {
        const int r = i >> 4, c = (i & 15) * 4;
        cp16(&sm.S0[r][c], p.ckpt + state + 4 * i);
        cp16(&sm.G[r][c], p.gckpt + state + 4 * i);
    }

    // the sequence whose stored states hold this place: the last one whose first is not behind it
    int a = 0, b = p.S - 1;
    while (a < b) {
        const int m = (a + b + 1) >> 1;
        if (ckpt_base(p.seq_start[m], m) <= place) a = m;
        else b = m - 1;
    }
    int lo, hi;
    const bool whole = sequence_of(p, a, lo, hi);
    const int64_t first = ckpt_base(lo, a);
    if (!whole || place < first || place - first >= (hi - lo + C - 1) / C) {
        cp_wait();
        return;
    }
    const int64_t t0 = lo + (place - first) * C;
    const int nt = static_cast<int>(min(static_cast<int64_t>(C), hi - t0));

    // ---- load
    const int et = tid >> 4, ec = (tid & 15) * 4;        // this thread's 4 elements of every [16, 64] array
    const int64_t in_at = (t0 + et) * p.ld + static_cast<int64_t>(h) * kHead + ec;
    const int64_t out_at = ((t0 + et) * p.H + h) * kHead + ec;
    const bool in = et < nt;
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto get = [&](int i) { return in ? load4(static_cast<const T*>(p.in[i]) + in_at) : none; };
    const auto mul = [](float4 x, float4 y) { return make_float4(x.x * y.x, x.y * y.y, x.z * y.z, x.w * y.w); };
    const auto row4 = [&](float (*to)[LD], float4 v) { *reinterpret_cast<float4*>(&to[et][ec]) = v; };
    float4 xd;
    {
        const float4 xr = get(0), xk = get(2), xv = get(3), xa = get(4), xb = get(5);
        xd = get(1);
        const float4 xy = in ? load4(static_cast<const T*>(p.dy) + out_at) : none;
        row4(sm.V, xv);
        row4(sm.dY, xy);
        row4(sm.W, in ? make_float4(decay_m1(xd.x), decay_m1(xd.y), decay_m1(xd.z), decay_m1(xd.w)) : none);
        __syncthreads();
        if (tid < kHead) {                               // W_t
            float w = 1.f;
#pragma unroll
            for (int t = 0; t < C; ++t) {
                w = fmaf(w, sm.W[t][tid], w);
                sm.W[t][tid] = w;
            }
        }
        __syncthreads();
        const float4 w = ld4(&sm.W[et][ec]);
        const float4 wp = et ? ld4(&sm.W[et - 1][ec]) : make_float4(1.f, 1.f, 1.f, 1.f);
        const float4 iw = make_float4(1.f / w.x, 1.f / w.y, 1.f / w.z, 1.f / w.w);
        row4(sm.R, mul(xr, w));
        row4(sm.A, mul(xa, wp));
        row4(sm.B, mul(xb, iw));
        row4(sm.K, mul(xk, iw));
        cp_wait();
        for (int i = tid; i < kHead * kHead / 4; i += THREADS) {             // (what this thread has brought)
            const int r = i >> 4, c = (i & 15) * 4;
            float4* g = reinterpret_cast<float4*>(&sm.G[r][c]);
            *g = mul(*g, ld4(&sm.W[C - 1][c]));
        }
    }
    __syncthreads();

    // ---- the 16 x 16 products that need no solution; two warps begin dR, one takes S0's part of Z
    const int warp = tid >> 5, lane = tid & 31, pair = warp >> 1;
    const Lane l = {lane >> 2, lane & 3, 32 * (warp & 1)};
    Half acc;
    acc.clear();
    if (warp == 0) square(sm.ab, l, sm.A, sm.B, true);
    else if (warp == 1) square(sm.ak, l, sm.A, sm.K, true);
    else if (warp == 2) square(sm.rb, l, sm.R, sm.B, false);
    else if (warp == 3) square(sm.rk, l, sm.R, sm.K, false);
    else if (warp == 4) square(sm.yv, l, sm.dY, sm.V, false);
    else if (warp >= 6) times<kHead, false>(acc, l, sm.dY, sm.S0);
    else {
        float z0 = 0.f, z1 = 0.f;
#pragma unroll 4
        for (int i = 0; i < kHead; ++i) {
            z0 = fmaf(sm.S0[i][lane], sm.G[i][lane], z0);
            z1 = fmaf(sm.S0[i][32 + lane], sm.G[i][32 + lane], z1);
        }
        sm.z[0][lane] = z0;
        sm.z[0][32 + lane] = z1;
    }
    __syncthreads();

    // ---- right-hand sides; each pair of warps takes one [16, 64] result, the last begins dK beside dR
    Half more;
    more.clear();
    if (pair == 0) {
        times_rows(acc, l, sm.A, sm.S0);
        times<C, false>(acc, l, sm.ak, sm.V);
        put(acc, l, sm.U);
    } else if (pair == 1) {
        times_rows(acc, l, sm.B, sm.G);
        times<C, true>(acc, l, sm.rb, sm.dY);
        put(acc, l, sm.E);
    } else if (pair == 2) {
        times_rows(acc, l, sm.K, sm.G);
        times<C, true>(acc, l, sm.rk, sm.dY);
    } else {
        times<C, false>(acc, l, sm.yv, sm.K);            // dR: all but its part with U
        acc.fold();
        times<kHead, false>(more, l, sm.V, sm.G);
        weigh(more, l, sm.K, sm.z[2]);
        more.fold();
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

    // ---- the parts that need no more 16 x 16 products, and those products
    if (pair < 2) acc.clear();
    if (pair == 0) times<kHead, false>(acc, l, sm.E, sm.S0);             // dA
    else if (pair == 1) {                                                // dB
        times<kHead, false>(acc, l, sm.U, sm.G);
        weigh(acc, l, sm.B, sm.z[1]);
    } else if (warp == 4) square(sm.yu, l, sm.dY, sm.U, false);
    else if (warp == 5) square(sm.eu, l, sm.E, sm.U, true);
    else if (warp == 6) square(sm.ev, l, sm.E, sm.V, true);
    if (pair == 2) {                                                     // dV
        times<C, true>(acc, l, sm.ak, sm.E);
        acc.fold();
    }
    __syncthreads();
    if (pair == 0) {
        times<C, false>(acc, l, sm.eu, sm.B);
        times<C, false>(acc, l, sm.ev, sm.K);
    } else if (pair == 1) {
        times<C, true>(acc, l, sm.yu, sm.R);
        times<C, true>(acc, l, sm.eu, sm.A);
    } else if (pair == 3) {
        times<C, false>(acc, l, sm.yu, sm.B);
        times<C, true>(more, l, sm.yv, sm.R);
        times<C, true>(more, l, sm.ev, sm.A);
    }
    __syncthreads();                                     // S0 and G are free from here
    float (*dA)[LD] = &sm.S0[0], (*dB)[LD] = &sm.S0[16], (*dV)[LD] = &sm.S0[32], (*dR)[LD] = &sm.S0[48];
    float (*dK)[LD] = &sm.G[0], (*dl)[LD] = &sm.G[16];
    put(acc, l, pair == 0 ? dA : pair == 1 ? dB : pair == 2 ? dV : dR);
    if (pair == 3) put(more, l, dK);
    __syncthreads();

    // ---- out, and what each token adds to the decay's gradient
    {
        const float4 w = ld4(&sm.W[et][ec]);
        const float4 wp = et ? ld4(&sm.W[et - 1][ec]) : make_float4(1.f, 1.f, 1.f, 1.f);
        const float4 iw = make_float4(1.f / w.x, 1.f / w.y, 1.f / w.z, 1.f / w.w);
        const float4 gr = ld4(&dR[et][ec]), gk = ld4(&dK[et][ec]), gb = ld4(&dB[et][ec]);
        float4 d = mul(ld4(&sm.R[et][ec]), gr);
        const float4 dk = mul(ld4(&sm.K[et][ec]), gk), db = mul(ld4(&sm.B[et][ec]), gb);
        d = make_float4(d.x - dk.x - db.x, d.y - dk.y - db.y, d.z - dk.z - db.z, d.w - dk.w - db.w);
        if (et + 1 < C) {
            const float4 n = mul(ld4(&sm.A[et + 1][ec]), ld4(&dA[et + 1][ec]));
            d = make_float4(d.x + n.x, d.y + n.y, d.z + n.z, d.w + n.w);
        }
        row4(dl, d);
        if (in) {
            const auto out = [&](int i, float4 v) { store4(static_cast<T*>(p.out[i]) + out_at, v); };
            out(0, mul(gr, w));
            out(2, mul(gk, iw));
            out(3, ld4(&dV[et][ec]));
            out(4, mul(ld4(&dA[et][ec]), wp));
            out(5, mul(gb, iw));
        }
    }
    __syncthreads();
    if (tid < kHead) {
        float sum = sm.z[0][tid] + sm.z[1][tid] + sm.z[2][tid];
#pragma unroll
        for (int t = C - 1; t >= 0; --t) {
            sum += dl[t][tid];
            dl[t][tid] = sum;
        }
    }
    __syncthreads();
    if (in) {
        const float4 g = ld4(&dl[et][ec]);
        const auto dd = [](float dlogw, float d) { return dlogw * (-kDecay * decay_gate_slope(d)); };
        store4(static_cast<T*>(p.out[1]) + out_at, make_float4(dd(g.x, xd.x), dd(g.y, xd.y), dd(g.z, xd.z), dd(g.w, xd.w)));
    }
}

template <typename T>
cudaError_t launch(const TmixArgs& a, cudaStream_t s) {
    static_assert(sizeof(Smem) <= 113 * 1024, "two CTAs per SM");
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
