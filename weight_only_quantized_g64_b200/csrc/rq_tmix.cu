// rq_tmix.cu -- the time-mix recurrence over sequences (and, run backwards,
// the gradient of its state) and over single tokens.
//
// Sequences, forwards.  Tokens are taken in chunks of C = 16.  With the decay
// divided out inside a chunk (W_t = prod_{s <= t} w_s; R_t = W_t r_t, A_t =
// W_{t-1} a_t, B_t = b_t / W_t, K_t = k_t / W_t as rows of 16 x 64 matrices; w >
// 0.545, so 1 / W <= 1.7e4), L keeping t >= s and M keeping t > s of a 16 x 16
// matrix, and T = (1 - M(A B^T))^-1, the chunk maps the state S before it to
//   Y = R' S^T + M' V,     S <- (S + (S A'^T) B + V^T K') diag(W_last)
//   A' = T A,  R' = R + L(R B^T) A',  N = T M(A K^T),
//   K' = K + N^T B,  M' = L(R K^T) + L(R B^T) N:
// matrix products only, and the rows of S still do not meet.  Four warps hold 16
// rows of S each, in the registers of the tensor cores' accumulators, which are
// also their first operand once the summed index is taken in the order 2q, 2q+1
// instead of q, q+4.  Two groups of four warps prepare A', R', B, K', M' of the
// chunks ahead in turn (with the same products): one chunk's preparation is a
// chain of small dependent steps, longer than its use (8192 tokens of 64 heads, the
// longest sequence 58 % of them: one group 1.09 ms, two 0.80, three 1.01, which
// leave less to the row warps).
//
// About 204 + 87 MMAs per warp and chunk (rq_tf32.cuh), 8 cycles each, bound the
// kernel from below: 2300 cycles a chunk.  It takes 5000 (64 heads of 1024 tokens:
// the row warps by themselves 104 us, the preparing warps by themselves 137,
// together 176): both sides are chains of dependent products and share the issue
// slots.  (Two CTAs per head that prepare for one another through distributed
// shared memory: 4500 cycles with four preparing groups, and more where other heads
// wait for an SM.)  Plain fp32 FMAs over pairs of tokens (rq_tmix_pairs.cu, which
// takes few heads) spend their time on shuffles and on reading each token's
// vectors for every row: 1.12 ms for 0.80.
//
// The products see every token of a chunk at once, so a value that is not finite
// would reach earlier tokens through a factor of 0.  A chunk with one in r, d, k,
// a or b, which reach every row, is therefore taken token by token, as the
// formula is written; one in v leaves the products, and makes its row NaN from
// its token on.
//
// Backwards: with G the gradient of the state behind a chunk, times W_last,
//   G <- G + (G B'^T) A + dY^T R',   B' = T^T B,
// and G is stored behind each chunk.
#include "rq_tf32.cuh"
#include "rq_tmix.cuh"

namespace rq {
namespace {

constexpr int C = kTmixChunk;
constexpr int LA = kHead + 8;                // rows read 8 bytes at a time along the keys: 8 banks apart
constexpr int LB = kHead + 4;                // rows read in pairs of tokens: 2 rows 8 banks apart
constexpr int LS = C + 8;
constexpr int GROUPS = 2, BUFFERS = 2;       // preparing groups, and chunks that each may have ready
static_assert(C == 16 && kHead == 64);
// 16-byte accesses: every row, and so every array, is a multiple of 16 bytes
static_assert(LA % 4 == 0 && LB % 4 == 0 && LS % 4 == 0 && kHead % 8 == 0);

// What the row warps need of a chunk.  Forwards / backwards: A' / B', R' / -, B /
// A, K' / R', M' / -, v / dy.
template <typename T, bool REV>
struct alignas(16) Chunk {
    float a[C][LA];
    float r[REV ? 1 : C][LA];
    float b[C][LB], k[C][LB];
    float m[REV ? 1 : C][LS];
    // W of the last token as x + y, applied as S x + S y: (W - 1, 1) above 1/2, where S W = S + S (W - 1) keeps W's
    // distance from 1 (W itself, rounded to 24 bits, would carry the same error into the state in every chunk), and
    // (W, 0) below, where W - 1 would lose W's own bits
    float last[2][kHead];
    T v[C][kHead + 8];
    int bad;                                 // a value of the chunk is not finite
};
template <typename T, bool REV>
struct alignas(16) Group {
    Chunk<T, REV> ch[BUFFERS];
    float x[C][LA], R[C][LA];                // the chunk in preparation: A / B, R
    float y[REV ? C : 1][LB];                // - / A'
    float abt[C][LS], rb[C][LS], t[C][LS];   // M(A B^T) transposed, L(R B^T), T
    // log2 W of the warps' own tokens.  Memory of its own: it is written before the group first meets in a chunk, when
    // a slower warp may still read any of the above for the chunk before
    float parts[4][kHead];
    float ak[REV ? 1 : C][LS], rk[REV ? 1 : C][LS], n[REV ? 1 : C][LS];
};
template <typename T, bool REV>
struct alignas(16) Smem {
    Group<T, REV> group[GROUPS];
    float y[REV ? 1 : 4][C][C + 4];          // of each row warp
};

// Named barriers: 1 + group: its own steps; then for each group and buffer one
// that says "ready" and one that says "free".  Each is used by 128 threads that
// arrive and 128 that wait, once a turn.
__device__ __forceinline__ void group_sync(int group) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory");
}
__device__ __forceinline__ bool group_any(int group, bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(p ? 1u : 0u), "r"(1 + group)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ int ready_id(int c) { return 1 + GROUPS + (c % GROUPS) * BUFFERS + c / GROUPS % BUFFERS; }
__device__ __forceinline__ int free_id(int c) { return ready_id(c) + GROUPS * BUFFERS; }
static_assert(1 + GROUPS + 2 * GROUPS * BUFFERS <= 16);
__device__ __forceinline__ void arrive_at(int id) { asm volatile("barrier.cta.arrive %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void wait_at(int id) { asm volatile("barrier.cta.sync %0, 256;" ::"r"(id) : "memory"); }

// ---------------------------------------------------- the preparing warps --
// Thread: 8 channels of one token, the tokens 4 w .. 4 w + 3 in warp w.
struct Raw {
    Raw8 in[6];                              // r, d, k, v (or dy), a, b
};
template <typename T, bool REV>
__device__ __forceinline__ void load_chunk(const TmixArgs& p, Raw& raw, int64_t t0, int nt, int h, int pt) {
    const int t = pt >> 3;
    if (t >= nt) return;
    const int64_t head = static_cast<int64_t>(h) * kHead + (pt & 7) * 8, at = (t0 + t) * p.ld + head;
#pragma unroll
    for (int v = 0; v < 6; ++v) {
        if (REV && v == 2) continue;
        if (REV && v == 3) raw.in[v] = load8(static_cast<const T*>(p.dy) + (t0 + t) * p.H * kHead + head);
        else raw.in[v] = load8(static_cast<const T*>(p.in[v]) + at);
    }
}

template <typename T, bool REV, typename Next>
__device__ __forceinline__ void prepare(Group<T, REV>& sm, Chunk<T, REV>& ch, int group, const Raw& raw, int nt, int pt,
                                        Next&& next) {
    const int warp = pt >> 5, lane = pt & 31, g = lane >> 2, q = lane & 3;
    const int token = pt >> 3, k0 = (pt & 7) * 8;
    float r[8], w[8], k[8], a[8], b[8];
    bool bad = false;
    {
        // a token behind the last changes nothing: zeros, and a decay of 1
        const bool in = token < nt;
        const auto take = [&](int v, float* f) {
            if (in) {
                cvt8<T>(raw.in[v], f);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = 0.f;
            }
        };
        uint4* to = reinterpret_cast<uint4*>(&ch.v[token][k0]);
        to[0] = in ? raw.in[3].u[0] : make_uint4(0u, 0u, 0u, 0u);
        if constexpr (sizeof(T) == 4) to[1] = in ? raw.in[3].u[1] : make_uint4(0u, 0u, 0u, 0u);
        take(0, r);
        take(1, w);
        if (!REV) take(2, k);
        take(4, a);
        take(5, b);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum += (fabsf(r[j]) + fabsf(a[j])) + (fabsf(b[j]) + (REV ? 0.f : fabsf(k[j])));
            bad |= w[j] != w[j];
            w[j] = in ? log2_decay(w[j]) : 0.f;
        }
        bad |= !(sum < 1e30f);               // (and none so large that its product with 1 / W is not finite)
        next();                              // the inputs of the chunk after this one, into raw
    }
    if constexpr (!REV) {
        bad = group_any(group, bad);
        if (pt == 0) ch.bad = bad;
        if (bad) {                           // the inputs themselves, for the formula
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ch.a[token][k0 + j] = a[j];
                ch.r[token][k0 + j] = r[j];
                ch.b[token][k0 + j] = b[j];
                ch.k[token][k0 + j] = k[j];
            }
            return;
        }
    }
    const auto put8 = [](float* to, const float* f) {
        reinterpret_cast<float4*>(to)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(f[4], f[5], f[6], f[7]);
    };
    // log2 W: sums over the tokens, in the warp and then of the warps before
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float o = __shfl_up_sync(0xffffffffu, w[j], 8);
        w[j] += lane >= 8 ? o : 0.f;
        o = __shfl_up_sync(0xffffffffu, w[j], 16);
        w[j] += lane >= 16 ? o : 0.f;
    }
    if (lane >= 24) put8(&sm.parts[warp][k0], w);
    group_sync(group);
    float before[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) before[j] = 0.f;
    for (int i = 0; i < warp; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(&sm.parts[i][k0]), y = *reinterpret_cast<const float4*>(&sm.parts[i][k0 + 4]);
        before[0] += x.x; before[1] += x.y; before[2] += x.z; before[3] += x.w;
        before[4] += y.x; before[5] += y.y; before[6] += y.z; before[7] += y.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float up = __shfl_up_sync(0xffffffffu, w[j], 8);
        const float prev = exp2_approx(before[j] + (lane >= 8 ? up : 0.f));
        w[j] += before[j];
        const float W = exp2_approx(w[j]), back = exp2_approx(-w[j]);
        r[j] *= W;
        a[j] *= prev;
        b[j] *= back;
        if (!REV) k[j] *= back;
        if (token == C - 1) {
            ch.last[0][k0 + j] = w[j] > -1.f ? expm1_near(w[j] * kLn2) : W;
            ch.last[1][k0 + j] = w[j] > -1.f ? 1.f : 0.f;
        }
    }
    put8(&sm.R[token][k0], r);
    put8(REV ? &ch.b[token][k0] : &sm.x[token][k0], a);
    put8(REV ? &sm.x[token][k0] : &ch.b[token][k0], b);
    if (!REV) put8(&ch.k[token][k0], k);
    group_sync(group);

    // the 16 x 16 products, one per warp
    if (!REV || warp < 2) {
        const bool second = REV ? warp == 1 : warp >= 2;         // R, else A
        const float* x = second ? &sm.R[0][0] : REV ? &ch.b[0][0] : &sm.x[0][0];
        const int lx = second || !REV ? LA : LB;
        const float* z = REV ? &sm.x[0][0] : warp & 1 ? &ch.k[0][0] : &ch.b[0][0];
        const int lz = REV ? LA : LB;
        Sums<2> c;                           // two column halves
        c.clear();
#pragma unroll 2                             // (4: backward walks 4 % slower, for the instruction cache)
        for (int k = 0; k < kHead; k += 8) {
            const float* row = x + g * lx + k + 2 * q;
            const float2 u = *reinterpret_cast<const float2*>(row), v = *reinterpret_cast<const float2*>(row + 8 * lx);
            const float* col = z + g * lz + k + 2 * q;
            const float4 b[2] = {along(col), along(col + 8 * lz)};
            products(c, rows_of(u.x, u.y, v.x, v.y), b);
        }
        const int what = REV ? 2 * warp : warp;              // 0: A B^T, 1: A K^T, 2: R B^T, 3: R K^T
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = g + 8 * (j >> 1), s = 8 * n + 2 * q + (j & 1);
                const float v = t > s || (t == s && what >= 2) ? c.at(n, j) : 0.f;
                if (what == 0) sm.abt[s][t] = v;
                if (what == 2) sm.rb[t][s] = v;
                if constexpr (!REV) {
                    if (what == 1) sm.ak[t][s] = v;
                    if (what == 3) sm.rk[t][s] = v;
                }
            }
    }
    group_sync(group);

    // T (lanes 0..15: its columns) and N = T M(A K^T) (lanes 16..31), solved from the first row down
    if (warp == 0) {
        const int c = lane & 15;
        float x[C];
#pragma unroll
        for (int t = 0; t < C; ++t) {
            x[t] = t == c ? 1.f : 0.f;
            if constexpr (!REV) x[t] = lane < 16 ? x[t] : sm.ak[t][c];
        }
#pragma unroll
        for (int s = 0; s < C - 1; ++s) {
#pragma unroll
            for (int t4 = (s + 1) / 4 * 4; t4 < C; t4 += 4) {
                const float4 m = *reinterpret_cast<const float4*>(&sm.abt[s][t4]);
                x[t4] = fmaf(m.x, x[s], x[t4]);              // (zeros up to s: those are done)
                x[t4 + 1] = fmaf(m.y, x[s], x[t4 + 1]);
                x[t4 + 2] = fmaf(m.z, x[s], x[t4 + 2]);
                x[t4 + 3] = fmaf(m.w, x[s], x[t4 + 3]);
            }
        }
        if (lane < 16) {
#pragma unroll
            for (int t = 0; t < C; ++t) sm.t[t][c] = x[t];
        } else if constexpr (!REV) {
#pragma unroll
            for (int t = 0; t < C; ++t) sm.n[t][c] = x[t];
        }
    }
    group_sync(group);

    // 16 keys per warp, in two products of 8 columns
    const int kw = warp * 16;
    Sums<2> c;
    const auto put = [&](float* to, int ld) {
        c.fold();
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float* at = to + g * ld + kw + 8 * n + 2 * q;
            *reinterpret_cast<float2*>(at) = make_float2(c.c[n][0], c.c[n][1]);
            *reinterpret_cast<float2*>(at + 8 * ld) = make_float2(c.c[n][2], c.c[n][3]);
        }
    };
    const auto take = [&](const float* from, int ld) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float* at = from + g * ld + kw + 8 * n + 2 * q;
            const float2 x = *reinterpret_cast<const float2*>(at), y = *reinterpret_cast<const float2*>(at + 8 * ld);
            c.c[n][0] = x.x; c.c[n][1] = x.y; c.c[n][2] = y.x; c.c[n][3] = y.y;
        }
    };
    // c += m z, or with the columns of m, z the rows of 16 tokens
    const auto multiply = [&](const float (*m)[LS], bool columns, const float* z, int ld) {
#pragma unroll
        for (int s = 0; s < C; s += 8) {
            const float* at = z + (s + 2 * q) * ld + kw + g;
            const float4 b[2] = {down(at, ld), down(at + 8, ld)};
            products(c, columns ? columns_at(m, g, s + 2 * q) : rows_at(m, g, s + 2 * q), b);
        }
    };
    c.clear();
    if constexpr (!REV) {
        multiply(sm.t, false, &sm.x[0][0], LA);                  // A' = T A
        put(&ch.a[0][0], LA);
        take(&ch.k[0][0], LB);                                   // K' = K + N^T B
        multiply(sm.n, true, &ch.b[0][0], LB);
        put(&ch.k[0][0], LB);
        __syncwarp();
        take(&sm.R[0][0], LA);                                   // R' = R + L(R B^T) A'
        multiply(sm.rb, false, &ch.a[0][0], LA);
        put(&ch.r[0][0], LA);
        if (warp < 2) {                                          // M' = L(R K^T) + L(R B^T) N, 8 columns each
            Sums<1> e;
            e.clear();
            const float* at = &sm.rk[g][8 * warp + 2 * q];
            const float2 x = *reinterpret_cast<const float2*>(at), y = *reinterpret_cast<const float2*>(at + 8 * LS);
            e.c[0][0] = x.x; e.c[0][1] = x.y; e.c[0][2] = y.x; e.c[0][3] = y.y;
#pragma unroll
            for (int s = 0; s < C; s += 8) {
                const float4 b[1] = {down(&sm.n[s + 2 * q][8 * warp + g], LS)};
                products(e, rows_at(sm.rb, g, s + 2 * q), b);
            }
            *reinterpret_cast<float2*>(&ch.m[g][8 * warp + 2 * q]) = make_float2(e.at(0, 0), e.at(0, 1));
            *reinterpret_cast<float2*>(&ch.m[g + 8][8 * warp + 2 * q]) = make_float2(e.at(0, 2), e.at(0, 3));
        }
    } else {
        multiply(sm.t, false, &ch.b[0][0], LB);                  // A' = T A
        put(&sm.y[0][0], LB);
        c.clear();                                               // B' = T^T B
        multiply(sm.t, true, &sm.x[0][0], LA);
        put(&ch.a[0][0], LA);
        __syncwarp();
        take(&sm.R[0][0], LA);                                   // R' = R + L(R B^T) A'
        multiply(sm.rb, false, &sm.y[0][0], LB);
        put(&ch.k[0][0], LB);
    }
}

// --------------------------------------------------------- the row warps --
// S[n][j]: row g (j < 2) or g + 8, key 8 n + 2 q + j % 2
using State = float[8][4];

__device__ __forceinline__ void decay(State& S, const float (&last)[2][kHead], int q) {
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        const uint64_t x = *reinterpret_cast<const uint64_t*>(&last[0][8 * n + 2 * q]);
        const uint64_t y = *reinterpret_cast<const uint64_t*>(&last[1][8 * n + 2 * q]);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint64_t s = pack2(S[n][i], S[n][i + 1]);
            const float2 f = unpack2(fma2(s, x, mul2(s, y)));
            S[n][i] = f.x;
            S[n][i + 1] = f.y;
        }
    }
}

template <typename T>
__device__ __forceinline__ void forward_chunk(State& S, const Chunk<T, false>& ch, float (*y)[C + 4], int row, int lane) {
    const int g = lane >> 2, q = lane & 3;
    Sums<4> XY;                              // X, then Y
    int from[2] = {C, C};                    // first token of the row whose v is not finite
    XY.clear();
#pragma unroll
    for (int k = 0; k < 8; ++k) {            // X = S A'^T, Y = S R'^T
        const float4 b[4] = {along(&ch.a[g][8 * k + 2 * q]), along(&ch.a[8 + g][8 * k + 2 * q]),
                             along(&ch.r[g][8 * k + 2 * q]), along(&ch.r[8 + g][8 * k + 2 * q])};
        products(XY, rows_of(S[k][0], S[k][1], S[k][2], S[k][3]), b);
    }
    XY.fold();
    Sums<2> Y;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Y.c[n][j] = XY.c[n + 2][j];
            Y.small[n][j] = 0.f;
        }
    constexpr bool EXACT = sizeof(T) == 2;
    Rows x[2], v[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {            // Y += V^T M'^T
        x[s] = rows_of(XY.c[s][0], XY.c[s][1], XY.c[s][2], XY.c[s][3]);
        const T *v0 = &ch.v[8 * s + 2 * q][row + g], *v1 = v0 + kHead + 8;
        float vf[4] = {to_f32(v0[0]), to_f32(v1[0]), to_f32(v0[8]), to_f32(v1[8])};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (!(fabsf(vf[j]) < 1e30f)) {
                vf[j] = 0.f;
                from[j >> 1] = min(from[j >> 1], 8 * s + 2 * q + (j & 1));
            }
        v[s] = rows_of(vf[0], vf[1], vf[2], vf[3]);
        const float4 m[2] = {along(&ch.m[g][8 * s + 2 * q]), along(&ch.m[8 + g][8 * s + 2 * q])};
        products<EXACT>(Y, v[s], m);
    }
    Y.fold();
#pragma unroll
    for (int n = 0; n < 8; n += 4) {         // S += X B + V^T K'
        Sums<4> d;
        d.clear();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float4 b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = down(&ch.b[8 * s + 2 * q][8 * (n + i) + g], LB);
            products(d, x[s], b);
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = down(&ch.k[8 * s + 2 * q][8 * (n + i) + g], LB);
            products<EXACT>(d, v[s], b);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[n + i][j] += d.at(i, j);
    }
    decay(S, ch.last, q);
    if (__any_sync(0xffffffffu, min(from[0], from[1]) < C)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            from[i] = min(from[i], __shfl_xor_sync(0xffffffffu, from[i], 1));
            from[i] = min(from[i], __shfl_xor_sync(0xffffffffu, from[i], 2));
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (from[i] < C) S[n][2 * i + j] = NAN;
                    if (n < 2 && 8 * n + 2 * q + j >= from[i]) Y.c[n & 1][2 * i + j] = NAN;
                }
        }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) y[8 * n + 2 * q + (j & 1)][g + 8 * (j >> 1)] = Y.c[n][j];
}

// The formula as it is written, for chunks with values that are not finite.
template <typename T>
__device__ __forceinline__ void forward_tokens(State& S, const Chunk<T, false>& ch, const T* d, int64_t ld,
                                               float (*y)[C + 4], int row, int lane, int nt) {
    const int g = lane >> 2, q = lane & 3;
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
        const float *r = ch.r[t], *a = ch.a[t], *b = ch.b[t], *k = ch.k[t];
        float u[2] = {0.f, 0.f}, out[2] = {0.f, 0.f};
        const T* dt = d + t * ld;
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j >> 1] = fmaf(S[n][j], a[8 * n + 2 * q + (j & 1)], u[j >> 1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            u[i] += __shfl_xor_sync(0xffffffffu, u[i], 1);
            u[i] += __shfl_xor_sync(0xffffffffu, u[i], 2);
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float m[2] = {decay_m1(to_f32(dt[8 * n + 2 * q])), decay_m1(to_f32(dt[8 * n + 2 * q + 1]))};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = 8 * n + 2 * q + (j & 1), i = j >> 1;
                S[n][j] = fmaf(S[n][j], m[j & 1], S[n][j]);
                S[n][j] = fmaf(to_f32(ch.v[t][row + g + 8 * i]), k[key], S[n][j]);
                S[n][j] = fmaf(u[i], b[key], S[n][j]);
                out[i] = fmaf(S[n][j], r[key], out[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            out[i] += __shfl_xor_sync(0xffffffffu, out[i], 1);
            out[i] += __shfl_xor_sync(0xffffffffu, out[i], 2);
            if (q == 0) y[t][g + 8 * i] = out[i];
        }
    }
}

template <typename T>
__device__ __forceinline__ void backward_chunk(State& G, const Chunk<T, true>& ch, int row, int lane) {
    const int g = lane >> 2, q = lane & 3;
    decay(G, ch.last, q);
    Sums<2> X;
    X.clear();
#pragma unroll
    for (int k = 0; k < 8; ++k) {            // X = G B'^T
        const float4 b[2] = {along(&ch.a[g][8 * k + 2 * q]), along(&ch.a[8 + g][8 * k + 2 * q])};
        products(X, rows_of(G[k][0], G[k][1], G[k][2], G[k][3]), b);
    }
    X.fold();
    Rows x[2], v[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        x[s] = rows_of(X.c[s][0], X.c[s][1], X.c[s][2], X.c[s][3]);
        const T *v0 = &ch.v[8 * s + 2 * q][row + g], *v1 = v0 + kHead + 8;
        v[s] = rows_of(to_f32(v0[0]), to_f32(v1[0]), to_f32(v0[8]), to_f32(v1[8]));
    }
#pragma unroll
    for (int n = 0; n < 8; n += 4) {         // G += X A + dY^T R'
        Sums<4> d;
        d.clear();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float4 b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = down(&ch.b[8 * s + 2 * q][8 * (n + i) + g], LB);
            products(d, x[s], b);
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = down(&ch.k[8 * s + 2 * q][8 * (n + i) + g], LB);
            products<sizeof(T) == 2>(d, v[s], b);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) G[n + i][j] += d.at(i, j);
    }
}

// The sequence that is index-th in the order of lengths, the longest first: with
// more CTAs than SMs the last ones to start are then short (64 heads, sequences of
// 864, 864, 864, 864 and 4736 tokens: 1050 us in their own order, 770 in this).
// Of up to 32 sequences, whose lengths a warp holds; more are taken as they come.
__device__ __forceinline__ int by_length(const TmixArgs& p, int index) {
    if (p.S > 32) return index;
    const int lane = threadIdx.x & 31;
    const int64_t len = lane < p.S ? static_cast<int64_t>(p.seq_start[lane + 1]) - p.seq_start[lane] : 0;
    const int mine = static_cast<int>(max(int64_t{0}, min(len, p.T)));      // (whatever bad offsets give)
    int longer = 0;
    for (int i = 0; i < p.S; ++i) {
        const int other = __shfl_sync(0xffffffffu, mine, i);
        longer += other > mine || (other == mine && i < lane);
    }
    return __ffs(__ballot_sync(0xffffffffu, lane < p.S && longer == index)) - 1;
}

// One CTA: one head of one sequence; warps 0..3 hold its rows, the others prepare.
template <typename T, bool REV>
__global__ void __launch_bounds__(128 * (1 + GROUPS), 1) tmix_scan_kernel(const TmixArgs p) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem<T, REV>& sm = *reinterpret_cast<Smem<T, REV>*>(smem_raw);
    const int h = blockIdx.x % p.H, seq = by_length(p, blockIdx.x / p.H);
    int lo, hi;
    if (!sequence_of(p, seq, lo, hi)) return;
    const int64_t slot = state_of(p, seq);
    const int chunks = (hi - lo + C - 1) / C;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const auto chunk_of = [&](int c) { return REV ? chunks - 1 - c : c; };
    const auto start_of = [&](int c) { return lo + static_cast<int64_t>(chunk_of(c)) * C; };
    const auto tokens_in = [&](int c) { return min(C, hi - lo - chunk_of(c) * C); };

    if (warp >= 4) {
        const int group = (warp - 4) / 4, pt = threadIdx.x & 127;
        Group<T, REV>& mine = sm.group[group];
        Raw raw;
        const auto load = [&](int c) {
            if (c < chunks) load_chunk<T, REV>(p, raw, start_of(c), tokens_in(c), h, pt);
        };
        load(group);
        for (int c = group; c < chunks; c += GROUPS) {
            if (c >= GROUPS * BUFFERS) wait_at(free_id(c));
            prepare<T, REV>(mine, mine.ch[c / GROUPS % BUFFERS], group, raw, tokens_in(c), pt, [&] { load(c + GROUPS); });
            arrive_at(ready_id(c));
        }
        return;
    }

    const int g = lane >> 2, q = lane & 3, row = 16 * warp;
    const int64_t head_state = (slot * p.H + h) * kHead * kHead;
    const auto place = [&](int n, int i) { return (row + g + 8 * i) * kHead + 8 * n + 2 * q; };
    State S;
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float2 f = make_float2(0.f, 0.f);
            if (p.state_in != nullptr && slot >= 0) f = *reinterpret_cast<const float2*>(p.state_in + head_state + place(n, i));
            S[n][2 * i] = f.x;
            S[n][2 * i + 1] = f.y;
        }
    const auto store_state = [&](float* to) {
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<float2*>(to + place(n, i)) = make_float2(S[n][2 * i], S[n][2 * i + 1]);
    };
    float* const ck = REV ? p.gckpt : p.ckpt;
    for (int c = 0; c < chunks; ++c) {
        if (ck != nullptr) store_state(ck + ((ckpt_base(lo, seq) + chunk_of(c)) * p.H + h) * kHead * kHead);
        const Chunk<T, REV>& ch = sm.group[c % GROUPS].ch[c / GROUPS % BUFFERS];
        wait_at(ready_id(c));
        if constexpr (REV) {
            backward_chunk<T>(S, ch, row, lane);
        } else {
            if (ch.bad)
                forward_tokens<T>(S, ch, static_cast<const T*>(p.in[1]) + start_of(c) * p.ld + static_cast<int64_t>(h) * kHead,
                                  p.ld, sm.y[warp], row, lane, tokens_in(c));
            else forward_chunk<T>(S, ch, sm.y[warp], row, lane);
        }
        if (c + GROUPS * BUFFERS < chunks) arrive_at(free_id(c));        // (as often as it is waited for)
        if constexpr (!REV) {
            __syncwarp();
            const int t = lane >> 1, r = 8 * (lane & 1);
            if (t < tokens_in(c)) {
                T* to = static_cast<T*>(p.out[0]) + ((start_of(c) + t) * p.H + h) * kHead + row + r;
                store4(to, *reinterpret_cast<const float4*>(&sm.y[warp][t][r]));
                store4(to + 4, *reinterpret_cast<const float4*>(&sm.y[warp][t][r + 4]));
            }
            __syncwarp();
        }
    }
    if (p.state_out != nullptr && slot >= 0) store_state(p.state_out + head_state);
}

template <typename T, bool REV>
cudaError_t launch_scan(const TmixArgs& a, cudaStream_t s) {
    constexpr int smem = sizeof(Smem<T, REV>);
    static_assert(smem <= 227 * 1024);
    const cudaError_t e = allow_smem<tmix_scan_kernel<T, REV>>(smem);
    if (e != cudaSuccess) return e;
    tmix_scan_kernel<T, REV><<<a.S * a.H, 128 * (1 + GROUPS), smem, s>>>(a);
    return cudaGetLastError();
}

// ------------------------------------------------------------ single token --
// One CTA per head of one request; four lanes share a row, a lane holds two
// rows.  Bound by the state's bytes: 16 KB read and 16 KB written per head; 32
// requests of 64 heads 12.4 us, 5.6 TB/s.
template <typename T>
__global__ void __launch_bounds__(128) tmix_step_kernel(const TmixArgs p) {
    __shared__ __align__(16) float wm1[kHead];       // read as float4
    const int h = blockIdx.x % p.H, b = blockIdx.x / p.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 3;
    const int row = warp * 16 + (lane >> 2);         // and row + 8
    const int64_t slot = state_of(p, b);
    const int64_t head_state = (slot * p.H + h) * kHead * kHead;
    const int64_t at = static_cast<int64_t>(b) * p.ld + static_cast<int64_t>(h) * kHead;
    float4 S[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            S[r][i] = p.state_in != nullptr && slot >= 0
                          ? *reinterpret_cast<const float4*>(p.state_in + head_state + (row + 8 * r) * kHead +
                                                             16 * i + 4 * q)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float4 R[4], K[4], A[4], B[4];
    const T* const* in = reinterpret_cast<const T* const*>(p.in);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t o = at + 16 * i + 4 * q;
        A[i] = load4(in[4] + o);
        K[i] = load4(in[2] + o);
        B[i] = load4(in[5] + o);
        R[i] = load4(in[0] + o);
    }
    const float v[2] = {to_f32(in[3][at + row]), to_f32(in[3][at + row + 8])};
    if (threadIdx.x < kHead) wm1[threadIdx.x] = decay_m1(to_f32(in[1][at + threadIdx.x]));
    const auto dot4 = [](float4 a, float4 b, float c) {
        return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
    };
    float sa[2] = {0.f, 0.f}, y[2] = {0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sa[r] = dot4(S[r][i], A[i], sa[r]);
        sa[r] += __shfl_xor_sync(0xffffffffu, sa[r], 1);
        sa[r] += __shfl_xor_sync(0xffffffffu, sa[r], 2);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 w = *reinterpret_cast<const float4*>(&wm1[16 * i + 4 * q]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float4& s = S[r][i];
            s.x = fmaf(sa[r], B[i].x, fmaf(v[r], K[i].x, fmaf(s.x, w.x, s.x)));
            s.y = fmaf(sa[r], B[i].y, fmaf(v[r], K[i].y, fmaf(s.y, w.y, s.y)));
            s.z = fmaf(sa[r], B[i].z, fmaf(v[r], K[i].z, fmaf(s.z, w.z, s.z)));
            s.w = fmaf(sa[r], B[i].w, fmaf(v[r], K[i].w, fmaf(s.w, w.w, s.w)));
            y[r] = dot4(s, R[i], y[r]);
            if (p.state_out != nullptr && slot >= 0)
                *reinterpret_cast<float4*>(p.state_out + head_state + (row + 8 * r) * kHead + 16 * i + 4 * q) = s;
        }
    }
    T* out = static_cast<T*>(p.out[0]) + (static_cast<int64_t>(b) * p.H + h) * kHead;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        y[r] += __shfl_xor_sync(0xffffffffu, y[r], 1);
        y[r] += __shfl_xor_sync(0xffffffffu, y[r], 2);
        if (q == 0) out[row + 8 * r] = from_f32<T>(y[r]);
    }
}

}  // namespace

cudaError_t launch_tmix_scan(const TmixArgs& a, bool half, bool reverse, cudaStream_t s) {
    // Up to a head (of all sequences together, empty ones too: their lengths are on the
    // device) for every four SMs, most SMs would be without one of this kernel's CTAs,
    // and its first chunk takes 10 us; pairs of tokens split a head over eight CTAs.
    // Forwards and the gradients' call in us, one fp16 sequence, pairs / this kernel: 12
    // heads of 128 tokens 19, 30 / 30, 38, of 1024 104, 128 / 176, 190; 37 of 1024 141, 247
    // / 176, 262; 32 of 512 74, 112 / 93, 131; 40 of 512 101, 146 / 93, 145; 48 102, 159
    // / 93, 159; 64 144, 198 / 93, 179; 128 256, 380 / 93, 271.
    if (static_cast<int64_t>(a.S) * a.H * 4 <= num_sms()) return launch_tmix_pairs(a, half, reverse, s);
    if (half) return reverse ? launch_scan<__half, true>(a, s) : launch_scan<__half, false>(a, s);
    return reverse ? launch_scan<float, true>(a, s) : launch_scan<float, false>(a, s);
}

cudaError_t launch_tmix_step(const TmixArgs& a, bool half, cudaStream_t s) {
    if (half) tmix_step_kernel<__half><<<a.S * a.H, 128, 0, s>>>(a);
    else tmix_step_kernel<float><<<a.S * a.H, 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace rq
