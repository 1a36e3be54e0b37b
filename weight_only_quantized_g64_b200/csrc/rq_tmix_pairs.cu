// rq_tmix_pairs.cu -- the time-mix recurrence over sequences for few heads: pairs
// of tokens in plain fp32 arithmetic.
//
// The rows of the state are spread over lanes and stay in registers for the
// whole sequence: eight lanes share a row (8 keys each), eight CTAs a head (with
// four, and two rows per lane, 12 heads of 1024 tokens took 123 us for 101).
// Tokens are taken in pairs, so that one reduction over the eight lanes serves
// two:
//   x1 = S a1,  x2 = S (w1 a2),  z1 = S (w1 r1)
//   u1 = x1,  u2 = x2 + u1 (b1.a2) + v1 (k1.a2),  y1 = z1 + u1 (b1.r1) + v1 (k1.r1)
//   S <- S diag(w1 w2) + u1 (w2 b1)^T + v1 (w2 k1)^T + u2 b2^T + v2 k2^T,  y2 = S r2
// which is also 9 multiplications per element of S instead of 10.  Four producer
// warps load the next 16 tokens and form these vectors (the decay costs an
// exponential and a reciprocal per channel) while the others take the current
// ones (12 heads of 1024 fp32 tokens, forwards + backwards: 104 + 83 us; with two
// producer warps 109 + 92, fp16 101 + 80 where four take 103 + 81).
// What bounds it: the chain of a pair (two dot products, four shuffles, one
// update: 360 cycles with one row per lane, 390 beside the producers), and with
// many rows on an SM the reads of each pair's nine vectors from shared memory.
// rq_tmix.cu says where it is left for the kernel on the tensor cores.
//
// The backward direction is the same walk with other roles: with G the
// gradient of the state, for t descending G <- G + dy_t r_t^T, then
// G <- G diag(w_t) + (G b_t) a_t^T; for a pair
//   g2 = G b2 + dy2 (r2.b2)
//   g1 = G (w2 b1) + dy2 (w2 r2 . b1) + g2 (a2.b1) + dy1 (r1.b1)
//   G <- G diag(w1 w2) + dy2 (w1 w2 r2)^T + g2 (w1 a2)^T + dy1 (w1 r1)^T + g1 a1^T
// and G is stored behind each chunk of kTmixChunk tokens.
#include <type_traits>

#include "rq_tmix.cuh"

namespace rq {
namespace {

constexpr int UNROLL = 4;                    // pairs
constexpr int NCW = 2;                       // row warps of a CTA
constexpr int ROWS = NCW * 4;                // of a CTA: a head is spread over eight
constexpr int CT = kTmixChunk;               // tokens staged at once
constexpr int NPW = 4;                       // producer warps: a pair of tokens and 4 channels per thread
static_assert(NPW * 32 == CT / 2 * kHead / 4);
// staged vectors of a pair.  Forward: w1 w2 - 1, a1, w1 a2, w1 r1, w2 b1, w2 k1, b2, k2, r2; backward: w1 w2 - 1, b2,
// w2 b1, w1 w2 r2, w1 a2, w1 r1, a1
constexpr int nvec(bool rev) { return rev ? 7 : 9; }

template <bool REV>
struct Stage {
    float vec[nvec(REV)][CT / 2][kHead];
    float row[CT][ROWS];                     // v, or dy
    float4 dots[CT / 2];                     // b1.a2, k1.a2, b1.r1, k1.r1; backward r2.b2, w2 r2.b1, a2.b1, r1.b1
};
template <bool REV>
struct Smem {
    Stage<REV> st[2];
    float y[REV ? 1 : 2][REV ? 1 : CT][ROWS];
};

// The producers' part of a chunk: tokens [t0, t0 + nt) of head h, from global
// memory into registers (4 channels of two neighbouring tokens per thread) ...
template <typename T>
struct Raw4 {
    std::conditional_t<sizeof(T) == 4, uint4, uint2> u;
};
template <typename T>
__device__ __forceinline__ void cvt4(const Raw4<T>& r, float* f) {
    if constexpr (sizeof(T) == 4) {
        const float4 v = *reinterpret_cast<const float4*>(&r.u);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    } else {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&r.u.x));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&r.u.y));
        f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
    }
}
template <typename T>
struct Raw {
    Raw4<T> in[2][5];                        // r, d, k, a, b (k forward only)
    Raw8 row[(CT * ROWS / 8 + NPW * 32 - 1) / (NPW * 32)];
};
template <typename T, bool REV>
__device__ __forceinline__ void load_chunk(const TmixArgs& p, Raw<T>& raw, int64_t t0, int nt, int h, int row0,
                                           int pt) {
    const int64_t head = static_cast<int64_t>(h) * kHead;
    const int c = (pt & 15) * 4;
    const auto get = [](const void* from, int64_t at) {
        return Raw4<T>{__ldg(reinterpret_cast<const decltype(Raw4<T>::u)*>(static_cast<const T*>(from) + at))};
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * (pt >> 4) + i;
        if (t >= nt) continue;
        const int64_t at = (t0 + t) * p.ld + head + c;
        raw.in[i][0] = get(p.in[0], at);
        raw.in[i][1] = get(p.in[1], at);
        if (!REV) raw.in[i][2] = get(p.in[2], at);
        raw.in[i][3] = get(p.in[4], at);
        raw.in[i][4] = get(p.in[5], at);
    }
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(raw.row) / sizeof(Raw8)); ++i) {
        const int piece = pt + i * NPW * 32, t = piece / (ROWS / 8), rc = (piece % (ROWS / 8)) * 8;
        if (t >= nt) continue;
        const T* rows = REV ? static_cast<const T*>(p.dy) + (t0 + t) * p.H * kHead
                            : static_cast<const T*>(p.in[3]) + (t0 + t) * p.ld;
        raw.row[i] = load8(rows + head + row0 + rc);
    }
}
// ... and from there, as the vectors of the pairs, into a stage.  A token behind the last of the sequence is one that
// changes nothing: zeros, and a decay of 1.
template <typename T, bool REV>
__device__ __forceinline__ void stage_chunk(Stage<REV>& st, const Raw<T>& raw, int nt, int pt) {
    const int pair = pt >> 4, c = (pt & 15) * 4;
    if (2 * pair < nt) {                     // whole groups of 16 threads
        float r[2][4], w[2][4], k[2][4], a[2][4], b[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool in = 2 * pair + i < nt;
            cvt4<T>(raw.in[i][0], r[i]);
            cvt4<T>(raw.in[i][1], w[i]);
            cvt4<T>(raw.in[i][3], a[i]);
            cvt4<T>(raw.in[i][4], b[i]);
            if (!REV) cvt4<T>(raw.in[i][2], k[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[i][j] = in ? decay_m1(w[i][j]) : 0.f;
                if (i == 1 && !in) r[i][j] = a[i][j] = b[i][j] = k[i][j] = 0.f;
            }
        }
        float f[nvec(REV)][4];
        float4 dots = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // x (1 + m): one rounding
            const float m1 = w[0][j], m2 = w[1][j];
            f[0][j] = fmaf(m1, m2, m1 + m2);
            const float wr1 = fmaf(r[0][j], m1, r[0][j]), wa2 = fmaf(a[1][j], m1, a[1][j]);
            const float wb1 = fmaf(b[0][j], m2, b[0][j]);
            if constexpr (!REV) {
                f[1][j] = a[0][j];
                f[2][j] = wa2;
                f[3][j] = wr1;
                f[4][j] = wb1;
                f[5][j] = fmaf(k[0][j], m2, k[0][j]);
                f[6][j] = b[1][j];
                f[7][j] = k[1][j];
                f[8][j] = r[1][j];
                dots.x = fmaf(b[0][j], a[1][j], dots.x);
                dots.y = fmaf(k[0][j], a[1][j], dots.y);
                dots.z = fmaf(b[0][j], r[0][j], dots.z);
                dots.w = fmaf(k[0][j], r[0][j], dots.w);
            } else {
                const float wr2 = fmaf(r[1][j], m2, r[1][j]);
                f[1][j] = b[1][j];
                f[2][j] = wb1;
                f[3][j] = fmaf(wr2, m1, wr2);
                f[4][j] = wa2;
                f[5][j] = wr1;
                f[6][j] = a[0][j];
                dots.x = fmaf(r[1][j], b[1][j], dots.x);
                dots.y = fmaf(wr2, b[0][j], dots.y);
                dots.z = fmaf(a[1][j], b[0][j], dots.z);
                dots.w = fmaf(r[0][j], b[0][j], dots.w);
            }
        }
#pragma unroll
        for (int v = 0; v < nvec(REV); ++v) {
            *reinterpret_cast<float4*>(&st.vec[v][pair][c]) = make_float4(f[v][0], f[v][1], f[v][2], f[v][3]);
        }
        const uint32_t mates = 0xffffu << (threadIdx.x & 16);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            dots.x += __shfl_xor_sync(mates, dots.x, o);
            dots.y += __shfl_xor_sync(mates, dots.y, o);
            dots.z += __shfl_xor_sync(mates, dots.z, o);
            dots.w += __shfl_xor_sync(mates, dots.w, o);
        }
        if ((pt & 15) == 0) st.dots[pair] = dots;
    }
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(raw.row) / sizeof(Raw8)); ++i) {
        const int piece = pt + i * NPW * 32, t = piece / (ROWS / 8), rc = (piece % (ROWS / 8)) * 8;
        if (t >= CT || t >= ((nt + 1) & ~1)) continue;
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (t < nt) cvt8<T>(raw.row[i], f);
        float4* to = reinterpret_cast<float4*>(&st.row[t][rc]);
        to[0] = make_float4(f[0], f[1], f[2], f[3]);
        to[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// Sums of two values over eight lanes: lanes 0 .. 3 keep the first (in v[0]), 4 .. 7
// the second.  Two sets at a time, so that the shuffles of one pass while those of
// the other are on their way.
template <bool TWO>
__device__ __forceinline__ void sum_lanes(float (&v)[2], float (&o)[2], int lane) {
    const bool upper = lane & 4;
    float give = upper ? v[0] : v[1], give2 = upper ? o[0] : o[1];
    v[0] = upper ? v[1] : v[0];
    if (TWO) o[0] = upper ? o[1] : o[0];
#pragma unroll
    for (int mask = 4; mask >= 1; mask /= 2) {
        if (mask < 4) give = v[0], give2 = o[0];
        give = __shfl_xor_sync(0xffffffffu, give, mask);
        if (TWO) give2 = __shfl_xor_sync(0xffffffffu, give2, mask);
        v[0] += give;
        if (TWO) o[0] += give2;
    }
}

template <typename T>
__device__ __forceinline__ void store_y(const TmixArgs& p, const float (*y)[ROWS], int64_t t0, int nt, int h,
                                        int row0, int pt) {
    T* out = static_cast<T*>(p.out[0]);
    for (int piece = pt; piece < nt * (ROWS / 4); piece += NPW * 32) {
        const int t = piece / (ROWS / 4), c = (piece % (ROWS / 4)) * 4;
        store4(out + ((t0 + t) * p.H + h) * kHead + row0 + c, *reinterpret_cast<const float4*>(&y[t][c]));
    }
}

// One CTA: NCW compute warps of 4 rows each, of one head of one sequence.
template <typename T, bool REV>
__global__ void __launch_bounds__((NCW + NPW) * 32) tmix_pairs_kernel(const TmixArgs p) {
    constexpr int SPLIT = kHead / ROWS;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem<REV>& sm = *reinterpret_cast<Smem<REV>*>(smem_raw);

    const int part = blockIdx.x % SPLIT;
    const int h = (blockIdx.x / SPLIT) % p.H;
    const int seq = blockIdx.x / SPLIT / p.H;
    const int row0 = part * ROWS;
    int lo, hi;
    if (!sequence_of(p, seq, lo, hi)) return;
    const int64_t slot = state_of(p, seq);
    const int nchunk = (hi - lo + CT - 1) / CT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const auto chunk_of = [&](int c) { return REV ? nchunk - 1 - c : c; };
    const auto tokens_in = [&](int c) { return min(CT, hi - lo - c * CT); };

    if (warp >= NCW) {                       // producers
        // a chunk's loads are issued one chunk ahead of its conversion
        const int pt = threadIdx.x - NCW * 32;
        Raw<T> raw;
        const auto load = [&](int c) {
            if (c < nchunk)
                load_chunk<T, REV>(p, raw, lo + static_cast<int64_t>(chunk_of(c)) * CT, tokens_in(chunk_of(c)),
                                         h, row0, pt);
        };
        const auto stage = [&](int c) {
            if (c < nchunk) stage_chunk<T, REV>(sm.st[c & 1], raw, tokens_in(chunk_of(c)), pt);
        };
        load(0);
        stage(0);
        load(1);
        __syncthreads();
        for (int c = 0; c < nchunk; ++c) {
            stage(c + 1);
            load(c + 2);
            if constexpr (!REV) {
                if (c > 0) store_y<T>(p, sm.y[(c - 1) & 1], lo + static_cast<int64_t>(c - 1) * CT, CT, h,
                                            row0, pt);
            }
            __syncthreads();
        }
        if constexpr (!REV) {
            if (nchunk > 0) store_y<T>(p, sm.y[(nchunk - 1) & 1], lo + static_cast<int64_t>(nchunk - 1) * CT,
                                             tokens_in(nchunk - 1), h, row0, pt);
        }
        return;
    }

    // compute warps: lane (g, q) holds keys 4 q + 0..3 and 32 + 4 q + 0..3 of row wrow
    const int q = lane & 7, wrow = warp * 4 + (lane >> 3);
    uint64_t S[4];
    const int64_t head_state = (slot * p.H + h) * kHead * kHead;
    const int64_t mine = static_cast<int64_t>(row0 + wrow) * kHead + 4 * q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.state_in != nullptr && slot >= 0)
            f = *reinterpret_cast<const float4*>(p.state_in + head_state + mine + 32 * i);
        S[2 * i] = pack2(f.x, f.y);
        S[2 * i + 1] = pack2(f.z, f.w);
    }
    float* const ck = REV ? p.gckpt : p.ckpt;
    const auto store_state = [&](float* dst) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 a = unpack2(S[2 * i]), b = unpack2(S[2 * i + 1]);
            *reinterpret_cast<float4*>(dst + mine + 32 * i) = make_float4(a.x, a.y, b.x, b.y);
        }
    };
    struct Keys {
        uint64_t v[4];
    };
    __syncthreads();
    for (int c = 0; c < nchunk; ++c) {
        const int ch = chunk_of(c), nt = tokens_in(ch), pairs = (nt + 1) / 2;
        if (ck != nullptr) store_state(ck + ((ckpt_base(lo, seq) + ch) * p.H + h) * kHead * kHead);
        const Stage<REV>& st = sm.st[c & 1];
        // y of a pair is summed over the lanes while the next pair's products are on their way
        float last[2] = {};
        const auto write_y = [&](int pair) {             // last[0]: this lane's sum
            const float out = last[0];
            // (as assembly: the compiler would let no load of the next pair pass a store to shared memory)
            const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&sm.y[c & 1][2 * pair + q / 4][wrow]));
            if (q % 4 == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(out));
        };
#pragma unroll UNROLL
        for (int n = 0; n < pairs; ++n) {
            const int pair = REV ? pairs - 1 - n : n;
            const auto vec = [&](int v) {
                const float* f = &st.vec[v][pair][4 * q];
                const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(f), y = *reinterpret_cast<const ulonglong2*>(f + 32);
                return Keys{{x.x, x.y, y.x, y.y}};
            };
            const auto dot = [&](const Keys& k) {
                const float2 f = unpack2(add2(fma2(S[2], k.v[2], mul2(S[0], k.v[0])), fma2(S[3], k.v[3], mul2(S[1], k.v[1]))));
                return f.x + f.y;
            };
            const auto add = [&](const Keys& k, float f) {
                const uint64_t ff = pack2(f, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) S[i] = fma2(ff, k.v[i], S[i]);
            };
            const float row1 = st.row[2 * pair][wrow], row2 = st.row[2 * pair + 1][wrow];
            const float4 dots = st.dots[pair];
            // the two dot products of the update, summed over the lanes and back in all of them
            float x[2] = {dot(vec(1)), dot(vec(2))}, y = 0.f;
            if constexpr (!REV) y = dot(vec(3));
            sum_lanes<!REV>(x, last, lane);
            float u1 = __shfl_sync(0xffffffffu, x[0], 0, 8), u2 = __shfl_sync(0xffffffffu, x[0], 4, 8);
            if (!REV && n > 0) write_y(pair - 1);
            {
                const Keys w = vec(0);
#pragma unroll
                for (int i = 0; i < 4; ++i) S[i] = fma2(S[i], w.v[i], S[i]);
            }
            if constexpr (!REV) {
                add(vec(5), row1);
                add(vec(7), row2);
                u2 = fmaf(row1, dots.y, fmaf(u1, dots.x, u2));
                // once for the row: the sum over the lanes follows
                last[0] = q == 0 ? fmaf(row1, dots.w, fmaf(u1, dots.z, y)) : y;
                add(vec(4), u1);
                add(vec(6), u2);
                last[1] = dot(vec(8));
            } else {
                add(vec(3), row2);
                add(vec(5), row1);
                // x: G b2 and G (w2 b1)
                u1 = fmaf(row2, dots.x, u1);
                u2 = fmaf(row1, dots.w, fmaf(u1, dots.z, fmaf(row2, dots.y, u2)));
                add(vec(4), u1);
                add(vec(6), u2);
            }
        }
        if constexpr (!REV) {
            sum_lanes<false>(last, last, lane);
            write_y(pairs - 1);
        }
        __syncthreads();
    }
    if (p.state_out != nullptr && slot >= 0) store_state(p.state_out + head_state);
}

template <typename T, bool REV>
cudaError_t launch_scan(const TmixArgs& a, cudaStream_t s) {
    constexpr size_t smem = sizeof(Smem<REV>);
    const cudaError_t e = allow_smem<tmix_pairs_kernel<T, REV>>(smem);
    if (e != cudaSuccess) return e;
    tmix_pairs_kernel<T, REV><<<a.S * a.H * (kHead / ROWS), (NCW + NPW) * 32, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tmix_pairs(const TmixArgs& a, bool half, bool reverse, cudaStream_t s) {
    if (half) return reverse ? launch_scan<__half, true>(a, s) : launch_scan<__half, false>(a, s);
    return reverse ? launch_scan<float, true>(a, s) : launch_scan<float, false>(a, s);
}

}  // namespace rq
