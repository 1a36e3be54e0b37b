// rq_tmix.cu -- the time-mix recurrence over sequences (and, run backwards,
// the gradient of its state) and over single tokens.
//
// Sequences: every row of the 64 x 64 state is its own recurrence, so the
// rows are spread over lanes and stay in registers for the whole sequence:
// four lanes share a row (16 keys each), a lane holds RPL rows.  Per token a
// lane reads its 16 keys of five vectors from shared memory once for all its
// rows; the dot products finish with two shuffles.  Four producer warps load
// and convert the next chunk of tokens (the decay costs an exponential and a
// sigmoid per channel) while the others run through the current one.
// What bounds it: 5 * 64 * 64 fp32 FMA per token and head (packed in pairs),
// and for few heads the chain of one dot product and its shuffles per token.
//
// The backward direction is the same walk with other roles: with G the
// gradient of the state,
//   G <- G + dy_t r_t^T;   G <- G diag(w_t) + (G b_t) a_t^T      (t descending)
// and G is stored behind each chunk of kTmixChunk tokens.
#include "rq_tmix.cuh"

namespace rq {
namespace {

constexpr int CT = kTmixChunk;               // tokens staged at once
constexpr int NPW = 4;                       // producer warps: one piece of each vector per thread
static_assert(NPW * 32 == CT * kHead / 8);
// vectors staged per token: decay - 1, then forward k, a, b, r; backward r, b, a
constexpr int nvec(bool rev) { return rev ? 4 : 5; }

template <int ROWS, bool REV>
struct Stage {
    float vec[nvec(REV)][CT][kHead];
    float row[CT][ROWS];                     // v, or dy
};
template <int ROWS, bool REV>
struct Smem {
    Stage<ROWS, REV> st[2];
    float y[REV ? 1 : 2][REV ? 1 : CT][ROWS];
};

// The producers' part of a chunk: tokens [t0, t0 + nt) of head h, from global
// memory into registers (one piece of 8 elements of each vector per thread) ...
template <typename T, int ROWS, bool REV>
struct Raw {
    Raw8 vec[nvec(REV)], row;
};
template <typename T, int ROWS, bool REV>
__device__ __forceinline__ void load_chunk(const TmixArgs& p, Raw<T, ROWS, REV>& raw, int64_t t0, int nt, int h,
                                           int row0, int pt) {
    // in[]: r, d, k, v, a, b.  Order of the staged vectors (source indices):
    constexpr int src[5] = {1, REV ? 0 : 2, REV ? 5 : 4, REV ? 4 : 5, 0};
    const int t = pt >> 3, c = (pt & 7) * 8;
    const int64_t head = static_cast<int64_t>(h) * kHead;
    if (t < nt) {
#pragma unroll
        for (int v = 0; v < nvec(REV); ++v)
            raw.vec[v] = load8(static_cast<const T*>(p.in[src[v]]) + (t0 + t) * p.ld + head + c);
    }
    const int rt = pt / (ROWS / 8), rc = (pt % (ROWS / 8)) * 8;
    if (rt < nt) {
        const T* rows = REV ? static_cast<const T*>(p.dy) + (t0 + rt) * p.H * kHead
                            : static_cast<const T*>(p.in[3]) + (t0 + rt) * p.ld;
        raw.row = load8(rows + head + row0 + rc);
    }
}
// ... and, converted, from there into a stage.
template <typename T, int ROWS, bool REV>
__device__ __forceinline__ void stage_chunk(Stage<ROWS, REV>& st, const Raw<T, ROWS, REV>& raw, int nt, int pt) {
    const int t = pt >> 3, c = (pt & 7) * 8;
    const auto put = [](float* to, const float* f) {
        reinterpret_cast<float4*>(to)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(f[4], f[5], f[6], f[7]);
    };
    float f[8];
    if (t < nt) {
#pragma unroll
        for (int v = 0; v < nvec(REV); ++v) {
            cvt8<T>(raw.vec[v], f);
            if (v == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = decay_m1(f[j]);
            }
            put(&st.vec[v][t][c], f);
        }
    }
    const int rt = pt / (ROWS / 8), rc = (pt % (ROWS / 8)) * 8;
    if (rt < nt) {
        cvt8<T>(raw.row, f);
        put(&st.row[rt][rc], f);
    }
}

template <typename T, int ROWS>
__device__ __forceinline__ void store_y(const TmixArgs& p, const float (*y)[ROWS], int64_t t0, int nt, int h,
                                        int row0, int pt) {
    T* out = static_cast<T*>(p.out[0]);
    for (int piece = pt; piece < nt * (ROWS / 4); piece += NPW * 32) {
        const int t = piece / (ROWS / 4), c = (piece % (ROWS / 4)) * 4;
        store4(out + ((t0 + t) * p.H + h) * kHead + row0 + c, *reinterpret_cast<const float4*>(&y[t][c]));
    }
}

// One CTA: NCW compute warps of 8 RPL rows each, of one head of one sequence.
template <typename T, int RPL, int NCW, bool REV>
__global__ void __launch_bounds__((NCW + NPW) * 32) tmix_scan_kernel(const TmixArgs p) {
    constexpr int ROWS = NCW * 8 * RPL, SPLIT = kHead / ROWS;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem<ROWS, REV>& sm = *reinterpret_cast<Smem<ROWS, REV>*>(smem_raw);

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
        Raw<T, ROWS, REV> raw;
        const auto load = [&](int c) {
            if (c < nchunk)
                load_chunk<T, ROWS, REV>(p, raw, lo + static_cast<int64_t>(chunk_of(c)) * CT, tokens_in(chunk_of(c)),
                                         h, row0, pt);
        };
        const auto stage = [&](int c) {
            if (c < nchunk) stage_chunk<T, ROWS, REV>(sm.st[c & 1], raw, tokens_in(chunk_of(c)), pt);
        };
        load(0);
        stage(0);
        load(1);
        __syncthreads();
        for (int c = 0; c < nchunk; ++c) {
            stage(c + 1);
            load(c + 2);
            if constexpr (!REV) {
                if (c > 0) store_y<T, ROWS>(p, sm.y[(c - 1) & 1], lo + static_cast<int64_t>(c - 1) * CT, CT, h,
                                            row0, pt);
            }
            __syncthreads();
        }
        if constexpr (!REV) {
            if (nchunk > 0) store_y<T, ROWS>(p, sm.y[(nchunk - 1) & 1], lo + static_cast<int64_t>(nchunk - 1) * CT,
                                             tokens_in(nchunk - 1), h, row0, pt);
        }
        return;
    }

    // compute warps: lane (g, q) holds rows wrow .. wrow + RPL - 1, keys 16 i + 4 q + 0..3
    const int q = lane & 3, wrow = (warp * 8 + (lane >> 2)) * RPL;
    uint64_t S[RPL][8];
    const int64_t head_state = (slot * p.H + h) * kHead * kHead;
#pragma unroll
    for (int r = 0; r < RPL; ++r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.state_in != nullptr && slot >= 0)
                f = *reinterpret_cast<const float4*>(p.state_in + head_state + (row0 + wrow + r) * kHead + 16 * i +
                                                     4 * q);
            S[r][2 * i] = pack2(f.x, f.y);
            S[r][2 * i + 1] = pack2(f.z, f.w);
        }
    }
    float* const ck = REV ? p.gckpt : p.ckpt;
    const auto store_state = [&](float* dst) {
#pragma unroll
        for (int r = 0; r < RPL; ++r) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = unpack2(S[r][2 * i]), b = unpack2(S[r][2 * i + 1]);
                *reinterpret_cast<float4*>(dst + (row0 + wrow + r) * kHead + 16 * i + 4 * q) =
                    make_float4(a.x, a.y, b.x, b.y);
            }
        }
    };
    __syncthreads();
    for (int c = 0; c < nchunk; ++c) {
        const int ch = chunk_of(c), nt = tokens_in(ch);
        if (ck != nullptr) store_state(ck + ((ckpt_base(lo, seq) + ch) * p.H + h) * kHead * kHead);
        const Stage<ROWS, REV>& st = sm.st[c & 1];
#pragma unroll 2
        for (int s = 0; s < nt; ++s) {
            const int t = REV ? nt - 1 - s : s;
            const auto vec = [&](int v, int i) {
                return *reinterpret_cast<const ulonglong2*>(&st.vec[v][t][16 * i + 4 * q]);
            };
            float row[RPL];
#pragma unroll
            for (int r = 0; r < RPL; ++r) row[r] = st.row[t][wrow + r];
            if constexpr (REV) {             // G += dy r^T before the dot product
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const ulonglong2 x = vec(1, i);
#pragma unroll
                    for (int r = 0; r < RPL; ++r) {
                        const uint64_t rr = pack2(row[r], row[r]);
                        S[r][2 * i] = fma2(rr, x.x, S[r][2 * i]);
                        S[r][2 * i + 1] = fma2(rr, x.y, S[r][2 * i + 1]);
                    }
                }
            }
            // q = S a (backward: G b)
            float dot[RPL];
            {
                uint64_t acc[RPL][2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const ulonglong2 x = vec(2, i);
#pragma unroll
                    for (int r = 0; r < RPL; ++r) {
                        acc[r][0] = i ? fma2(S[r][2 * i], x.x, acc[r][0]) : mul2(S[r][0], x.x);
                        acc[r][1] = i ? fma2(S[r][2 * i + 1], x.y, acc[r][1]) : mul2(S[r][1], x.y);
                    }
                }
#pragma unroll
                for (int r = 0; r < RPL; ++r) {
                    const float2 f = unpack2(add2(acc[r][0], acc[r][1]));
                    dot[r] = f.x + f.y;
                }
            }
#pragma unroll
            for (int r = 0; r < RPL; ++r) dot[r] += __shfl_xor_sync(0xffffffffu, dot[r], 1);
#pragma unroll
            for (int r = 0; r < RPL; ++r) dot[r] += __shfl_xor_sync(0xffffffffu, dot[r], 2);
            // S = S + (w - 1) S (+ v k^T), then + q b^T
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const ulonglong2 w = vec(0, i);
#pragma unroll
                for (int r = 0; r < RPL; ++r) {
                    S[r][2 * i] = fma2(S[r][2 * i], w.x, S[r][2 * i]);
                    S[r][2 * i + 1] = fma2(S[r][2 * i + 1], w.y, S[r][2 * i + 1]);
                }
                if constexpr (!REV) {
                    const ulonglong2 x = vec(1, i);
#pragma unroll
                    for (int r = 0; r < RPL; ++r) {
                        const uint64_t rr = pack2(row[r], row[r]);
                        S[r][2 * i] = fma2(rr, x.x, S[r][2 * i]);
                        S[r][2 * i + 1] = fma2(rr, x.y, S[r][2 * i + 1]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const ulonglong2 x = vec(3, i);
#pragma unroll
                for (int r = 0; r < RPL; ++r) {
                    const uint64_t dd = pack2(dot[r], dot[r]);
                    S[r][2 * i] = fma2(dd, x.x, S[r][2 * i]);
                    S[r][2 * i + 1] = fma2(dd, x.y, S[r][2 * i + 1]);
                }
            }
            if constexpr (!REV) {            // y = S r
                uint64_t acc[RPL][2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const ulonglong2 x = vec(4, i);
#pragma unroll
                    for (int r = 0; r < RPL; ++r) {
                        acc[r][0] = i ? fma2(S[r][2 * i], x.x, acc[r][0]) : mul2(S[r][0], x.x);
                        acc[r][1] = i ? fma2(S[r][2 * i + 1], x.y, acc[r][1]) : mul2(S[r][1], x.y);
                    }
                }
#pragma unroll
                for (int r = 0; r < RPL; ++r) {
                    const float2 f = unpack2(add2(acc[r][0], acc[r][1]));
                    float y = f.x + f.y;
                    y += __shfl_xor_sync(0xffffffffu, y, 1);
                    y += __shfl_xor_sync(0xffffffffu, y, 2);
                    if (q == 0) sm.y[c & 1][t][wrow + r] = y;
                }
            }
        }
        __syncthreads();
    }
    if (p.state_out != nullptr && slot >= 0) store_state(p.state_out + head_state);
}

template <typename T, int RPL, int NCW, bool REV>
cudaError_t launch_scan(const TmixArgs& a, cudaStream_t s) {
    constexpr int ROWS = NCW * 8 * RPL;
    constexpr size_t smem = sizeof(Smem<ROWS, REV>);
    const cudaError_t e = allow_smem<tmix_scan_kernel<T, RPL, NCW, REV>>(smem);
    if (e != cudaSuccess) return e;
    tmix_scan_kernel<T, RPL, NCW, REV><<<a.S * a.H * (kHead / ROWS), (NCW + NPW) * 32, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T, bool REV>
cudaError_t scan_by_size(const TmixArgs& a, cudaStream_t s) {
#ifndef VAR_RPL
#define VAR_RPL 2
#define VAR_NCW 4
#endif
    return launch_scan<T, VAR_RPL, VAR_NCW, REV>(a, s);
}

// ------------------------------------------------------------ single token --
// One CTA per head of one request; four lanes share a row, a lane holds two
// rows.  Bound by the state's bytes: 16 KB read and 16 KB written per head.
template <typename T>
__global__ void __launch_bounds__(128) tmix_step_kernel(const TmixArgs p) {
    __shared__ float wm1[kHead];
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
    if (half) return reverse ? scan_by_size<__half, true>(a, s) : scan_by_size<__half, false>(a, s);
    return reverse ? scan_by_size<float, true>(a, s) : scan_by_size<float, false>(a, s);
}

cudaError_t launch_tmix_step(const TmixArgs& a, bool half, cudaStream_t s) {
    if (half) tmix_step_kernel<__half><<<a.S * a.H, 128, 0, s>>>(a);
    else tmix_step_kernel<float><<<a.S * a.H, 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace rq
