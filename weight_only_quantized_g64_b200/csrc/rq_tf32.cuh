// rq_tf32.cuh -- fp32 matrix products on the warp-level tensor cores.
//
// Every operand is split into two tf32 parts (22 bits of it), and lo*hi + hi*lo +
// hi*hi go into the fp32 accumulator; what is lost is about 2^-22 of each product.
// fp16 values are one part, exactly.  An SM retires 512 tf32 multiplications a
// cycle, 171 of them useful; plain fp32 FMAs would be 128, with an operand read
// from shared memory for each.
//
// mma.m16n8k8: lane (g, q) = (lane / 4, lane % 4) holds of the first operand rows
// g and g + 8, of the second column g, and of the sum rows g and g + 8, columns 2q
// and 2q + 1.  The summed index is taken in the order 2q, 2q + 1 (instead of q,
// q + 4), so that a sum can be the first operand of the next product as it is.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace rq {

// x = hi + lo: hi rounded to 11 bits, lo the rest, which the MMA cuts to 11 bits.
// Bit operations: the conversions to tf32 run at a fraction of their rate.  (A
// NaN may lose itself in hi, and is then in lo.)
struct Two {
    uint32_t hi, lo;
};
__device__ __forceinline__ Two split(float x) {
    const uint32_t hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    return {hi, __float_as_uint(x - __uint_as_float(hi))};
}
// {hi, hi, lo, lo} of two values
__device__ __forceinline__ float4 quad(float x, float y) {
    const Two a = split(x), b = split(y);
    return make_float4(__uint_as_float(a.hi), __uint_as_float(b.hi), __uint_as_float(a.lo), __uint_as_float(b.lo));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The first operand of one step (8 of the summed index) in two parts: rows g and
// g + 8, and of each the elements 2q and 2q + 1 of the step.
struct Rows {
    uint32_t hi[4], lo[4];
};
__device__ __forceinline__ Rows rows_of(float g0, float g1, float h0, float h1) {
    Rows r;
    const Two a = split(g0), b = split(h0), c = split(g1), d = split(h1);
    r.hi[0] = a.hi; r.hi[1] = b.hi; r.hi[2] = c.hi; r.hi[3] = d.hi;
    r.lo[0] = a.lo; r.lo[1] = b.lo; r.lo[2] = c.lo; r.lo[3] = d.lo;
    return r;
}
// N products of one step: the second operands are elements 2q and 2q + 1 of the
// step, column g, as quads.  The sums of the small parts are kept apart: the
// tensor cores cut every sum off (instead of rounding it), and the large one is
// then cut once a step instead of three times.  One part after the other over all
// N, as an MMA waits 21 cycles for the one before it on the same sum.  EXACT: the
// first operand is its hi part.
template <int N>
struct Sums {
    float c[N][4], small[N][4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[n][j] = small[n][j] = 0.f;
    }
    __device__ __forceinline__ float at(int n, int j) const { return c[n][j] + small[n][j]; }
    __device__ __forceinline__ void fold() {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c[n][j] += small[n][j];
                small[n][j] = 0.f;
            }
    }
};
template <bool EXACT = false, int N>
__device__ __forceinline__ void products(Sums<N>& s, const Rows& a, const float4 (&b)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) mma(s.small[n], a.hi, __float_as_uint(b[n].z), __float_as_uint(b[n].w));
#pragma unroll
    for (int n = 0; n < N; ++n) mma(s.c[n], a.hi, __float_as_uint(b[n].x), __float_as_uint(b[n].y));
    if (!EXACT) {
#pragma unroll
        for (int n = 0; n < N; ++n) mma(s.small[n], a.lo, __float_as_uint(b[n].x), __float_as_uint(b[n].y));
    }
}
// Second operands from a matrix whose rows are the columns of the product (two
// neighbours of a row), and from one whose rows are the summed index (two rows).
__device__ __forceinline__ float4 along(const float* p) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    return quad(f.x, f.y);
}
__device__ __forceinline__ float4 down(const float* p, int ld) { return quad(p[0], p[ld]); }
template <int LD>
__device__ __forceinline__ Rows rows_at(const float (*m)[LD], int g, int k) {     // rows g, g + 8; elements k, k + 1
    const float2 x = *reinterpret_cast<const float2*>(&m[g][k]), y = *reinterpret_cast<const float2*>(&m[g + 8][k]);
    return rows_of(x.x, x.y, y.x, y.y);
}
template <int LD>
__device__ __forceinline__ Rows columns_at(const float (*m)[LD], int g, int k) {  // of the transposed matrix
    return rows_of(m[k][g], m[k + 1][g], m[k][g + 8], m[k + 1][g + 8]);
}

}  // namespace rq
