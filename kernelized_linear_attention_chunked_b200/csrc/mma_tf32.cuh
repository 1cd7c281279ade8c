// Warp-level fp32 matrix products on the tensor cores by split tf32 operands.
//
// mma.sync m16n8k8 takes tf32 operands (11 significant bits) and accumulates
// in fp32. An fp32 value is cut into x = hi + lo, hi = x rounded to tf32 and
// lo = x - hi (exact in fp32), and a product is taken as
//     lo_a hi_b + hi_a lo_b + hi_a hi_b,
// which leaves out lo_a lo_b (2^-22 of the product) and lo's own rounding
// (2^-21): the products are as good as fp32 ones. A value that came from bf16
// is its own hi (8 bits), so that operand needs no lo: TA / TB below say how
// many parts (1 or 2) an operand is cut into. One part of a general fp32
// operand is a rounding to 11 bits (toward zero, at most 2^-10), used only
// where the result is rounded to bf16 (2^-8) next.
//
// Measured on B200: one m16n8k8 tf32 (or m16n8k16 bf16) mma.sync per 8 cycles
// and SM quadrant, latency 20.6 cycles; three bf16 parts would need as many
// tensor cycles (6 x k16 against 3 x 2 x k8) and more instructions to form.
//
// Fragments use the k order (0 2 4 6 | 1 3 5 7) of each group of eight: the
// operands' k slots t and t + 4 hold k = 2t and 2t + 1. The order of a sum's
// terms is free as long as both operands agree, and in this one
//   - a K-major operand's two values of a lane are neighbours (one load), and
//   - an accumulator tile (row g, columns 2t, 2t + 1; row g + 8, the same) is,
//     register for register, an A operand whose k runs over its columns.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace kata {
namespace tf {

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// c = A B, on a zero accumulator.
__device__ __forceinline__ void mma0(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                     uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// x's tf32 part (nearest) and what is left of it. A NaN stays one in `lo`.
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

// A 16 x 8 A operand: {(g, 2t), (g + 8, 2t), (g, 2t + 1), (g + 8, 2t + 1)}.
template <int TA>
struct FragA {
    uint32_t hi[4], lo[4];
    __device__ __forceinline__ void set(float2 top, float2 bottom) {
        const float x[4] = {top.x, bottom.x, top.y, bottom.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (TA == 2)
                split(x[i], hi[i], lo[i]);
            else
                hi[i] = __float_as_uint(x[i]);
        }
    }
};

// acc += A B for one 16 x 8 A operand and one 8 x 8 B operand {(2t, g), (2t + 1, g)}.
// The tensor cores' accumulator drops the bits below its last place, always
// toward zero, so a long sum kept in it drifts. The eight terms of a step are
// summed there from zero and added to acc by an ordinary rounded addition:
// the error of a 64-term product falls from 5e-7 to 1.5e-7 of its norm.
//
// The parts of one tile depend on each other (20.6 cycles apart), so a step goes
// part by part over all NT tiles.
template <int TA, int TB, int NT>
__device__ __forceinline__ void mma_step(float (&acc)[NT][4], const FragA<TA> &a,
                                         const float2 (&b)[NT], int nt_end = NT) {
    float t[NT][4];
    uint32_t h0[NT], h1[NT], l0[NT], l1[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (n >= nt_end) continue;
        if (TB == 2) {
            split(b[n].x, h0[n], l0[n]);
            split(b[n].y, h1[n], l1[n]);
            mma0(t[n], a.hi, l0[n], l1[n]);
        } else {
            h0[n] = __float_as_uint(b[n].x);
            h1[n] = __float_as_uint(b[n].y);
            mma0(t[n], TA == 2 ? a.lo : a.hi, h0[n], h1[n]);
        }
    }
    if (TA == 2 && TB == 2) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (n < nt_end) mma(t[n], a.lo, h0[n], h1[n]);
    }
    if (TA == 2 || TB == 2) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (n < nt_end) mma(t[n], a.hi, h0[n], h1[n]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (n >= nt_end) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] += t[n][i];
    }
}

// Two k neighbours of an operand in shared memory, as floats. `K` says that k
// runs along the rows of memory (stride 1); otherwise k is the row index.
template <bool K>
__device__ __forceinline__ float2 pair(const float *p, int stride, int mn, int k) {
    if (K) return *reinterpret_cast<const float2 *>(p + mn * stride + k);
    return make_float2(p[k * stride + mn], p[(k + 1) * stride + mn]);
}
template <bool K>
__device__ __forceinline__ float2 pair(const __nv_bfloat16 *p, int stride, int mn, int k) {
    if (K) {
        const uint32_t u = *reinterpret_cast<const uint32_t *>(p + mn * stride + k);
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    }
    return make_float2(__bfloat162float(p[k * stride + mn]),
                       __bfloat162float(p[(k + 1) * stride + mn]));
}

// acc[NT] += A B over `kt1 - kt0` groups of eight k. fa(mn, k) and fb(mn, k)
// give two k neighbours of row mn of A (mn = 0 .. 15) and of column mn of B
// (mn = 0 .. 8 NT - 1). Columns from 8 * nt_end on are left alone.
template <int TA, int TB, int NT, class FA, class FB>
__device__ __forceinline__ void gemm(float (&acc)[NT][4], int kt0, int kt1, FA fa, FB fb,
                                     int nt_end = NT) {
    const int g = (threadIdx.x & 31) >> 2, t2 = 2 * (threadIdx.x & 3);
#pragma unroll 2
    for (int kt = kt0; kt < kt1; ++kt) {
        const int k = 8 * kt + t2;
        FragA<TA> a;
        a.set(fa(g, k), fa(g + 8, k));
        constexpr int G = NT % 2 == 0 ? 2 : 1;  // tiles at a time: more cost registers
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += G) {
            float2 b[G];
#pragma unroll
            for (int nt = 0; nt < G; ++nt)
                if (n0 + nt < nt_end) b[nt] = fb(8 * (n0 + nt) + g, k);
            mma_step<TA, TB, G>(*reinterpret_cast<float(*)[G][4]>(&acc[n0]), a, b, nt_end - n0);
        }
    }
}

template <int NT>
__device__ __forceinline__ void clear(float (&acc)[NT][4]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
}

// How many parts an operand read from the inputs has: bf16 values are exact in tf32.
template <typename T>
struct Parts;
template <>
struct Parts<float> {
    static constexpr int N = 2;
};
template <>
struct Parts<__nv_bfloat16> {
    static constexpr int N = 1;
};

}  // namespace tf
}  // namespace kata
