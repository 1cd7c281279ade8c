// Warp-level fp32 matrix products on the tensor cores by split tf32 operands.
//
// mma.sync m16n8k8 takes tf32 operands (11 significant bits) and accumulates
// in fp32. An fp32 value is cut into x = hi + lo, hi = x rounded to tf32 and
// lo = x - hi (exact in fp32), and a product is taken as
//     lo_a hi_b + hi_a lo_b + hi_a hi_b,
// which leaves out lo_a lo_b (2^-22 of the product) and lo's own rounding
// (2^-21): the products are as good as fp32 ones. A value that came from bf16
// is its own hi (8 bits), so that operand needs no lo: TA / TB below say how
// many parts (1 or 2) an operand is cut into; an operand with values of its own
// fp32 bits always takes two. What goes into a result that is rounded to bf16 next may
// be cut into two bf16 parts instead (mma_parts below).
//
// Measured on B200: one m16n8k8 tf32 (or m16n8k16 bf16) mma.sync per 8 cycles
// and SM quadrant, latency 20.6 cycles; three bf16 parts would need as many
// tensor cycles (6 x k16 against 3 x 2 x k8) and more instructions to form.
//
// A product advances sixteen k at a time, in two steps of eight whose k slots t
// and t + 4 hold two neighbours: lane (g, t) holds k = 2t, 2t + 1 and 2t + 8, 2t + 9.
// The order of a sum's terms is free as long as both operands agree, and in this
// one
//   - an accumulator tile (row g, columns 2t, 2t + 1; row g + 8, the same) is,
//     register for register, an A operand whose k runs over its columns,
//   - neighbours along a row of memory are one load, without bank conflicts where
//     rows start eight 32-bit banks apart (four for bf16). (One load of four
//     neighbours, k = 4t .., meets two-way conflicts there and measured 0.5 to 3 %
//     slower.)
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

// m16n8k16 on bf16 pairs: c += A B, and c = A B.
__device__ __forceinline__ void mma16(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16_0(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
}

// x's tf32 part (nearest) and what is left of it. A NaN stays one in `lo`.
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

// A 16 x 16 A operand as two 16 x 8 ones: {row g, row g + 8} x {first, second neighbour}.
template <int TA>
struct FragA {
    uint32_t hi[2][4], lo[2][4];
    // top and bottom: four k of row g and of row g + 8
    __device__ __forceinline__ void set(float4 top, float4 bottom) {
        const float x[2][4] = {{top.x, bottom.x, top.y, bottom.y}, {top.z, bottom.z, top.w, bottom.w}};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (TA == 2)
                    split(x[h][i], hi[h][i], lo[h][i]);
                else
                    hi[h][i] = __float_as_uint(x[h][i]);
            }
    }
};

// An A operand that is kept cut, in the order of its registers: 2 TA rows of 32 lanes x
// uint4 (conflict-free, and its readers do not cut it again).
template <int TA>
__device__ __forceinline__ void put_frag(uint4 *p, const FragA<TA> &f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        p[32 * h] = make_uint4(f.hi[h][0], f.hi[h][1], f.hi[h][2], f.hi[h][3]);
        if (TA == 2) p[64 + 32 * h] = make_uint4(f.lo[h][0], f.lo[h][1], f.lo[h][2], f.lo[h][3]);
    }
}
template <int TA>
__device__ __forceinline__ void get_frag(FragA<TA> &f, const uint4 *p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 u = p[32 * h];
        f.hi[h][0] = u.x, f.hi[h][1] = u.y, f.hi[h][2] = u.z, f.hi[h][3] = u.w;
        if (TA == 2) {
            const uint4 l = p[64 + 32 * h];
            f.lo[h][0] = l.x, f.lo[h][1] = l.y, f.lo[h][2] = l.z, f.lo[h][3] = l.w;
        }
    }
}

// A 16 x 8 B operand: four k of column g.
template <int TB>
struct FragB {
    uint32_t hi[4], lo[4];
    __device__ __forceinline__ void set(float4 v) {
        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (TB == 2)
                split(x[i], hi[i], lo[i]);
            else
                hi[i] = __float_as_uint(x[i]);
        }
    }
};

// acc += A B over KS sixteens of k.
// The tensor cores' accumulator drops the bits below its last place, always
// toward zero, so a long sum kept in it drifts. The terms of sixteen k are summed
// there from zero, the small parts first, and added to acc by an ordinary
// rounded addition: the error of a chain of products over 64 terms falls from
// 5e-7 to 2e-7 of its norm.
// Those terms depend on each other (20.6 cycles apart), so they go level by level
// over all KS * NT tiles; a warp that has its SM quadrant to itself wants four.
template <int TA, int TB, int NT, int KS>
__device__ __forceinline__ void mma_step(float (&acc)[NT][4], const FragA<TA> (&a)[KS],
                                         const FragB<TB> (&b)[KS][NT], int nt_end = NT) {
    float t[KS][NT][4];
    constexpr int SMALL = TA == 2 && TB == 2 ? 4 : TA == 2 || TB == 2 ? 2 : 0;
#pragma unroll
    for (int l = 0; l < SMALL + 2; ++l) {
        const int h = l < SMALL ? (l * 2) / (SMALL > 0 ? SMALL : 1) : l - SMALL;  // which eight
        const bool alo = l < SMALL && TA == 2 && (TB == 1 || (l & 1));
        const bool blo = l < SMALL && !alo;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n >= nt_end) continue;
                const uint32_t(&x)[4] = alo ? a[s].lo[h] : a[s].hi[h];
                const uint32_t *y = (blo ? b[s][n].lo : b[s][n].hi) + 2 * h;
                if (l == 0)
                    mma0(t[s][n], x, y[0], y[1]);
                else
                    mma(t[s][n], x, y[0], y[1]);
            }
    }
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n >= nt_end) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] += t[s][n][i];
        }
}

// k, k + 1, k + 8, k + 9 (k = 16 step + 2t) of row or column mn of an operand in
// shared memory. `K`: k runs along the rows of memory; otherwise it is the row
// index.
template <bool K>
__device__ __forceinline__ float4 quad(const float *p, int stride, int mn, int k) {
    if (K) {
        const float2 a = *reinterpret_cast<const float2 *>(p + mn * stride + k);
        const float2 b = *reinterpret_cast<const float2 *>(p + mn * stride + k + 8);
        return make_float4(a.x, a.y, b.x, b.y);
    }
    p += k * stride + mn;
    return make_float4(p[0], p[stride], p[8 * stride], p[9 * stride]);
}
__device__ __forceinline__ float2 unpack(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
// bf16: as pairs (k, k + 1 and k + 8, k + 9), or unpacked.
template <bool K>
__device__ __forceinline__ uint2 pair(const __nv_bfloat16 *p, int stride, int mn, int k) {
    if (K)
        return make_uint2(*reinterpret_cast<const uint32_t *>(p + mn * stride + k),
                          *reinterpret_cast<const uint32_t *>(p + mn * stride + k + 8));
    // a transposed 16 x 8 matrix load: lanes 0 .. 15 name the rows, and lane (g, t)
    // gets rows 2t, 2t + 1 and 2t + 8, 2t + 9 of column g. Every lane of the warp
    // asks for the same mn - g and k - 2t; rows are 16-byte aligned.
    const int lane = threadIdx.x & 31;
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(
        p + (k - 2 * (lane & 3) + (lane & 15)) * stride + mn - (lane >> 2)));
    uint32_t u, v;
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                 : "=r"(u), "=r"(v)
                 : "r"(at)
                 : "memory");
    return make_uint2(u, v);
}
template <bool K>
__device__ __forceinline__ float4 quad(const __nv_bfloat16 *p, int stride, int mn, int k) {
    const uint2 u = pair<K>(p, stride, mn, k);
    const float2 a = unpack(u.x), b = unpack(u.y);
    return make_float4(a.x, a.y, b.x, b.y);
}
// The quads of rows or columns g and g + 8 at once; p and k: the sixteen's start.
struct Quads {
    float4 a, b;
};
template <bool K>
__device__ __forceinline__ Quads quads(const float *p, int stride, int k) {
    const int g = (threadIdx.x & 31) >> 2, t2 = 2 * (threadIdx.x & 3);
    return {quad<K>(p, stride, g, k + t2), quad<K>(p, stride, g + 8, k + t2)};
}
// Four 8 x 8 matrices of bf16; lanes 8 i .. 8 i + 7 name the rows of the i-th.
template <bool TRANS>
__device__ __forceinline__ uint4 ldmatrix4(const __nv_bfloat16 *row) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(row));
    uint4 r;
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                     : "r"(at)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                     : "r"(at)
                     : "memory");
    return r;
}
// Rows or columns g (x, y: k's halves) and g + 8 (z, w) as bf16 pairs.
template <bool K>
__device__ __forceinline__ uint4 pairs(const __nv_bfloat16 *p, int stride, int k) {
    const int lane = threadIdx.x & 31;
    return ldmatrix4<!K>(K ? p + ((lane & 7) + 8 * (lane >> 4)) * stride + k + (lane & 8)
                           : p + (k + (lane & 15)) * stride + 8 * (lane >> 4));
}
template <bool K>
__device__ __forceinline__ Quads quads(const __nv_bfloat16 *p, int stride, int k) {
    const uint4 r = pairs<K>(p, stride, k);
    const float2 a = unpack(r.x), b = unpack(r.y), c = unpack(r.z), d = unpack(r.w);
    return {make_float4(a.x, a.y, b.x, b.y), make_float4(c.x, c.y, d.x, d.y)};
}

// Operands cut into bf16 parts, for m16n8k16 products: three parts (24 bits and more) of an
// fp32 value against bf16 values take three of those instead of four m16n8k8 of two tf32
// parts, with three quarters of the bytes, and the bf16 side needs no unpacking. Two parts
// (16 bits) are for what goes into a result that is rounded to bf16 next: against bf16
// values two products, against two parts three, where one tf32 part each (11 bits, off by
// up to 2^-10) takes two.
template <int P>
__device__ __forceinline__ void cut(float x, float y, uint32_t (&part)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        part[i] = *reinterpret_cast<const uint32_t *>(&h);
        const float2 f = unpack(part[i]);
        x -= f.x;
        y -= f.y;
    }
}
// A 16 x 16 A operand: four k of row g and of row g + 8
template <int P>
struct PartsA {
    uint4 p[P];
    __device__ __forceinline__ void set(float4 top, float4 bottom) {
        uint32_t a[4][P];
        cut(top.x, top.y, a[0]);
        cut(bottom.x, bottom.y, a[1]);
        cut(top.z, top.w, a[2]);
        cut(bottom.z, bottom.w, a[3]);
#pragma unroll
        for (int i = 0; i < P; ++i) p[i] = make_uint4(a[0][i], a[1][i], a[2][i], a[3][i]);
    }
    // one row of 32 lanes per part
    __device__ __forceinline__ void put(uint4 *d) const {
#pragma unroll
        for (int i = 0; i < P; ++i) d[32 * i] = p[i];
    }
    __device__ __forceinline__ void get(const uint4 *d) {
#pragma unroll
        for (int i = 0; i < P; ++i) p[i] = d[32 * i];
    }
};
// A 16 x 8 B operand: four k of column g; P = 1: bf16 pairs as they are
template <int P>
struct PartsB {
    uint2 p[P];
    __device__ __forceinline__ void set(float4 v) {
        uint32_t a[2][P];
        cut(v.x, v.y, a[0]);
        cut(v.z, v.w, a[1]);
#pragma unroll
        for (int i = 0; i < P; ++i) p[i] = make_uint2(a[0][i], a[1][i]);
    }
    __device__ __forceinline__ void set(uint2 v) { p[0] = v; }
};
// acc += A B over sixteen k, A in two parts: summed from zero, the small parts first, as in
// mma_step.
template <int PB, int NT>
__device__ __forceinline__ void mma_parts(float (&acc)[NT][4], const PartsA<2> &a,
                                          const PartsB<PB> (&b)[NT]) {
    float t[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) mma16_0(t[n], a.p[1], b[n].p[0].x, b[n].p[0].y);
    if (PB == 2) {
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16(t[n], a.p[0], b[n].p[PB - 1].x, b[n].p[PB - 1].y);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) mma16(t[n], a.p[0], b[n].p[0].x, b[n].p[0].y);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] += t[n][i];
}

// Lane (g, t) holds columns 2t, 2t + 1 of row g of an 8 x 8 tile (bf16: in one
// register) and gets those of its transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t u) {
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(u));
    return u;
}
__device__ __forceinline__ float2 transpose8(float x, float y) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    const uint32_t lo = transpose8(__byte_perm(a, b, 0x5410)), hi = transpose8(__byte_perm(a, b, 0x7632));
    return make_float2(__uint_as_float(__byte_perm(lo, hi, 0x5410)),
                       __uint_as_float(__byte_perm(lo, hi, 0x7632)));
}

// A quad times c[.] of its k.
__device__ __forceinline__ float4 scaled(float4 x, const float *c, int k) {
    return make_float4(x.x * c[k], x.y * c[k + 1], x.z * c[k + 8], x.w * c[k + 9]);
}

// acc[NT] += A B over the sixteens of k from `s0` to `s1`. fa(m, k) and fb(n, k)
// give quads of row m of A (0 .. 15) and of column n of B (0 .. 8 NT - 1).
// Columns from 8 * nt_end on are left alone.
template <int TA, int TB, int NT, int UNROLL = 1, class FA, class FB>
__device__ __forceinline__ void gemm(float (&acc)[NT][4], int s0, int s1, FA fa, FB fb,
                                     int nt_end = NT) {
    const int g = (threadIdx.x & 31) >> 2, t2 = 2 * (threadIdx.x & 3);
    constexpr int G = NT % 2 == 0 ? 2 : 1;  // tiles at a time: more cost registers
#pragma unroll UNROLL
    for (int st = s0; st < s1; ++st) {
        const int k = 16 * st + t2;
        FragA<TA> a[1];
        a[0].set(fa(g, k), fa(g + 8, k));
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += G) {
            FragB<TB> b[1][G];
#pragma unroll
            for (int n = 0; n < G; ++n)
                if (n0 + n < nt_end) b[0][n].set(fb(8 * (n0 + n) + g, k));
            mma_step<TA, TB, G, 1>(*reinterpret_cast<float(*)[G][4]>(&acc[n0]), a, b, nt_end - n0);
        }
    }
}

// The same with A in two bf16 parts, B in PB: fb gives a quad (PB = 2) or bf16 pairs (1).
template <int PB, int NT, class FA, class FB>
__device__ __forceinline__ void gemm_parts(float (&acc)[NT][4], int s0, int s1, FA fa, FB fb) {
    const int g = (threadIdx.x & 31) >> 2, t2 = 2 * (threadIdx.x & 3);
    constexpr int G = NT % 2 == 0 ? 2 : 1;
#pragma unroll 1
    for (int st = s0; st < s1; ++st) {
        const int k = 16 * st + t2;
        PartsA<2> a;
        a.set(fa(g, k), fa(g + 8, k));
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += G) {
            PartsB<PB> b[G];
#pragma unroll
            for (int n = 0; n < G; ++n) b[n].set(fb(8 * (n0 + n) + g, k));
            mma_parts<PB, G>(*reinterpret_cast<float(*)[G][4]>(&acc[n0]), a, b);
        }
    }
}

// Rows of shared memory times rows: kk += A B^T and (two) qk += A2 B^T over `steps`
// sixteens of k; row block A, A2 of 16, and eight rows of B from 16 nt + b0 on per
// tile nt < nt_end. Tiles go in pairs: of the last one a second may be computed in
// vain.
template <int NT>
__device__ __forceinline__ void grams(float (&kk)[NT][4], float (&qk)[NT][4], bool two,
                                      const float *A, const float *A2, const float *B, int stride,
                                      int b0, int steps, int nt_end) {
    const int g = (threadIdx.x & 31) >> 2, t2 = 2 * (threadIdx.x & 3);
#pragma unroll 1
    for (int st = 0; st < steps; ++st) {
        const int k = 16 * st + t2;
        FragA<2> a[1], a2[1];
        a[0].set(quad<true>(A, stride, g, k), quad<true>(A, stride, g + 8, k));
        if (two) a2[0].set(quad<true>(A2, stride, g, k), quad<true>(A2, stride, g + 8, k));
#pragma unroll
        for (int nt = 0; nt < NT; nt += 2) {
            if (nt >= nt_end) continue;
            FragB<2> b[1][2];
#pragma unroll
            for (int e = 0; e < 2; ++e) b[0][e].set(quad<true>(B, stride, 16 * (nt + e) + b0 + g, k));
            mma_step<2, 2, 2, 1>(*reinterpret_cast<float(*)[2][4]>(&kk[nt]), a, b);
            if (two) mma_step<2, 2, 2, 1>(*reinterpret_cast<float(*)[2][4]>(&qk[nt]), a2, b);
        }
    }
}
// The same of bf16: m16n8k16, whose products are exact as well, takes sixteen k in the
// cycles of eight tf32 ones, and its operands need no unpacking.
template <int NT>
__device__ __forceinline__ void grams(float (&kk)[NT][4], float (&qk)[NT][4], bool two,
                                      const __nv_bfloat16 *A, const __nv_bfloat16 *A2,
                                      const __nv_bfloat16 *B, int stride, int b0, int steps,
                                      int nt_end) {
    const int lane = threadIdx.x & 31;
    const int at = (lane & 15) * stride + 8 * (lane >> 4);  // rows, then the second eight k
    const __nv_bfloat16 *bt = B + (b0 + (lane & 7) + 16 * (lane >> 4)) * stride + (lane & 8);
#pragma unroll 1
    for (int st = 0; st < steps; ++st) {
        const uint4 a = ldmatrix4<false>(A + at + 16 * st);
        const uint4 a2 = two ? ldmatrix4<false>(A2 + at + 16 * st) : a;
#pragma unroll
        for (int nt = 0; nt < NT; nt += 2) {
            if (nt >= nt_end) continue;
            const uint4 b = ldmatrix4<false>(bt + 16 * nt * stride + 16 * st);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x[4], y[4];
                mma16_0(x, a, e ? b.z : b.x, e ? b.w : b.y);
                if (two) mma16_0(y, a2, e ? b.z : b.x, e ? b.w : b.y);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    kk[nt + e][i] += x[i];
                    if (two) qk[nt + e][i] += y[i];
                }
            }
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
