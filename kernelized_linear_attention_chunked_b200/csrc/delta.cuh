// The chunked form of the gated delta rule, shared by the prefill (delta.cu)
// and the gradients (delta_backward.cu).
//
// Per (batch, head), with the state S [d, d] (key rows, value columns):
//     e_t = v_t - exp(g_t) S_{t-1}^T k_t,
//     S_t = exp(g_t) S_{t-1} + beta_t k_t e_t^T,      o_t = scale S_t^T q_t.
// Over a chunk of C = 64 tokens, with G_i = g_1 + .. + g_i, a_i = exp(G_i),
// D_ij = exp(G_i - G_j) and the chunk's first state S0:
//     E = V - diag(a) K S0 - N diag(beta) E,  N = tril(K K^T, -1) * D
//       = X V - X diag(a) K S0,               X = (1 + N diag(beta))^-1
//     O = scale (diag(a) Q S0 + M diag(beta) E),          M = tril(Q K^T) * D
//     S_C = a_C S0 + K^T diag(beta c) E,                  c_j = exp(G_C - G_j).
// Every exponent is a sum of log decays from an earlier token to a later one,
// so nothing overflows where g <= 0. G is summed and subtracted in 64 bits (a
// difference of two large sums keeps its digits after a strong decay), and a
// g below -200 counts as -200: exp of it is 0 in fp32 either way, and a g of
// minus infinity (the state starts anew) does not make inf - inf.
//
// A two-product chain was taken over a one-product one (S_C = A_c S0 + B_c with the
// d x d matrix A_c formed beforehand): that needs four more 64^3 products per chunk
// where there are now four.
//
// Two launches. delta_prep: one CTA per (chunk, head), everything that needs
// no state (W = X diag(a) K, XV, M). delta_chain: one CTA per (head, 16
// value columns) walks the chunks; columns of the state are independent, so
// the slices never meet. Its two products per chunk, E = XV - W S0 and
// S_C = .. + K^T (..E), are the serial part, so the inverse is applied to K
// and V beforehand: that leaves one product between a state and its error
// instead of two.
//
// The gradients run the same chain backwards (REV below): with dS the gradient
// of the chunk's last state,
//     Z = X^T diag(beta) (scale M^T dO + diag(c) K dS)
//     dS0 = a_C dS + scale Q^T diag(a) dO - K^T diag(a) Z,
// which has the same shape: Z = Z0 + W' dS with W' = X^T diag(beta c) K and
// Z0 = scale X^T diag(beta) M^T dO.
//
// Measured on B200 (bf16; both launches, each by itself under ncu): B2 H16 T16384 d64
// 186 + 325 us (485 a call), B4 H8 T2048 d32 21 + 30, B3 H5 T1531 d128 23 + 60. ncu at
// B2 H16 T4096 d64: delta_prep 60 % of issue slots, tensor pipe 37 %, shared memory 62 %,
// its CTAs a sequence of short dependent steps (32 warps per SM); delta_chain 128 CTAs of
// 148 SMs, about 2200 cycles per chunk, of which its critical products take 640: issue
// 41 %, tensor 40 %, shared memory 62 %.
//
// All products keep fp32 accuracy by split tf32 operands (mma_tf32.cuh): the
// state, its gradient, dg and dbeta are fp32 results. Only Q S0 and M E of bf16 inputs,
// which go into an o that is rounded to 8 bits next, take operands of 16 bits (two bf16
// parts): o is then off by its own rounding, 1.66e-3 of its norm. (With one tf32 part of
// each, 11 bits, it was 1.75e-3 to 1.81e-3.)
#pragma once

#include "kata_common.cuh"
#include "kata_internal.h"
#include "mma_tf32.cuh"
#include "tc_tiles.cuh"

namespace kata {
namespace delta {

constexpr int kC = 64;    // tokens per chunk
constexpr int kTS = 72;   // row stride of a 64 x 64 fp32 tile in shared memory
constexpr int kAS = 68;   // of the one whose rows are read least
constexpr int kCoef = 256;  // floats of coefficients per chunk: a' [64], c' [64], a_C
constexpr float kMinLog = -200.f;
constexpr int kLoaders = 128;     // threads of delta_chain that copy
constexpr int kChainThreads = 256 + kLoaders;

// Row stride of a [64, D] tile in shared memory: rows start four 32-bit banks
// apart (eight for fp32), so a K-major fragment load has no bank conflict.
template <int D>
constexpr int row_stride() {
    return D + 8;
}

// Per-chunk scratch. "Fragment order" of a [64, n] matrix: the 16 x 8
// accumulator tiles row block by row block, each as 32 lanes x float4, so that
// a tile moves with one coalesced 128-bit access per lane.
struct Scratch {
    float *W;     // [chunks][64 D], fragment order
    float *Y;     // [chunks][64 D], fragment order: XV, or Z0
    float *M;     // [chunks][64 * 64], fragment order: scale M diag(beta); bf16 inputs: each
                  // two neighbours as two pairs of bf16 parts
    float *coef;  // [chunks][kCoef]
};

struct Args {
    const void *q, *k, *v, *d_o;
    const float *g, *beta;
    const float *S_in;  // first state (REV: gradient of the last one); NULL = zero
    float *S_out;       // last state (REV: gradient of the first one); NULL: not written
    void *o;
    float *keepY;       // [chunks][64][D]: E (REV: Z)
    float *keepS;       // [chunks][D][D]: each chunk's first state (REV: gradient of its last)
    int T, nc;
    float scale;
};

__device__ __forceinline__ void cp16(void *dst, const void *src, bool have) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    const int n = have ? 16 : 0;  // 0: sixteen zero bytes, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// waits until at most N of this thread's groups are on their way
template <int N>
__device__ __forceinline__ void cp_wait_ahead() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Rows [t0, t0 + ROWS) of the [nrows, D] matrix that starts at row `row0`, columns [c0, c0 + N), to
// a tile with row stride `stride`; rows from nrows on become zero.
// NTH threads take part, tid = 0 .. NTH - 1.
template <typename T, int N, int NTH, int ROWS = kC>
__device__ __forceinline__ void load_tile(T *dst, int stride, const T *src, size_t row0, int t0,
                                          int nrows, int D, int c0, int tid) {
    constexpr int PER = 16 / sizeof(T);
    constexpr int CH = N / PER;
    constexpr int RPP = NTH / CH;  // rows per pass
    static_assert(NTH % CH == 0, "whole rows per pass");
    const int r0 = tid / CH, c = (tid % CH) * PER;
    const T *s = src + (row0 + t0 + r0) * (size_t)D + c0 + c;
    T *d = dst + r0 * stride + c;
    if (t0 + ROWS <= nrows) {
#pragma unroll
        for (int r = 0; r < ROWS; r += RPP)
            if (ROWS % RPP == 0 || r0 + r < ROWS) cp16(d + r * stride, s + (size_t)r * D, true);
    } else {
        for (int r = 0; r < ROWS && r0 + r < ROWS; r += RPP) {
            const bool have = t0 + r0 + r < nrows;
            cp16(d + r * stride, have ? s + (size_t)r * D : src, have);
        }
    }
}

// The running sums of one chunk's log decays, in base 2 and as two floats each (a
// 64-bit sum's upper and lower part): an exponent is taken as (hi_i - hi_j) +
// (lo_i - lo_j), whose error is 2^-24 of the difference, not of the sums. One
// warp; v: tokens 2 lane and 2 lane + 1 of the chunk.
__device__ __forceinline__ float2 load_decays(const float *g, size_t row0, int t0, int T) {
    const int t = t0 + 2 * (threadIdx.x & 31);
    return make_float2(t < T ? g[row0 + t] : 0.f, t + 1 < T ? g[row0 + t + 1] : 0.f);
}
__device__ __forceinline__ void cumulate(float2 v, float *hi, float *lo) {
    const int lane = threadIdx.x & 31;
    const double x0 = v.x < kMinLog ? kMinLog : v.x;
    double x1 = v.y < kMinLog ? kMinLog : v.y;
    x1 += x0;
    double sum = x1;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += up;
    }
    constexpr double kLog2e = 1.4426950408889634;
    const double s0 = (sum - x1 + x0) * kLog2e, s1 = sum * kLog2e;
    const float h0 = (float)s0, h1 = (float)s1;
    *reinterpret_cast<float2 *>(hi + 2 * lane) = make_float2(h0, h1);
    *reinterpret_cast<float2 *>(lo + 2 * lane) =
        make_float2((float)(s0 - (double)h0), (float)(s1 - (double)h1));
}

// exp(G_i - G_j) for two neighbouring j of the sums hi, lo.
__device__ __forceinline__ float2 decay2(float hi_i, float lo_i, const float *hi, const float *lo,
                                         int j) {
    const float2 h = *reinterpret_cast<const float2 *>(hi + j);
    const float2 l = *reinterpret_cast<const float2 *>(lo + j);
    return make_float2(exp2f((hi_i - h.x) + (lo_i - l.x)), exp2f((hi_i - h.y) + (lo_i - l.y)));
}

// sX = (1 + A)^-1 for the strictly lower triangular A (64 x 64, row
// strides kTS and kAS), by the CTA's first four warps. Diagonal 16 x 16 blocks by forward substitution,
// one column per lane; then the blocks below them, 16 to 32 to 64 rows, by
//     X21 = -X22 (A21 X11),
// where a warp's own columns need no other warp's. The blocks above the
// diagonal hold the intermediate products and are not part of the result.
__device__ __forceinline__ void invert(const float *sA, float *sX, int warp, int lane) {
    using namespace tf;
    const int g = lane >> 2, t2 = 2 * (lane & 3);
    if (warp < 4) {
        const int j = lane & 15;
        const float *A = sA + 16 * warp * kAS + 16 * warp;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == j ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < 15; ++m)  // x[m] is final: take it out of the rows below
#pragma unroll
            for (int i = m + 1; i < 16; ++i) x[i] = fmaf(-A[i * kAS + m], x[m], x[i]);
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sX[(16 * warp + i) * kTS + 16 * warp + j] = x[i];
        }
    }
    __syncthreads();
    if (warp < 4) {  // blocks (1, 0) and (3, 2): warp w takes eight columns of pair w / 2
        const int r0 = 32 * (warp >> 1), c = r0 + 8 * (warp & 1);
        float acc[1][4];
        clear(acc);
        gemm<2, 2, 1>(
            acc, 0, 1,
            [&](int m, int k) { return quad<true>(sA + (r0 + 16) * kAS + r0, kAS, m, k); },
            [&](int n, int k) { return quad<false>(sX + r0 * kTS + c, kTS, n, k); });
        float *P = sX + r0 * kTS + c + 16;
        *reinterpret_cast<float2 *>(P + g * kTS + t2) = make_float2(acc[0][0], acc[0][1]);
        *reinterpret_cast<float2 *>(P + (g + 8) * kTS + t2) = make_float2(acc[0][2], acc[0][3]);
        __syncwarp();
        clear(acc);
        gemm<2, 2, 1>(
            acc, 0, 1,
            [&](int m, int k) { return quad<true>(sX + (r0 + 16) * kTS + r0 + 16, kTS, m, k); },
            [&](int n, int k) { return quad<false>(P, kTS, n, k); });
        float *O = sX + (r0 + 16) * kTS + c;
        *reinterpret_cast<float2 *>(O + g * kTS + t2) = make_float2(-acc[0][0], -acc[0][1]);
        *reinterpret_cast<float2 *>(O + (g + 8) * kTS + t2) = make_float2(-acc[0][2], -acc[0][3]);
    }
    __syncthreads();
    if (warp < 4) {  // the lower left 32 x 32 block: warp w takes its columns 8 w .. 8 w + 7
        const int c = 8 * warp;
        float *P = sX + 32 + c;
        // rows m0 .. of A (32 columns) times a 32 x 8 B: both sixteens of k at once, or one
        auto product = [&](float(&acc)[1][4], const float *A, int as, const float *B, bool first,
                           bool second) {
            FragA<2> a[2];
            FragB<2> b[2][1];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                a[s].set(quad<true>(A, as, g, 16 * s + t2), quad<true>(A, as, g + 8, 16 * s + t2));
                float4 x = quad<false>(B, kTS, g, 16 * s + t2);
                if (!(s ? second : first)) x = make_float4(0.f, 0.f, 0.f, 0.f);
                b[s][0].set(x);
            }
            mma_step<2, 2, 1, 2>(acc, a, b);
        };
        auto put = [&](float *O, const float(&acc)[1][4], float sign) {
            *reinterpret_cast<float2 *>(O + g * kTS + t2) = make_float2(sign * acc[0][0], sign * acc[0][1]);
            *reinterpret_cast<float2 *>(O + (g + 8) * kTS + t2) =
                make_float2(sign * acc[0][2], sign * acc[0][3]);
        };
        float acc[2][1][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {  // X11 has nothing above its diagonal blocks
            clear(acc[mt]);
            product(acc[mt], sA + (32 + 16 * mt) * kAS, kAS, sX + c, warp < 2, true);
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) put(P + 16 * mt * kTS, acc[mt], 1.f);
        __syncwarp();
        clear(acc[0]);  // nor X22, so its first row block takes one sixteen
        gemm<2, 2, 1>(
            acc[0], 0, 1, [&](int m, int k) { return quad<true>(sX + 32 * kTS + 32, kTS, m, k); },
            [&](int n, int k) { return quad<false>(P, kTS, n, k); });
        clear(acc[1]);
        product(acc[1], sX + 48 * kTS + 32, kTS, P, true, true);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) put(sX + (32 + 16 * mt) * kTS + c, acc[mt], -1.f);
    }
    __syncthreads();
}

template <typename Tin, int D, bool BACK>
struct PrepSmem {
    static constexpr int KS = row_stride<D>();
    static constexpr int IN = kC * KS * (int)sizeof(Tin);
    static constexpr int P = kC * KS * 4;  // BACK: diag(beta) M^T dO, over V
    static constexpr int T = kC * kTS * 4, X = IN, Q = X;  // X over Q
    static constexpr int K = 0, V = X + (IN > T ? IN : T), DO = V + (BACK ? P : IN);
    static constexpr int A = DO + (BACK ? IN : 0), M = A + kC * kAS * 4;
    static constexpr int COEF = M + (BACK ? T : 0);  // beta, a, beta c, G (hi, lo)
    static constexpr int BYTES = COEF + 5 * kC * 4;
    // four CTAs per SM where their shared memory allows it, at 64 registers (d64 184 -> 174
    // us at B2 H16 T16384); otherwise the registers are the compiler's choice (with as few
    // d128 took 21.8 us instead of 20.2 at B3 H5 T1531)
    static constexpr int CTAS = sizeof(Tin) == 2 && 4 * (BYTES + 1024) <= 228 * 1024 ? 4 : 1;
};

// Tiles first .. first + N - 1 of row block rb of a [64, D] matrix in fragment order.
template <int D, int N>
__device__ __forceinline__ void store_frags(float *dst, const float (&acc)[N][4], int rb, int first,
                                            int lane) {
    float4 *d = reinterpret_cast<float4 *>(dst) + (size_t)(rb * (D / 8) + first) * 32 + lane;
#pragma unroll
    for (int nt = 0; nt < N; ++nt)
        d[nt * 32] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
}

// The same, each 16 x 8 tile transposed: a lane's four values are rows 2t, 2t + 1, 2t + 8,
// 2t + 9 of column g.
template <int D, int N>
__device__ __forceinline__ void store_frags_t(float *dst, const float (&acc)[N][4], int rb, int first,
                                              int lane) {
    float4 *d = reinterpret_cast<float4 *>(dst) + (size_t)(rb * (D / 8) + first) * 32 + lane;
#pragma unroll
    for (int nt = 0; nt < N; ++nt) {
        const float2 a = tf::transpose8(acc[nt][0], acc[nt][1]), b = tf::transpose8(acc[nt][2], acc[nt][3]);
        d[nt * 32] = make_float4(a.x, a.y, b.x, b.y);
    }
}

// What each chunk needs of itself alone. 8 warps: 16 rows (warp % 4) and half the
// columns each, of a triangular product every other eight.
// f: the forward chain's operands; r: the reverse chain's (BACK only).
template <typename Tin, int D, bool BACK>
__global__ void __launch_bounds__(256, PrepSmem<Tin, D, BACK>::CTAS)
    delta_prep(Args p, Scratch f, Scratch r) {
    using namespace tf;
    using L = PrepSmem<Tin, D, BACK>;
    constexpr int KS = L::KS, TI = Parts<Tin>::N;
    extern __shared__ __align__(16) uint8_t sm[];
    Tin *sK = reinterpret_cast<Tin *>(sm + L::K), *sQ = reinterpret_cast<Tin *>(sm + L::Q);
    Tin *sV = reinterpret_cast<Tin *>(sm + L::V), *sO = reinterpret_cast<Tin *>(sm + L::DO);
    float *sA = reinterpret_cast<float *>(sm + L::A), *sX = reinterpret_cast<float *>(sm + L::X);
    float *sM = reinterpret_cast<float *>(sm + L::M), *sP = reinterpret_cast<float *>(sm + L::V);
    float *beta = reinterpret_cast<float *>(sm + L::COEF), *ca = beta + kC, *bc = ca + kC;
    float *ghi = bc + kC, *glo = ghi + kC;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, t2 = 2 * (lane & 3);
    const size_t ch = blockIdx.x;  // head * nc + chunk
    const size_t head = ch / p.nc;
    const int t0 = (int)(ch % p.nc) * kC;
    const size_t row0 = head * (size_t)p.T;

    if (tid == 0) sm100::launch_dependents();  // the walks: they wait for this grid's end
    sm100::grid_dependency_wait();             // whatever the stream ran before
    float2 v2 = make_float2(0.f, 0.f);
    if (warp == 0) v2 = load_decays(p.g, row0, t0, p.T);
    load_tile<Tin, D, 256>(sK, KS, static_cast<const Tin *>(p.k), row0, t0, p.T, D, 0, tid);
    if (BACK || p.o)
        load_tile<Tin, D, 256>(sQ, KS, static_cast<const Tin *>(p.q), row0, t0, p.T, D, 0, tid);
    load_tile<Tin, D, 256>(sV, KS, static_cast<const Tin *>(p.v), row0, t0, p.T, D, 0, tid);
    if (BACK)
        load_tile<Tin, D, 256>(sO, KS, static_cast<const Tin *>(p.d_o), row0, t0, p.T, D, 0, tid);
    cp_commit();
    if (warp == 0) cumulate(v2, ghi, glo);
    if (tid >= 192) {
        const int t = t0 + tid - 192;
        beta[tid - 192] = t < p.T ? p.beta[row0 + t] : 0.f;
    }
    cp_wait_all();
    __syncthreads();
    if (tid < kC) {
        const float a = exp2f(ghi[tid] + glo[tid]);
        const float c = exp2f((ghi[kC - 1] - ghi[tid]) + (glo[kC - 1] - glo[tid]));
        ca[tid] = a;
        bc[tid] = beta[tid] * c;
        float *cf = f.coef + ch * kCoef;
        cf[tid] = p.scale * a;
        cf[kC + tid] = bc[tid];
        if (tid == kC - 1) cf[2 * kC] = a;
        if (BACK) {
            float *cr = r.coef + ch * kCoef;
            cr[tid] = p.scale * a;
            cr[kC + tid] = -a;
            if (tid == kC - 1) cr[2 * kC] = a;
        }
    }
    __syncthreads();

    const int rb = warp & 3, hf = warp >> 2, m0 = 16 * rb;
    const int nt_end = rb + 1;  // this warp's column tiles up to the diagonal block
    const bool wantQ = BACK || p.o;
    {
        // K K^T and Q K^T
        float kk[4][4], qk[4][4];
        clear(kk);
        clear(qk);
        grams(kk, qk, wantQ, sK + m0 * KS, sQ + m0 * KS, sK, KS, 8 * hf, D / 16, nt_end);
        float4 *d = BACK ? nullptr
                         : reinterpret_cast<float4 *>(f.M + ch * (kC * kC)) + (size_t)rb * 8 * 32 + lane;
        const float gh[2] = {ghi[m0 + gr], ghi[m0 + gr + 8]}, gl[2] = {glo[m0 + gr], glo[m0 + gr + 8]};
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            if (nt >= nt_end) continue;
            const int j = 8 * (2 * nt + hf) + t2;
            const float2 be = *reinterpret_cast<const float2 *>(beta + j);
            float m[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = m0 + gr + 8 * h;
                const float2 dec = decay2(gh[h], gl[h], ghi, glo, j);
                // (above the diagonal a decay may be infinite: chosen away, not multiplied)
                *reinterpret_cast<float2 *>(sA + i * kAS + j) =
                    make_float2(i > j ? kk[nt][2 * h] * dec.x * be.x : 0.f,
                                i > j + 1 ? kk[nt][2 * h + 1] * dec.y * be.y : 0.f);
                m[2 * h] = i >= j ? qk[nt][2 * h] * dec.x : 0.f;
                m[2 * h + 1] = i >= j + 1 ? qk[nt][2 * h + 1] * dec.y : 0.f;
                if (BACK) *reinterpret_cast<float2 *>(sM + i * kTS + j) = make_float2(m[2 * h], m[2 * h + 1]);
            }
            if (!BACK && wantQ) {
                const float s0 = p.scale * be.x, s1 = p.scale * be.y;
                float4 x = make_float4(s0 * m[0], s1 * m[1], s0 * m[2], s1 * m[3]);
                if constexpr (TI == 1) {
                    uint32_t u[2], v[2];
                    cut(x.x, x.y, u);
                    cut(x.z, x.w, v);
                    x = make_float4(__uint_as_float(u[0]), __uint_as_float(u[1]), __uint_as_float(v[0]),
                                    __uint_as_float(v[1]));
                }
                d[(2 * nt + hf) * 32] = x;
            }
        }
    }
    __syncthreads();
    invert(sA, sX, warp, lane);

    constexpr int ND = D / 16;  // this warp's tiles of a [64, D] product
    const int d0 = hf * (D / 2), td = hf * ND;
    float acc[ND][4];
    clear(acc);
    gemm<2, TI, ND>(  // X V
        acc, 0, rb + 1, [&](int m, int k) { return quad<true>(sX + m0 * kTS, kTS, m, k); },
        [&](int n, int k) { return quad<false>(sV + d0, KS, n, k); });
    store_frags_t<D>(f.Y + ch * (kC * D), acc, rb, td, lane);
    auto kcols = [&](int n, int k) { return quad<false>(sK + d0, KS, n, k); };
    clear(acc);
    gemm<2, TI, ND>(  // X diag(a) K
        acc, 0, rb + 1,
        [&](int m, int k) {
            return scaled(quad<true>(sX + m0 * kTS, kTS, m, k), ca, k);
        },
        kcols);
    store_frags<D>(f.W + ch * (kC * D), acc, rb, td, lane);
    if (!BACK) return;

    // Z0 = X^T (scale diag(beta) M^T dO), W' = X^T diag(beta c) K: the
    // transposed factors reach from a row's own block to the last one
    clear(acc);
    gemm<2, TI, ND>(
        acc, rb, 4, [&](int m, int k) { return quad<false>(sM + m0, kTS, m, k); },
        [&](int n, int k) { return quad<false>(sO + d0, KS, n, k); });
    __syncthreads();  // every warp has read V
    {
        const float s0 = p.scale * beta[m0 + gr], s1 = p.scale * beta[m0 + gr + 8];
#pragma unroll
        for (int nt = 0; nt < ND; ++nt) {
            float *x = sP + (m0 + gr) * KS + d0 + 8 * nt + t2;
            *reinterpret_cast<float2 *>(x) = make_float2(s0 * acc[nt][0], s0 * acc[nt][1]);
            *reinterpret_cast<float2 *>(x + 8 * KS) = make_float2(s1 * acc[nt][2], s1 * acc[nt][3]);
        }
    }
    __syncthreads();
    clear(acc);
    gemm<2, 2, ND>(
        acc, rb, 4, [&](int m, int k) { return quad<false>(sX + m0, kTS, m, k); },
        [&](int n, int k) { return quad<false>(sP + d0, KS, n, k); });
    store_frags_t<D>(r.Y + ch * (kC * D), acc, rb, td, lane);
    clear(acc);
    gemm<2, TI, ND>(
        acc, rb, 4,
        [&](int m, int k) {
            return scaled(quad<false>(sX + m0, kTS, m, k), bc, k);
        },
        kcols);
    store_frags<D>(r.W + ch * (kC * D), acc, rb, td, lane);
}

constexpr int kSlice = 16;  // value columns per CTA: the rows of one operand tile

template <typename Tin, int D, bool REV>
struct ChainSmem {
    static constexpr int KS = row_stride<D>();
    static constexpr int DS = kSlice + 8;  // row stride of the dO slice
    static constexpr int IN = kC * KS * (int)sizeof(Tin);
    static constexpr int FRAG = 1024;      // a 16 x 16 A operand, or one tf32 part of it
    // the state in two parts; the chunk's errors whole, or in three bf16 parts
    static constexpr int S = 0, YC = S + D / 16 * 2 * FRAG, SIDE = YC + kC / 16 * 3 * FRAG / 2;
    // what passes between the chain and the side warps: E or (REV) Q^T diag(scale a) dO
    // forward, bf16 inputs: the state in two bf16 parts, for the outputs
    static constexpr int SB = SIDE + (REV ? D / 16 * FRAG : kC / 16 * tf::Parts<Tin>::N * FRAG);
    static constexpr int STAGE = SB + (REV || sizeof(Tin) == 4 ? 0 : D / 16 * FRAG);
    // one stage: K, Q, coefficients, (REV) the dO slice
    static constexpr int K = 0, Q = IN, COEF = 2 * IN, DO = COEF + kCoef * 4;
    static constexpr int STAGE_BYTES = DO + (REV ? kC * DS * (int)sizeof(Tin) : 0);
    // as many as fit, up to four: three chunks ahead
    static constexpr int FIT = (227 * 1024 - STAGE) / STAGE_BYTES;
    static constexpr int STAGES = FIT < 4 ? FIT : 4;
    static_assert(STAGES >= 2, "a stage in use and one on its way");
    static constexpr int BYTES = STAGE + STAGES * STAGE_BYTES;
};

// The walk over the chunks, one CTA per (head, 16 value columns): `cta` of them. Everything
// is transposed, so that the 16 value columns are the rows of the products,
//     E^T = XV^T - S0^T W^T,  S_C^T = a_C S0^T + (c beta E)^T K,
//     O^T = scale S0^T Q^T diag(a) + E^T M^T,
// and an accumulator is, register for register, the A operand of the product that
// follows: 128-bit reads where the plain form took four times as many scalar ones (d = 64
// 341 -> 310 us at B2 H16 T16384, d = 32 33 -> 31 us at B4 H8 T2048). The state is
// cut into tf32 parts by the warp that makes it, the errors by their readers (the other
// ways round: errors cut by their maker 316 us, the state by its readers too 321). For the
// outputs of bf16 inputs that warp cuts state and errors into bf16 parts as well, and
// delta_prep cuts M (B2 H16 T16384 d64, both launches: 486 us; the state's tf32 parts read for
// them instead 535, M cut by its readers 530 to 544). A chunk
// of d = 64 takes 2200 cycles: 1100 for E, 1000 for the state and the outputs' end. Bound by
// the length of these steps and by shared memory (1250 of those cycles move data).
// Measured without gain: the outputs a chunk behind the chain with barriers of their
// own (d64 the same, d32 33 -> 36 us), their products two sixteens at a time (d32 31 -> 34),
// M by the copying warps (d32 31 -> 34).
// Warps 0-3 carry the chain: they hold the state in registers (fp32, D / 4 of its rows
// each) and take two dependent products per chunk. Warps 4-7 take the products that
// hang off it: the outputs (forward) or Q^T dO (REV). Warps 8-11 bring K, Q and
// the coefficients by asynchronous copies up to three chunks ahead, and call
// the next chunks' W, XV and M into L2; those come straight from there into
// the fragments that use them, one chunk ahead.
template <typename Tin, int D, bool REV, bool KEEP>
__device__ __forceinline__ void walk_chunks(const Args &p, const Scratch &w, const unsigned cta) {
    using namespace tf;
    using L = ChainSmem<Tin, D, REV>;
    constexpr int KS = L::KS, TI = Parts<Tin>::N;
    constexpr int MT = D >= 64 ? D / 64 : 1;  // sixteens of the state's rows per chain warp
    constexpr int KP = D >= 32 ? 2 : 1;       // sixteens of k at a time
    // (c beta E)^T in three bf16 parts, for bf16 K: cutting takes longer on the critical
    // path, which pays where a warp uses a part twice (d128 68 -> 63 us at B3 H5 T1531; d64
    // 315 -> 324 us at B2 H16 T16384; d128 with whole ones 68)
    constexpr bool CUT3 = TI == 1 && MT > 1;
    extern __shared__ __align__(16) uint8_t sm[];
    uint4 *sS = reinterpret_cast<uint4 *>(sm + L::S), *sCut = reinterpret_cast<uint4 *>(sm + L::YC);
    float4 *sYc = reinterpret_cast<float4 *>(sm + L::YC);
    uint4 *sE = reinterpret_cast<uint4 *>(sm + L::SIDE);
    uint4 *sSb = reinterpret_cast<uint4 *>(sm + L::SB);
    float4 *sG = reinterpret_cast<float4 *>(sm + L::SIDE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, t2 = 2 * (lane & 3), rw = warp & 3;
    const size_t head = cta / (D / kSlice);
    const int slice = cta % (D / kSlice), c0 = slice * kSlice;
    const size_t row0 = head * (size_t)p.T;
    const int m0 = 16 * rw;
    const bool wantO = !REV && p.o != nullptr;
    const size_t ch0 = head * p.nc;
    auto chunk_of = [&](int i) { return REV ? p.nc - 1 - i : i; };

    if (warp >= 8) {
        // ---------------- copies ----------------
        const int lt = tid - 256;
        auto fetch = [&](int i) {
            if (i < p.nc) {
                uint8_t *s = sm + L::STAGE + (i % L::STAGES) * L::STAGE_BYTES;
                const int c = chunk_of(i);
                load_tile<Tin, D, kLoaders>(reinterpret_cast<Tin *>(s + L::K), KS,
                                            static_cast<const Tin *>(p.k), row0, c * kC, p.T, D, 0, lt);
                if (REV || wantO)
                    load_tile<Tin, D, kLoaders>(reinterpret_cast<Tin *>(s + L::Q), KS,
                                                static_cast<const Tin *>(p.q), row0, c * kC, p.T, D, 0,
                                                lt);
                if (REV)
                    load_tile<Tin, kSlice, kLoaders>(reinterpret_cast<Tin *>(s + L::DO), L::DS,
                                                     static_cast<const Tin *>(p.d_o), row0, c * kC, p.T,
                                                     D, c0, lt);
                const float *cf = w.coef + (ch0 + c) * kCoef;
                if (lt < kCoef / 4) cp16(s + L::COEF + lt * 16, cf + lt * 4, true);
                if (slice == 0 && lt == kLoaders - 1) {
                    prefetch_l2(w.W + (ch0 + c) * (kC * D), kC * D * 4);
                    prefetch_l2(w.Y + (ch0 + c) * (kC * D), kC * D * 4);
                    if (wantO) prefetch_l2(w.M + (ch0 + c) * (kC * kC), kC * kC * 4);
                }
            }
            cp_commit();  // one group per chunk, empty past the end
        };
        for (int i = 0; i < L::STAGES - 1; ++i) fetch(i);
        cp_wait_ahead<L::STAGES - 2>();
        __syncthreads();
        for (int i = 0; i < p.nc; ++i) {
            fetch(i + L::STAGES - 1);  // over the stage of chunk i - 1
            __syncthreads();
            cp_wait_ahead<L::STAGES - 2>();
            __syncthreads();
        }
        return;
    }

    const bool chain = warp < 4;
    // The state, transposed, in accumulator layout: value columns c0 + gr (+ 8 for e = 2, 3),
    // rows srow(mt, nt) (+ 1 for e = 1, 3). An accumulator pair as quads: rows gr, gr + 8.
    float S[MT][2][4];
    const bool owns = chain && (D >= 64 || warp < D / 16);
    auto srow = [&](int mt, int nt) { return 16 * (MT * warp + mt) + 8 * nt + t2; };
    auto top = [](const float(&x)[2][4]) { return make_float4(x[0][0], x[0][1], x[1][0], x[1][1]); };
    auto bottom = [](const float(&x)[2][4]) { return make_float4(x[0][2], x[0][3], x[1][2], x[1][3]); };
    auto put_state = [&]() {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            FragA<2> f;
            f.set(top(S[mt]), bottom(S[mt]));
            put_frag(sS + (MT * warp + mt) * 128 + lane, f);
            if (TI == 1 && wantO) {
                PartsA<2> h;
                h.set(top(S[mt]), bottom(S[mt]));
                h.put(sSb + (MT * warp + mt) * 64 + lane);
            }
        }
    };
    if (owns) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    S[mt][nt][e] = p.S_in ? p.S_in[(head * D + srow(mt, nt) + (e & 1)) * D + c0 + gr +
                                                   8 * (e >> 1)]
                                          : 0.f;
        put_state();
    }
    // the next chunk's W and XV (chain) or M (outputs), as fragments
    constexpr int NW = D / 8 > 8 ? D / 8 : 8;
    float4 W[NW], Y0[2];
    const ptrdiff_t dir = REV ? -1 : 1;
    const float4 *wp = reinterpret_cast<const float4 *>(w.W + (ch0 + chunk_of(0)) * (kC * D)) +
                       (size_t)rw * (D / 8) * 32 + lane;
    const float4 *yp = reinterpret_cast<const float4 *>(w.Y + (ch0 + chunk_of(0)) * (kC * D)) +
                       (size_t)(rw * (D / 8) + slice * 2) * 32 + lane;
    const float4 *mp = reinterpret_cast<const float4 *>(w.M + (ch0 + chunk_of(0)) * (kC * kC)) +
                       (size_t)rw * 8 * 32 + lane;
    const int kts = 2 * (rw + 1);  // eights of M's columns up to the diagonal block
    auto load_frags = [&]() {
        if (chain) {
#pragma unroll
            for (int kt = 0; kt < D / 8; ++kt) W[kt] = wp[kt * 32];
#pragma unroll
            for (int h = 0; h < 2; ++h) Y0[h] = yp[h * 32];
            wp += dir * (kC * D / 4);
            yp += dir * (kC * D / 4);
        } else if (wantO) {
#pragma unroll
            for (int kt = 0; kt < 8; ++kt)
                if (kt < kts) W[kt] = mp[kt * 32];
            mp += kC * kC / 4;
        }
    };
    load_frags();
    __syncthreads();

    for (int i = 0; i < p.nc; ++i) {
        const int c = chunk_of(i);
        const uint8_t *st = sm + L::STAGE + (i % L::STAGES) * L::STAGE_BYTES;
        const Tin *sK = reinterpret_cast<const Tin *>(st + L::K);
        const Tin *sQ = reinterpret_cast<const Tin *>(st + L::Q);
        const Tin *sO = reinterpret_cast<const Tin *>(st + L::DO);
        const float *coef = reinterpret_cast<const float *>(st + L::COEF);
        float o[2][4];
        // sixteen of k of W's or M's 16 rows as B operands
        auto frag_w = [&](auto &b, int ks) {
            const float4 w0 = W[2 * ks], w1 = W[2 * ks + 1];
            b[0].set(make_float4(w0.x, w0.y, w1.x, w1.y));
            b[1].set(make_float4(w0.z, w0.w, w1.z, w1.w));
        };
        if (chain) {
            // E = XV - W S0 (REV: Z = Z0 + W' dS)
            float acc[2][4];
            clear(acc);
#pragma unroll
            for (int k0 = 0; k0 < D / 16; k0 += KP) {
                FragA<2> a[KP];
                FragB<2> b[KP][2];
#pragma unroll
                for (int s = 0; s < KP; ++s) {
                    get_frag(a[s], sS + (k0 + s) * 128 + lane);
                    frag_w(b[s], k0 + s);
                }
                mma_step<2, 2, 2, KP>(acc, a, b);
            }
            const float2 c0_ = *reinterpret_cast<const float2 *>(coef + kC + m0 + t2);
            const float2 c1_ = *reinterpret_cast<const float2 *>(coef + kC + m0 + t2 + 8);
            float4 y[2] = {top(acc), bottom(acc)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float sg = REV ? 1.f : -1.f;
                y[h] = make_float4(fmaf(sg, y[h].x, Y0[h].x), fmaf(sg, y[h].y, Y0[h].y),
                                   fmaf(sg, y[h].z, Y0[h].z), fmaf(sg, y[h].w, Y0[h].w));
            }
            auto times = [&](float4 x) {
                return make_float4(c0_.x * x.x, c0_.y * x.y, c1_.x * x.z, c1_.y * x.w);
            };
            if constexpr (CUT3) {
                PartsA<3> f;
                f.set(times(y[0]), times(y[1]));
                f.put(sCut + rw * 96 + lane);
            } else {
                sYc[rw * 64 + lane] = times(y[0]);
                sYc[rw * 64 + 32 + lane] = times(y[1]);
            }
            if (wantO) {
                if constexpr (TI == 1) {
                    PartsA<2> e;
                    e.set(y[0], y[1]);
                    e.put(sE + rw * 64 + lane);
                } else {
                    FragA<2> e;
                    e.set(y[0], y[1]);
                    put_frag(sE + rw * 128 + lane, e);
                }
            }
            if (KEEP) {
                float *d = p.keepY + ((ch0 + c) * kC + m0 + t2) * D + c0 + gr;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    d[8 * h] = y[h].x;
                    d[D + 8 * h] = y[h].y;
                    d[8 * D + 8 * h] = y[h].z;
                    d[9 * D + 8 * h] = y[h].w;
                }
            }
            if (i + 1 < p.nc) load_frags();
        } else if (wantO) {
            clear(o);
#pragma unroll 1
            for (int ks = 0; ks < D / 16; ++ks) {
                if constexpr (TI == 1) {
                    PartsA<2> a;
                    PartsB<1> b[2];
                    a.get(sSb + ks * 64 + lane);
                    const uint4 x = pairs<true>(sQ + m0 * KS, KS, 16 * ks);
                    b[0].set(make_uint2(x.x, x.y));
                    b[1].set(make_uint2(x.z, x.w));
                    mma_parts<1, 2>(o, a, b);
                } else {
                    FragA<2> a[1];
                    FragB<2> b[1][2];
                    get_frag(a[0], sS + ks * 128 + lane);
                    const Quads x = quads<true>(sQ + m0 * KS, KS, 16 * ks);
                    b[0][0].set(x.a);
                    b[0][1].set(x.b);
                    mma_step<2, 2, 2, 1>(o, a, b);
                }
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const float2 s = *reinterpret_cast<const float2 *>(coef + m0 + 8 * nt + t2);
                o[nt][0] *= s.x;
                o[nt][1] *= s.y;
                o[nt][2] *= s.x;
                o[nt][3] *= s.y;
            }
        } else if (REV) {
            for (int ms = rw; ms < D / 16; ms += 4) {
                float acc[2][4];
                clear(acc);
#pragma unroll 1
                for (int ks = 0; ks < kC / 16; ++ks) {
                    FragA<2> a[1];
                    FragB<TI> b[1][2];
                    const Quads x = quads<false>(sO, L::DS, 16 * ks);
                    a[0].set(scaled(x.a, coef, 16 * ks + t2), scaled(x.b, coef, 16 * ks + t2));
                    const Quads y = quads<false>(sQ + 16 * ms, KS, 16 * ks);
                    b[0][0].set(y.a);
                    b[0][1].set(y.b);
                    mma_step<2, TI, 2, 1>(acc, a, b);
                }
                sG[ms * 64 + lane] = top(acc);
                sG[ms * 64 + 32 + lane] = bottom(acc);
            }
        }
        __syncthreads();
        if (owns) {
            // S = a_C S + K^T (c' Y) (REV: + Q^T dO): the chunk's share is summed
            // by itself, then added, so that rounding does not grow with the chunks
            const float aC = coef[2 * kC];
            float acc[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) clear(acc[mt]);
#pragma unroll
            for (int k0 = 0; k0 < kC / 16; k0 += 2) {
                if constexpr (CUT3) {
                    uint4 a[2][3];
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int j = 0; j < 3; ++j) a[s][j] = sCut[(k0 + s) * 96 + 32 * j + lane];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint4 b[2];
                        float t[2][2][4];
#pragma unroll
                        for (int s = 0; s < 2; ++s)
                            b[s] = pairs<false>(sK + 16 * (MT * warp + mt), KS, 16 * (k0 + s));
#pragma unroll
                        for (int j = 2; j >= 0; --j)  // the small parts first
#pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                if (j == 2) {
                                    mma16_0(t[s][0], a[s][j], b[s].x, b[s].y);
                                    mma16_0(t[s][1], a[s][j], b[s].z, b[s].w);
                                } else {
                                    mma16(t[s][0], a[s][j], b[s].x, b[s].y);
                                    mma16(t[s][1], a[s][j], b[s].z, b[s].w);
                                }
                            }
#pragma unroll
                        for (int s = 0; s < 2; ++s)
#pragma unroll
                            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[mt][nt][e] += t[s][nt][e];
                    }
                } else {
                    FragA<2> a[2];
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        a[s].set(sYc[(k0 + s) * 64 + lane], sYc[(k0 + s) * 64 + 32 + lane]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        FragB<TI> b[2][2];
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const Quads x = quads<false>(sK + 16 * (MT * warp + mt), KS, 16 * (k0 + s));
                            b[s][0].set(x.a);
                            b[s][1].set(x.b);
                        }
                        mma_step<2, TI, 2, 2>(acc[mt], a, b);
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (KEEP) {  // the state before this chunk
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            p.keepS[((ch0 + c) * D + srow(mt, nt) + (e & 1)) * D + c0 + gr +
                                    8 * (e >> 1)] = S[mt][nt][e];
                }
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[mt][nt][e] = fmaf(aC, S[mt][nt][e], acc[mt][nt][e]);
                if (REV) {
                    const float4 *d = sG + (MT * warp + mt) * 64 + lane;
                    const float4 g0 = d[0], g1 = d[32];
                    S[mt][0][0] += g0.x, S[mt][0][1] += g0.y, S[mt][1][0] += g0.z, S[mt][1][1] += g0.w;
                    S[mt][0][2] += g1.x, S[mt][0][3] += g1.y, S[mt][1][2] += g1.z, S[mt][1][3] += g1.w;
                }
            }
            put_state();
        } else if (wantO && !chain) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                if (ks > rw) continue;
                if constexpr (TI == 1) {
                    PartsA<2> a;
                    PartsB<2> b[2];
                    a.get(sE + ks * 64 + lane);
                    const float4 w0 = W[2 * ks], w1 = W[2 * ks + 1];
                    b[0].p[0] = make_uint2(__float_as_uint(w0.x), __float_as_uint(w1.x));
                    b[0].p[1] = make_uint2(__float_as_uint(w0.y), __float_as_uint(w1.y));
                    b[1].p[0] = make_uint2(__float_as_uint(w0.z), __float_as_uint(w1.z));
                    b[1].p[1] = make_uint2(__float_as_uint(w0.w), __float_as_uint(w1.w));
                    mma_parts<2, 2>(o, a, b);
                } else {
                    FragA<2> a[1];
                    FragB<2> b[1][2];
                    get_frag(a[0], sE + ks * 128 + lane);
                    frag_w(b[0], ks);
                    mma_step<2, 2, 2, 1>(o, a, b);
                }
            }
            if (i + 1 < p.nc) load_frags();
            Tin *od = static_cast<Tin *>(p.o);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const int t = c * kC + m0 + 8 * nt + gr;
                Tin *d = od + (row0 + t) * (size_t)D + c0 + t2;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (sizeof(Tin) == 2) {
                        const __nv_bfloat162 x = __floats2bfloat162_rn(o[nt][2 * h], o[nt][2 * h + 1]);
                        const uint32_t y = transpose8(*reinterpret_cast<const uint32_t *>(&x));
                        if (t < p.T) *reinterpret_cast<uint32_t *>(d + 8 * h) = y;
                    } else {
                        const float2 y = transpose8(o[nt][2 * h], o[nt][2 * h + 1]);
                        if (t < p.T) *reinterpret_cast<float2 *>(d + 8 * h) = y;
                    }
                }
            }
        }
        __syncthreads();
    }
    if (owns && p.S_out) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    p.S_out[(head * D + srow(mt, nt) + (e & 1)) * D + c0 + gr + 8 * (e >> 1)] =
                        S[mt][nt][e];
    }
}

template <typename Tin, int D>
__global__ void __launch_bounds__(kChainThreads, 1) delta_chain(Args p, Scratch w) {
    sm100::grid_dependency_wait();  // delta_prep
    walk_chunks<Tin, D, false, false>(p, w, blockIdx.x);
}

// The gradients' two walks in one launch, the longer one's CTAs first: neither
// needs the other, and few heads leave most SMs idle (34 -> 20 us for both at
// B1 H6 T777 d32 fp32; no difference where either fills the GPU).
template <typename Tin, int D>
__global__ void __launch_bounds__(kChainThreads, 1)
    delta_walks(Args back, Scratch wb, Args forth, Scratch wf) {
    const unsigned half = gridDim.x / 2;
    sm100::grid_dependency_wait();  // delta_prep
    if (threadIdx.x == 0) sm100::launch_dependents();
    if (blockIdx.x < half)
        walk_chunks<Tin, D, true, true>(back, wb, blockIdx.x);
    else
        walk_chunks<Tin, D, false, true>(forth, wf, blockIdx.x - half);
}

template <typename Tin, int D, bool BACK>
cudaError_t launch_prep(const Args &p, const Scratch &f, const Scratch &r, long heads,
                        cudaStream_t stream) {
    constexpr int bytes = PrepSmem<Tin, D, BACK>::BYTES;
    static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
    cudaError_t e = tc::set_smem_once<delta_prep<Tin, D, BACK>>(bytes);
    if (e != cudaSuccess) return e;
    e = tc::launch_overlapped(delta_prep<Tin, D, BACK>, (unsigned)(heads * p.nc), 256, bytes, stream, p,
                              f, r);
    return e != cudaSuccess ? e : after_launch();
}

template <typename Tin, int D>
cudaError_t launch_chain(const Args &p, const Scratch &w, long heads, cudaStream_t stream) {
    constexpr int bytes = ChainSmem<Tin, D, false>::BYTES;
    static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
    cudaError_t e = tc::set_smem_once<delta_chain<Tin, D>>(bytes);
    if (e != cudaSuccess) return e;
    e = tc::launch_overlapped(delta_chain<Tin, D>, (unsigned)(heads * (D / kSlice)), kChainThreads, bytes,
                              stream, p, w);
    return e != cudaSuccess ? e : after_launch();
}

template <typename Tin, int D>
cudaError_t launch_walks(const Args &back, const Scratch &wb, const Args &forth, const Scratch &wf,
                         long heads, cudaStream_t stream) {
    constexpr int b0 = ChainSmem<Tin, D, true>::BYTES;
    constexpr int b1 = ChainSmem<Tin, D, false>::BYTES, bytes = b0 > b1 ? b0 : b1;
    static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
    cudaError_t e = tc::set_smem_once<delta_walks<Tin, D>>(bytes);
    if (e != cudaSuccess) return e;
    e = tc::launch_overlapped(delta_walks<Tin, D>, (unsigned)(2 * heads * (D / kSlice)), kChainThreads,
                              bytes, stream, back, wb, forth, wf);
    return e != cudaSuccess ? e : after_launch();
}

inline int chunks_of(int T) { return (T + kC - 1) / kC; }

}  // namespace delta
}  // namespace kata
