// Gradients of the gated delta rule's chunked prefill.
//
// With the chunk's quantities as in delta.cuh, U = diag(beta) E, dO the
// gradient of O and dS that of the chunk's last state:
//     dU = scale M^T dO + diag(c) K dS,    Z = X^T diag(beta) dU,
//     F  = dU - N^T Z  (so that Z = diag(beta) F)
//     dV = Z,   dbeta_i = E_i . F_i,
//     PM = scale tril(dO U^T) * D,   PN = -tril(Z U^T, -1) * D
//     dQ = PM K + scale diag(a) dO S0^T
//     dK = R + L,  R = PN K - diag(a) Z S0^T              (k_i as the reader)
//                  L = PM^T Q + PN^T K + diag(c) U dS^T   (k_j as the written key)
// and for the running sums G of the log decays, since each term carries
// exp(G_i - G_j) with i the reading and j the written token, with
// x_ij = PM_ij (q_i.k_j) + PN_ij (k_i.k_j) and w_j = k_j . (c_j U_j dS^T),
//     dG_i = sum_j x_ij - sum_j x_ji + scale a_i q_i.(S0 dO_i) - a_i k_i.(S0 Z_i) - w_i,
//     dg_t = sum_{i >= t in the chunk} dG_i + (a_C <S0, dS> + sum_j w_j).
//
// Three launches: delta_prep (the operands of both walks), delta_walks (the
// states and errors forwards, their gradients backwards), and delta_grad, one CTA
// per (chunk, head), for everything above. The states and errors of every chunk are
// kept in the workspace in fp32.
//
// delta_grad takes the value columns in slices of 32, so that d = 128 fits a
// CTA's shared memory, and sums the products over the columns in registers.
// 8 warps: row block warp % 4, and one half of the columns (of a 64 x 64
// product: every other 8 columns, so that the two halves of a triangular one
// have equal work). Products that share an operand go together. What dbeta and dg
// are made of is in two tf32 parts (mma_tf32.cuh); what only dQ and dK are made of
// (PM, PN, E, dS) is in two bf16 parts, 16 bits, for bf16 inputs, whose results are rounded
// to 8 bits next.
//
// Measured on B200 at B2 H16 T4096 d64 bf16, each by itself under ncu: delta_prep 93 us,
// delta_walks 150, delta_grad 196 (issue 52 %, tensor 38 %, shared memory 49 %, 16 warps per SM,
// their registers and 101 KB of shared memory per CTA in the way of more). Its two-way
// bank conflicts (transposed reads of fp32 tiles, a third of its wavefronts) cost
// nothing: without them it took as long.
#include "delta.cuh"

namespace kata {
namespace {

using namespace delta;

struct Grads {
    void *dq, *dk, *dv;
    float *dg, *dbeta;
    const float *E, *Z;   // [chunks][64][D]
    const float *S0, *dS; // [chunks][D][D]
};

template <typename Tin, int D>
struct GradSmem {
    static constexpr int SL = D < 32 ? D : 32;  // value columns per slice
    static constexpr int KS = row_stride<D>(), SS = SL + 8;
    static constexpr int IN = kC * KS * (int)sizeof(Tin);
    static constexpr int K = 0, Q = IN, DO = 2 * IN;
    static constexpr int E = DO + kC * SS * (int)sizeof(Tin), Z = E + kC * SS * 4;
    static constexpr int S0 = Z + kC * SS * 4, DS = S0 + D * SS * 4;
    static constexpr int M = DS + D * SS * 4, N = M + kC * kTS * 4;
    // beta, a, c, G (hi, lo); sums of column halves: dbeta, dG, w; column sums of x per row
    // block [4]; the chunk's sums per warp [8]
    static constexpr int VEC = N + kC * kTS * 4;
    static constexpr int BYTES = VEC + (15 * kC + 8) * 4;
};

template <typename Tin>
__device__ __forceinline__ void store2(Tin *d, float x, float y) {
    if constexpr (sizeof(Tin) == 2)
        *reinterpret_cast<__nv_bfloat162 *>(d) = __floats2bfloat162_rn(x, y);
    else
        *reinterpret_cast<float2 *>(d) = make_float2(x, y);
}

__device__ __forceinline__ float2 two(const float *p) { return *reinterpret_cast<const float2 *>(p); }
__device__ __forceinline__ float2 two(const __nv_bfloat16 *p) {
    return tf::unpack(*reinterpret_cast<const uint32_t *>(p));
}

template <typename Tin, int D>
__global__ void __launch_bounds__(256, D <= 64 ? 2 : 1) delta_grad(Args p, Grads gr_) {
    using namespace tf;
    using L = GradSmem<Tin, D>;
    constexpr int KS = L::KS, SS = L::SS, SL = L::SL, TI = Parts<Tin>::N;
    constexpr int NF = SL / 16;  // 8-column tiles of a slice per warp
    constexpr int ND = D / 16;   // 8-column tiles of d per warp
    extern __shared__ __align__(16) uint8_t sm[];
    Tin *sK = reinterpret_cast<Tin *>(sm + L::K), *sQ = reinterpret_cast<Tin *>(sm + L::Q);
    Tin *sO = reinterpret_cast<Tin *>(sm + L::DO);
    float *sE = reinterpret_cast<float *>(sm + L::E), *sZ = reinterpret_cast<float *>(sm + L::Z);
    float *sS0 = reinterpret_cast<float *>(sm + L::S0), *sDS = reinterpret_cast<float *>(sm + L::DS);
    float *sM = reinterpret_cast<float *>(sm + L::M), *sN = reinterpret_cast<float *>(sm + L::N);
    float *beta = reinterpret_cast<float *>(sm + L::VEC), *ca = beta + kC, *cc = ca + kC;
    float *ghi = cc + kC, *glo = ghi + kC;
    float *sdb = glo + kC, *sdG = sdb + 2 * kC, *sw = sdG + 2 * kC;
    float *sx = sw + 2 * kC, *send = sx + 4 * kC;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, t2 = 2 * (lane & 3);
    const int rb = warp & 3, hf = warp >> 2, m0 = 16 * rb;
    const size_t ch = blockIdx.x, head = ch / p.nc;
    const int t0 = (int)(ch % p.nc) * kC;
    const size_t row0 = head * (size_t)p.T;

    auto load_slice = [&](int c0) {
        load_tile<Tin, SL, 256>(sO, SS, static_cast<const Tin *>(p.d_o), row0, t0, p.T, D, c0, tid);
        load_tile<float, SL, 256>(sE, SS, gr_.E, ch * kC, 0, kC, D, c0, tid);
        load_tile<float, SL, 256>(sZ, SS, gr_.Z, ch * kC, 0, kC, D, c0, tid);
        load_tile<float, SL, 256, D>(sS0, SS, gr_.S0, ch * D, 0, D, D, c0, tid);
        load_tile<float, SL, 256, D>(sDS, SS, gr_.dS, ch * D, 0, D, D, c0, tid);
        cp_commit();
    };
    float2 v2 = make_float2(0.f, 0.f);
    if (warp == 0) v2 = load_decays(p.g, row0, t0, p.T);
    load_tile<Tin, D, 256>(sK, KS, static_cast<const Tin *>(p.k), row0, t0, p.T, D, 0, tid);
    load_tile<Tin, D, 256>(sQ, KS, static_cast<const Tin *>(p.q), row0, t0, p.T, D, 0, tid);
    sm100::grid_dependency_wait();  // delta_walks
    load_slice(0);
    if (warp == 0) cumulate(v2, ghi, glo);
    if (tid >= 192) {
        const int t = t0 + tid - 192;
        beta[tid - 192] = t < p.T ? p.beta[row0 + t] : 0.f;
    }
    cp_wait_all();
    __syncthreads();
    if (tid < kC) {
        ca[tid] = exp2f(ghi[tid] + glo[tid]);
        cc[tid] = exp2f((ghi[kC - 1] - ghi[tid]) + (glo[kC - 1] - glo[tid]));
    }
    // this warp's tiles of a 64 x 64 product: columns 8 (2 nt + hf), up to the diagonal block
    const int nt_end = rb + 1;
    auto col = [&](int nt, int e) { return 8 * (2 * nt + hf) + t2 + (e & 1); };
    auto row = [&](int e) { return m0 + gr + (e & 2 ? 8 : 0); };
    {
        float kk[4][4], qk[4][4];
        clear(kk);
        clear(qk);
        grams(kk, qk, true, sK + m0 * KS, sQ + m0 * KS, sK, KS, 8 * hf, D / 16, nt_end);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            if (nt >= nt_end) continue;
            const int j = col(nt, 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = row(2 * h);
                const float2 dec = decay2(ghi[i], glo[i], ghi, glo, j);
                *reinterpret_cast<float2 *>(sN + i * kTS + j) =
                    make_float2(i > j ? kk[nt][2 * h] * dec.x : 0.f,
                                i > j + 1 ? kk[nt][2 * h + 1] * dec.y : 0.f);
                *reinterpret_cast<float2 *>(sM + i * kTS + j) =
                    make_float2(i >= j ? qk[nt][2 * h] * dec.x : 0.f,
                                i >= j + 1 ? qk[nt][2 * h + 1] * dec.y : 0.f);
            }
        }
    }
    __syncthreads();

    float pm[4][4], pn[4][4], dq[ND][4], dr[ND][4], dl[ND][4];
    clear(pm);
    clear(pn);
    clear(dq);
    clear(dr);
    clear(dl);
    float db[2] = {0.f, 0.f}, w[2] = {0.f, 0.f}, end = 0.f;  // rows gr, gr + 8
    const float aC = ca[kC - 1];
    const int d0 = hf * (D / 2);  // this warp's columns of a [64, D] product
    for (int c0 = 0; c0 < D; c0 += SL) {
        if (c0 > 0) {
            __syncthreads();
            load_slice(c0);
            cp_wait_all();
            __syncthreads();
        }
        {  // F, and what it gives: dbeta, and the written keys' share of the decay
            const int f0 = hf * (SL / 2);
            float md[NF][4], kd[NF][4];
            clear(md);
            clear(kd);
            gemm<2, TI, NF>(
                md, rb, 4, [&](int m, int k) { return quad<false>(sM + m0, kTS, m, k); },
                [&](int n, int k) { return quad<false>(sO + f0, SS, n, k); });
#pragma unroll
            for (int nt = 0; nt < NF; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) md[nt][e] *= -p.scale;
            gemm<2, 2, NF>(
                md, rb, 4, [&](int m, int k) { return quad<false>(sN + m0, kTS, m, k); },
                [&](int n, int k) { return quad<false>(sZ + f0, SS, n, k); });
            gemm<TI, 2, NF>(
                kd, 0, D / 16, [&](int m, int k) { return quad<true>(sK + m0 * KS, KS, m, k); },
                [&](int n, int k) { return quad<false>(sDS + f0, SS, n, k); });
#pragma unroll
            for (int nt = 0; nt < NF; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = row(e);
                    const float E = sE[i * SS + f0 + 8 * nt + t2 + (e & 1)];
                    const float ckd = cc[i] * kd[nt][e];
                    db[e >> 1] = fmaf(E, ckd - md[nt][e], db[e >> 1]);
                    w[e >> 1] = fmaf(beta[i] * E, ckd, w[e >> 1]);
                }
        }
        for (int i = tid; i < D * SL; i += 256) {
            const int at = (i / SL) * SS + i % SL;
            end = fmaf(aC * sS0[at], sDS[at], end);
        }
#pragma unroll 1
        for (int ks = 0; ks < SL / 16; ++ks) {  // dO and Z against U's rows and S0's
            const int k = 16 * ks + t2;
            FragA<TI> ao[1];
            FragA<2> az[1];
            ao[0].set(quad<true>(sO + m0 * SS, SS, gr, k), quad<true>(sO + m0 * SS, SS, gr + 8, k));
            az[0].set(quad<true>(sZ + m0 * SS, SS, gr, k), quad<true>(sZ + m0 * SS, SS, gr + 8, k));
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                if (nt >= nt_end) continue;
                const int j = 8 * (2 * nt + hf) + gr;
                const float4 x = quad<true>(sE, SS, j, k);
                FragB<2> b[1][1];
                b[0][0].set(make_float4(beta[j] * x.x, beta[j] * x.y, beta[j] * x.z, beta[j] * x.w));
                mma_step<TI, 2, 1, 1>(*reinterpret_cast<float(*)[1][4]>(&pm[nt]), ao, b);
                mma_step<2, 2, 1, 1>(*reinterpret_cast<float(*)[1][4]>(&pn[nt]), az, b);
            }
#pragma unroll
            for (int nt = 0; nt < ND; ++nt) {
                FragB<2> b[1][1];
                b[0][0].set(quad<true>(sS0 + d0 * SS, SS, 8 * nt + gr, k));
                mma_step<TI, 2, 1, 1>(*reinterpret_cast<float(*)[1][4]>(&dq[nt]), ao, b);
                mma_step<2, 2, 1, 1>(*reinterpret_cast<float(*)[1][4]>(&dr[nt]), az, b);
            }
        }
        auto erows = [&](int m, int k) { return quad<true>(sE + m0 * SS, SS, m, k); };
        auto srows = [&](int n, int k) { return quad<true>(sDS + d0 * SS, SS, n, k); };
        if constexpr (TI == 1)
            gemm_parts<2, ND>(dl, 0, SL / 16, erows, srows);
        else
            gemm<2, 2, ND>(dl, 0, SL / 16, erows, srows);
        Tin *dv = static_cast<Tin *>(gr_.dv);
        for (int i = tid; i < kC * SL / 2; i += 256) {
            const int r = i / (SL / 2), c = 2 * (i % (SL / 2));
            if (t0 + r < p.T)
                store2(dv + (row0 + t0 + r) * (size_t)D + c0 + c, sZ[r * SS + c], sZ[r * SS + c + 1]);
        }
    }
    // x, its sums over rows and columns, and PM and PN in the places of M and N (each
    // thread overwrites the values that it alone reads here)
    __syncthreads();
    float dG[2] = {0.f, 0.f};
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        if (nt >= nt_end) continue;
        const int j = col(nt, 0);
        float2 cs = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = row(2 * h);
            const float2 dec = decay2(ghi[i], glo[i], ghi, glo, j);
            float2 *pM = reinterpret_cast<float2 *>(sM + i * kTS + j);
            float2 *pN = reinterpret_cast<float2 *>(sN + i * kTS + j);
            const float2 m = *pM, n = *pN;  // zero above the diagonal
            const float m0_ = p.scale * pm[nt][2 * h], m1_ = p.scale * pm[nt][2 * h + 1];
            const float x0 = m0_ * m.x - pn[nt][2 * h] * n.x, x1 = m1_ * m.y - pn[nt][2 * h + 1] * n.y;
            dG[h] += x0 + x1;
            cs.x += x0;
            cs.y += x1;
            *pM = make_float2(i >= j ? m0_ * dec.x : 0.f, i >= j + 1 ? m1_ * dec.y : 0.f);
            *pN = make_float2(i > j ? -pn[nt][2 * h] * dec.x : 0.f,
                              i > j + 1 ? -pn[nt][2 * h + 1] * dec.y : 0.f);
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            cs.x += __shfl_xor_sync(0xffffffffu, cs.x, off);
            cs.y += __shfl_xor_sync(0xffffffffu, cs.y, off);
        }
        if (gr == 0) *reinterpret_cast<float2 *>(sx + rb * kC + j) = cs;
    }
#pragma unroll
    for (int nt = 0; nt < ND; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = m0 + gr + 8 * h, n = d0 + 8 * nt + t2;
            const float2 kx = two(sK + i * KS + n), qx = two(sQ + i * KS + n);
            const float sa = p.scale * ca[i], bc = beta[i] * cc[i];
            float *q2 = &dq[nt][2 * h], *r2 = &dr[nt][2 * h], *l2 = &dl[nt][2 * h];
            q2[0] *= sa;
            q2[1] *= sa;
            r2[0] *= -ca[i];
            r2[1] *= -ca[i];
            dG[h] = fmaf(qx.x, q2[0], fmaf(qx.y, q2[1], dG[h]));
            dG[h] = fmaf(kx.x, r2[0], fmaf(kx.y, r2[1], dG[h]));
            r2[0] = fmaf(bc, l2[0], r2[0]);  // from here on dK
            r2[1] = fmaf(bc, l2[1], r2[1]);
        }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        end += w[h];
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            dG[h] += __shfl_xor_sync(0xffffffffu, dG[h], off);
            db[h] += __shfl_xor_sync(0xffffffffu, db[h], off);
            w[h] += __shfl_xor_sync(0xffffffffu, w[h], off);
        }
        if ((lane & 3) == 0) {
            sdG[hf * kC + m0 + gr + 8 * h] = dG[h];
            sdb[hf * kC + m0 + gr + 8 * h] = db[h];
            sw[hf * kC + m0 + gr + 8 * h] = w[h];
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) end += __shfl_xor_sync(0xffffffffu, end, off);
    if (lane == 0) send[warp] = end;
    __syncthreads();
#pragma unroll 1
    for (int ks = 0; ks < nt_end; ++ks) {  // PM and PN against K
        const int k = 16 * ks + t2;
        const float4 mt = quad<true>(sM + m0 * kTS, kTS, gr, k), mb = quad<true>(sM + m0 * kTS, kTS, gr + 8, k);
        const float4 nt_ = quad<true>(sN + m0 * kTS, kTS, gr, k), nb = quad<true>(sN + m0 * kTS, kTS, gr + 8, k);
        if constexpr (TI == 1) {
            PartsA<2> am, an;
            am.set(mt, mb);
            an.set(nt_, nb);
#pragma unroll
            for (int nt = 0; nt < ND; ++nt) {
                PartsB<1> b[1];
                b[0].set(pair<false>(sK + d0, KS, 8 * nt + gr, k));
                mma_parts<1, 1>(*reinterpret_cast<float(*)[1][4]>(&dq[nt]), am, b);
                mma_parts<1, 1>(*reinterpret_cast<float(*)[1][4]>(&dr[nt]), an, b);
            }
        } else {
            FragA<2> am[1], an[1];
            am[0].set(mt, mb);
            an[0].set(nt_, nb);
#pragma unroll
            for (int nt = 0; nt < ND; ++nt) {
                FragB<2> b[1][1];
                b[0][0].set(quad<false>(sK + d0, KS, 8 * nt + gr, k));
                mma_step<2, 2, 1, 1>(*reinterpret_cast<float(*)[1][4]>(&dq[nt]), am, b);
                mma_step<2, 2, 1, 1>(*reinterpret_cast<float(*)[1][4]>(&dr[nt]), an, b);
            }
        }
    }
    auto mcols = [&](int m, int k) { return quad<false>(sM + m0, kTS, m, k); };
    auto ncols = [&](int m, int k) { return quad<false>(sN + m0, kTS, m, k); };
    if constexpr (TI == 1) {
        gemm_parts<1, ND>(dr, rb, 4, mcols,
                          [&](int n, int k) { return pair<false>(sQ + d0, KS, n, k); });
        gemm_parts<1, ND>(dr, rb, 4, ncols,
                          [&](int n, int k) { return pair<false>(sK + d0, KS, n, k); });
    } else {
        gemm<2, 2, ND>(dr, rb, 4, mcols, [&](int n, int k) { return quad<false>(sQ + d0, KS, n, k); });
        gemm<2, 2, ND>(dr, rb, 4, ncols, [&](int n, int k) { return quad<false>(sK + d0, KS, n, k); });
    }
#pragma unroll
    for (int nt = 0; nt < ND; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = m0 + gr + 8 * h;
            if (t0 + i >= p.T) continue;
            const size_t at = (row0 + t0 + i) * (size_t)D + d0 + 8 * nt + t2;
            store2(static_cast<Tin *>(gr_.dq) + at, dq[nt][2 * h], dq[nt][2 * h + 1]);
            store2(static_cast<Tin *>(gr_.dk) + at, dr[nt][2 * h], dr[nt][2 * h + 1]);
        }
    if (warp == 0) {  // dg: sums from each token to the chunk's end, two tokens per lane
        double tail = 0.0;
        for (int w = 0; w < 8; ++w) tail += send[w];
        const int i = 2 * lane;
        double x0 = (double)sdG[i] + sdG[kC + i] - sw[i] - sw[kC + i];
        double x1 = (double)sdG[i + 1] + sdG[kC + i + 1] - sw[i + 1] - sw[kC + i + 1];
        for (int b = i / 16; b < 4; ++b) {  // the row blocks that see column i
            x0 -= sx[b * kC + i];
            x1 -= sx[b * kC + i + 1];
        }
        double sum = x0 + x1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double up = __shfl_down_sync(0xffffffffu, sum, off);
            if (lane + off < 32) sum += up;
        }
        if (t0 + i < p.T) gr_.dg[row0 + t0 + i] = (float)(sum + tail);
        if (t0 + i + 1 < p.T) gr_.dg[row0 + t0 + i + 1] = (float)(sum - x0 + tail);
    } else if (tid >= 64 && tid < 128) {
        const int i = tid - 64;
        if (t0 + i < p.T) gr_.dbeta[row0 + t0 + i] = sdb[i] + sdb[kC + i];
    }
}

// floats of scratch per chunk: the two walks' operands, what they keep
constexpr size_t chunk_floats(int d) {
    return 6 * (size_t)kC * d + 2 * (size_t)d * d + 2 * kCoef;
}

template <typename Tin, int D>
cudaError_t backward_d(const DeltaArgs &a, const DeltaGrads &g, cudaStream_t stream) {
    const int nc = chunks_of(a.T);
    const size_t chunks = (size_t)a.heads * nc, mat = chunks * kC * D, st = chunks * D * D;
    float *ws = static_cast<float *>(a.ws);
    const Scratch f{ws, ws + mat, nullptr, ws + 6 * mat + 2 * st};
    const Scratch r{ws + 2 * mat, ws + 3 * mat, nullptr, ws + 6 * mat + 2 * st + chunks * kCoef};
    float *E = ws + 4 * mat, *Z = ws + 5 * mat, *S0 = ws + 6 * mat, *dS = S0 + st;

    Args p{};
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.d_o = g.d_o;
    p.g = a.g;
    p.beta = a.beta;
    p.T = a.T;
    p.nc = nc;
    p.scale = a.scale;
    cudaError_t e = launch_prep<Tin, D, true>(p, f, r, a.heads, stream);
    if (e != cudaSuccess) return e;
    Args fw = p;
    fw.S_in = a.S_in;
    fw.keepY = E;
    fw.keepS = S0;
    Args bw = p;
    bw.S_in = g.dS_out;
    bw.S_out = g.dS_in;
    bw.keepY = Z;
    bw.keepS = dS;
    if ((e = launch_walks<Tin, D>(bw, r, fw, f, a.heads, stream)) != cudaSuccess) return e;

    constexpr int bytes = GradSmem<Tin, D>::BYTES;
    static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
    if ((e = tc::set_smem_once<delta_grad<Tin, D>>(bytes)) != cudaSuccess) return e;
    e = tc::launch_overlapped(delta_grad<Tin, D>, (unsigned)chunks, 256, bytes, stream, p,
                              Grads{g.dq, g.dk, g.dv, g.dg, g.dbeta, E, Z, S0, dS});
    return e != cudaSuccess ? e : after_launch();
}

template <typename Tin>
cudaError_t backward_t(const DeltaArgs &a, const DeltaGrads &g, cudaStream_t stream) {
    switch (a.d) {
        case 16: return backward_d<Tin, 16>(a, g, stream);
        case 32: return backward_d<Tin, 32>(a, g, stream);
        case 64: return backward_d<Tin, 64>(a, g, stream);
        case 128: return backward_d<Tin, 128>(a, g, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

size_t delta_backward_workspace_bytes(long heads, int T, int d) {
    return (size_t)heads * delta::chunks_of(T) * chunk_floats(d) * sizeof(float);
}

cudaError_t delta_backward(const DeltaArgs &a, const DeltaGrads &g, cudaStream_t stream) {
    return a.dtype == 0 ? backward_t<float>(a, g, stream) : backward_t<__nv_bfloat16>(a, g, stream);
}

}  // namespace kata
