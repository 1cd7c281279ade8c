// Gradients of the causal kernelized prefill from a zero state,
//     o_i = sum_{j<=i} s_ij^2 v_j / den_i,   s_ij = q_i.k_j,
//     den_i = sum_{j<=i} s_ij^2 + eps
// ("Kernelized Linear Attention: Breaking the Capacity Wall with Symmetric
// Cones", s2.2: the quadratic form). With dP_ij = dO_i.v_j and
// delta_i = dO_i.o_i = sum_j s_ij^2 dP_ij / den_i:
//     dS_ij = 2 s_ij (dP_ij - delta_i) / den_i
//     dQ_i = sum_j dS_ij k_j,  dK_j = sum_i dS_ij q_i,  dV_j = sum_i (s_ij^2 / den_i) dO_i.
// The weights are recomputed from q and k tile by tile, and delta from the
// inputs (o is not needed), so nothing is kept from the forward pass. Work is
// quadratic in T. Each sum is owned by one CTA: no atomics, the same bits on
// every run.
//
// This file: fp32 inputs, and bf16 inputs of any d, in split-tf32 products
// (mma_tf32.cuh), which keep fp32 accuracy. Two launches: bwd_query (one CTA
// per 64 queries: den and delta over the keys, then dQ) and bwd_key (one CTA
// per 64 keys: dK, dV). bwd_query leaves den and delta of every row for
// bwd_key.
//
// Rows with few keys need care: there delta_i is nearly dP_ij (row 0 has
// dP - delta = dP eps / den), and a score near zero enters as 1 / s^3. So delta
// is kept as two floats (hi + lo: dP - hi is exact when the two are close, and
// only then does lo matter) and summed in 64 bits, and the first tile's
// scores and dP (queries and keys 0 .. 63) are formed in 64 bits, the same in
// both kernels. From row 64 on, a row's den is a sum over more than 64 keys.
#include "delta.cuh"

namespace kata {
namespace {

using namespace tf;
using delta::cp_commit;
using delta::cp_wait_all;
using delta::load_tile;

constexpr int kB = 64;    // rows per tile
constexpr int kTS = 72;   // row stride of a 64 x 64 tile
constexpr int kThreads = 256;

struct Args {
    const void *q, *k, *v, *d_o;
    void *dq, *dk, *dv;
    float4 *stat;  // [heads * T]: 1 / den, 2 / den, delta hi, delta lo
    int T, nt;     // tokens, tiles per head
    float eps;
};

template <typename Tin, int D>
struct BwdSmem {
    static constexpr int RS = D + 8;
    static constexpr int IN = kB * RS * (int)sizeof(Tin);
    static constexpr int A0 = 0, A1 = IN;      // the CTA's own rows: q, dO or k, v
    static constexpr int B0 = 2 * IN;          // two stages of the other side's two tiles
    static constexpr int DS = 6 * IN;          // 64 x 64 products
    static constexpr int P = DS + kB * kTS * 4;
    static constexpr int STAT = P + kB * kTS * 4;  // bwd_key: two stages of 64 float4
    static constexpr int RED = STAT + 2 * kB * 16;  // bwd_query: row sums of two column halves
    static constexpr int BYTES = RED + 4 * kB * 8;
};

// s and dP of the first tile in 64 bits: rows of query side tiles q, o against
// key side tiles k, v.
template <typename Tin, int D>
__device__ __forceinline__ void dots64(const Tin *q, const Tin *o, const Tin *k, const Tin *v, int i,
                                       int j, double &s, double &dp) {
    constexpr int RS = BwdSmem<Tin, D>::RS;
    s = dp = 0.0;
    for (int c = 0; c < D; ++c) {
        s = fma((double)to_f32(q[i * RS + c]), (double)to_f32(k[j * RS + c]), s);
        dp = fma((double)to_f32(o[i * RS + c]), (double)to_f32(v[j * RS + c]), dp);
    }
}

template <typename Tin>
__device__ __forceinline__ void store2(Tin *d, float x, float y) {
    if constexpr (sizeof(Tin) == 2)
        *reinterpret_cast<__nv_bfloat162 *>(d) = __floats2bfloat162_rn(x, y);
    else
        *reinterpret_cast<float2 *>(d) = make_float2(x, y);
}

// out[rows m0 .., columns d0 ..] of a [64, D] tile of a [T, D] matrix
template <typename Tin, int D>
__device__ __forceinline__ void store_rows(void *dst, size_t row0, int t0, int T,
                                           const float (&acc)[D / 16][4], int m0, int d0, int gr,
                                           int t2) {
    Tin *o = static_cast<Tin *>(dst);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int t = t0 + m0 + gr + 8 * h;
        if (t >= T) continue;
#pragma unroll
        for (int nt = 0; nt < D / 16; ++nt)
            store2(o + (row0 + t) * (size_t)D + d0 + 8 * nt + t2, acc[nt][2 * h],
                   acc[nt][2 * h + 1]);
    }
}

// One CTA per (head, 64 queries). Two walks over the key tiles up to the
// diagonal: den and delta, then dQ. 8 warps: 16 rows (warp % 4) and half the
// columns each.
template <typename Tin, int D>
__global__ void __launch_bounds__(kThreads) bwd_query(Args p) {
    using L = BwdSmem<Tin, D>;
    constexpr int RS = L::RS, TI = Parts<Tin>::N;
    extern __shared__ __align__(16) uint8_t sm[];
    Tin *sQ = reinterpret_cast<Tin *>(sm + L::A0), *sO = reinterpret_cast<Tin *>(sm + L::A1);
    float *sDS = reinterpret_cast<float *>(sm + L::DS);
    double *red = reinterpret_cast<double *>(sm + L::RED);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, t2 = 2 * (lane & 3);
    const int m0 = 16 * (warp & 3), hf = warp >> 2, n0 = 32 * hf;
    const size_t head = blockIdx.x / p.nt;
    const int qt = p.nt - 1 - (int)(blockIdx.x % p.nt);  // the longest rows first
    const size_t row0 = head * (size_t)p.T;
    const int steps = 2 * (qt + 1);  // key tiles 0 .. qt, twice

    auto tileK = [&](int u) { return reinterpret_cast<Tin *>(sm + L::B0 + (u & 1) * 2 * L::IN); };
    auto tileV = [&](int u) { return tileK(u) + kB * RS; };
    auto prefetch = [&](int u) {
        const int t = (u % (qt + 1)) * kB;
        load_tile<Tin, D, kThreads>(tileK(u), RS, static_cast<const Tin *>(p.k), row0, t, p.T, D, 0, tid);
        load_tile<Tin, D, kThreads>(tileV(u), RS, static_cast<const Tin *>(p.v), row0, t, p.T, D, 0, tid);
        cp_commit();
    };
    load_tile<Tin, D, kThreads>(sQ, RS, static_cast<const Tin *>(p.q), row0, qt * kB, p.T, D, 0, tid);
    load_tile<Tin, D, kThreads>(sO, RS, static_cast<const Tin *>(p.d_o), row0, qt * kB, p.T, D, 0, tid);
    prefetch(0);
    cp_wait_all();
    __syncthreads();

    double den[2] = {0.0, 0.0}, num[2] = {0.0, 0.0};  // rows gr, gr + 8
    double d64[2], del64[2];
    float inv2[2], dhi[2], dlo[2];
    float dq[D / 16][4];
    clear(dq);
    for (int u = 0; u < steps; ++u) {
        if (u + 1 < steps) prefetch(u + 1);
        const int kt = u % (qt + 1);
        const bool second = u > qt;
        const Tin *k = tileK(u), *v = tileV(u);
        if (u == qt + 1) {  // the rows' sums are complete: join the lanes, then the column halves
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int off = 1; off < 4; off <<= 1) {
                    den[h] += __shfl_xor_sync(0xffffffffu, den[h], off);
                    num[h] += __shfl_xor_sync(0xffffffffu, num[h], off);
                }
                if ((lane & 3) == 0) {
                    red[hf * 2 * kB + m0 + gr + 8 * h] = den[h];
                    red[hf * 2 * kB + kB + m0 + gr + 8 * h] = num[h];
                }
            }
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = m0 + gr + 8 * h;
                d64[h] = red[i] + red[2 * kB + i] + (double)p.eps;
                del64[h] = d64[h] == 0.0 ? 0.0 : (red[kB + i] + red[3 * kB + i]) / d64[h];
                inv2[h] = d64[h] == 0.0 ? 0.f : (float)(2.0 / d64[h]);
                dhi[h] = (float)del64[h];
                dlo[h] = (float)(del64[h] - (double)dhi[h]);
                if (hf == 0 && (lane & 3) == 0 && qt * kB + i < p.T)
                    p.stat[row0 + qt * kB + i] = make_float4(0.5f * inv2[h], inv2[h], dhi[h], dlo[h]);
            }
        }
        float s[4][4], dp[4][4];
        if (kt == 0 && qt == 0) {
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int h = e >> 1, i = m0 + gr + 8 * h, j = n0 + 8 * nt + t2 + (e & 1);
                    double s64 = 0.0, dp64 = 0.0;
                    if (j <= i) dots64<Tin, D>(sQ, sO, k, v, i, j, s64, dp64);
                    if (!second) {
                        den[h] = fma(s64, s64, den[h]);
                        num[h] = fma(s64 * s64, dp64, num[h]);
                    } else {
                        s[nt][e] = d64[h] == 0.0
                                       ? 0.f
                                       : (float)(2.0 * s64 * (dp64 - del64[h]) / d64[h]);
                    }
                }
        } else {
            clear(s);
            clear(dp);
            auto qa = [&](int m, int kk) { return quad<true, true>(sQ + m0 * RS, RS, m, kk); };
            auto oa = [&](int m, int kk) { return quad<true, true>(sO + m0 * RS, RS, m, kk); };
            gemm<TI, TI, 4, true>(s, 0, D / 16, qa,
                            [&](int n, int kk) { return quad<true, true>(k + n0 * RS, RS, n, kk); });
            gemm<TI, TI, 4, true>(dp, 0, D / 16, oa,
                            [&](int n, int kk) { return quad<true, true>(v + n0 * RS, RS, n, kk); });
            float ds[2] = {0.f, 0.f}, ns[2] = {0.f, 0.f};
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int h = e >> 1, i = m0 + gr + 8 * h, j = n0 + 8 * nt + t2 + (e & 1);
                    const bool seen = kt < qt || j <= i;
                    if (!second) {
                        const float w = seen ? s[nt][e] * s[nt][e] : 0.f;
                        ds[h] += w;
                        ns[h] = fmaf(w, seen ? dp[nt][e] : 0.f, ns[h]);
                    } else {
                        s[nt][e] =
                            seen ? inv2[h] * s[nt][e] * ((dp[nt][e] - dhi[h]) - dlo[h]) : 0.f;
                    }
                }
            if (!second) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    den[h] += (double)ds[h];
                    num[h] += (double)ns[h];
                }
            }
        }
        if (second) {
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2 *>(sDS + (m0 + gr + 8 * h) * kTS + n0 + 8 * nt + t2) =
                        make_float2(s[nt][2 * h], s[nt][2 * h + 1]);
            __syncthreads();
            const int d0 = hf * (D / 2);
            gemm<2, TI, D / 16, false>(
                dq, 0, kB / 16, [&](int m, int kk) { return quad<true, false>(sDS + m0 * kTS, kTS, m, kk); },
                [&](int n, int kk) { return quad<false, false>(k + d0, RS, n, kk); });
        }
        cp_wait_all();
        __syncthreads();
    }
    store_rows<Tin, D>(p.dq, row0, qt * kB, p.T, dq, m0, hf * (D / 2), gr, t2);
}

// One CTA per (head, 64 keys): the query tiles from the diagonal on. Rows of
// its 64 x 64 tiles are keys: s^T = K Q^T, dP^T = V dO^T.
template <typename Tin, int D>
__global__ void __launch_bounds__(kThreads) bwd_key(Args p) {
    using L = BwdSmem<Tin, D>;
    constexpr int RS = L::RS, TI = Parts<Tin>::N;
    extern __shared__ __align__(16) uint8_t sm[];
    Tin *sK = reinterpret_cast<Tin *>(sm + L::A0), *sV = reinterpret_cast<Tin *>(sm + L::A1);
    float *sDS = reinterpret_cast<float *>(sm + L::DS), *sP = reinterpret_cast<float *>(sm + L::P);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, t2 = 2 * (lane & 3);
    const int m0 = 16 * (warp & 3), hf = warp >> 2, n0 = 32 * hf;
    const size_t head = blockIdx.x / p.nt;
    const int kt = (int)(blockIdx.x % p.nt);  // the keys that most queries see first
    const size_t row0 = head * (size_t)p.T;

    auto tileQ = [&](int u) { return reinterpret_cast<Tin *>(sm + L::B0 + (u & 1) * 2 * L::IN); };
    auto tileO = [&](int u) { return tileQ(u) + kB * RS; };
    auto stats = [&](int u) { return reinterpret_cast<float4 *>(sm + L::STAT) + (u & 1) * kB; };
    auto prefetch = [&](int u) {
        load_tile<Tin, D, kThreads>(tileQ(u), RS, static_cast<const Tin *>(p.q), row0, u * kB, p.T, D, 0, tid);
        load_tile<Tin, D, kThreads>(tileO(u), RS, static_cast<const Tin *>(p.d_o), row0, u * kB, p.T, D, 0, tid);
        if (tid < kB) {
            const bool have = u * kB + tid < p.T;
            delta::cp16(stats(u) + tid, p.stat + row0 + (have ? u * kB + tid : 0), have);
        }
        cp_commit();
    };
    load_tile<Tin, D, kThreads>(sK, RS, static_cast<const Tin *>(p.k), row0, kt * kB, p.T, D, 0, tid);
    load_tile<Tin, D, kThreads>(sV, RS, static_cast<const Tin *>(p.v), row0, kt * kB, p.T, D, 0, tid);
    prefetch(kt);
    cp_wait_all();
    __syncthreads();

    float dk[D / 16][4], dv[D / 16][4];
    clear(dk);
    clear(dv);
    const int d0 = hf * (D / 2);
    for (int u = kt; u < p.nt; ++u) {
        if (u + 1 < p.nt) prefetch(u + 1);
        const Tin *q = tileQ(u), *o = tileO(u);
        const float4 *st = stats(u);
        float s[4][4], dp[4][4];
        if (u == 0) {
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = m0 + gr + (e & 2 ? 8 : 0), i = n0 + 8 * nt + t2 + (e & 1);
                    const float4 t = st[i];
                    double s64 = 0.0, dp64 = 0.0;
                    if (j <= i) dots64<Tin, D>(q, o, sK, sV, i, j, s64, dp64);
                    dp[nt][e] = (float)(s64 * s64 * (double)t.x);
                    s[nt][e] = (float)((double)t.y * s64 * ((dp64 - (double)t.z) - (double)t.w));
                }
        } else {
            clear(s);
            clear(dp);
            gemm<TI, TI, 4, true>(
                s, 0, D / 16, [&](int m, int kk) { return quad<true, true>(sK + m0 * RS, RS, m, kk); },
                [&](int n, int kk) { return quad<true, true>(q + n0 * RS, RS, n, kk); });
            gemm<TI, TI, 4, true>(
                dp, 0, D / 16, [&](int m, int kk) { return quad<true, true>(sV + m0 * RS, RS, m, kk); },
                [&](int n, int kk) { return quad<true, true>(o + n0 * RS, RS, n, kk); });
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = m0 + gr + (e & 2 ? 8 : 0), i = n0 + 8 * nt + t2 + (e & 1);
                    const bool seen = u > kt || j <= i;
                    const float4 t = st[i];
                    const float x = s[nt][e];
                    s[nt][e] = seen ? t.y * x * ((dp[nt][e] - t.z) - t.w) : 0.f;
                    dp[nt][e] = seen ? x * x * t.x : 0.f;
                }
        }
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = (m0 + gr + 8 * h) * kTS + n0 + 8 * nt + t2;
                *reinterpret_cast<float2 *>(sDS + at) = make_float2(s[nt][2 * h], s[nt][2 * h + 1]);
                *reinterpret_cast<float2 *>(sP + at) = make_float2(dp[nt][2 * h], dp[nt][2 * h + 1]);
            }
        __syncthreads();
        gemm<2, TI, D / 16, false>(
            dk, 0, kB / 16, [&](int m, int kk) { return quad<true, false>(sDS + m0 * kTS, kTS, m, kk); },
            [&](int n, int kk) { return quad<false, false>(q + d0, RS, n, kk); });
        gemm<2, TI, D / 16, false>(
            dv, 0, kB / 16, [&](int m, int kk) { return quad<true, false>(sP + m0 * kTS, kTS, m, kk); },
            [&](int n, int kk) { return quad<false, false>(o + d0, RS, n, kk); });
        cp_wait_all();
        __syncthreads();
    }
    store_rows<Tin, D>(p.dk, row0, kt * kB, p.T, dk, m0, d0, gr, t2);
    store_rows<Tin, D>(p.dv, row0, kt * kB, p.T, dv, m0, d0, gr, t2);
}

template <typename Tin, int D>
cudaError_t run(const Args &p, long heads, cudaStream_t stream) {
    constexpr int bytes = BwdSmem<Tin, D>::BYTES;
    static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
    cudaError_t e;
    if ((e = delta::raise_smem<bwd_query<Tin, D>>(bytes)) != cudaSuccess) return e;
    if ((e = delta::raise_smem<bwd_key<Tin, D>>(bytes)) != cudaSuccess) return e;
    bwd_query<Tin, D><<<(unsigned)(heads * p.nt), kThreads, bytes, stream>>>(p);
    if ((e = after_launch()) != cudaSuccess) return e;
    bwd_key<Tin, D><<<(unsigned)(heads * p.nt), kThreads, bytes, stream>>>(p);
    return after_launch();
}

template <typename Tin>
cudaError_t run_d(const Args &p, long heads, int d, cudaStream_t stream) {
    switch (d) {
        case 16: return run<Tin, 16>(p, heads, stream);
        case 32: return run<Tin, 32>(p, heads, stream);
        case 64: return run<Tin, 64>(p, heads, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

size_t prefill_backward_workspace_bytes(int dtype, long heads, int T, int d) {
    return prefill_backward_tc_applies(dtype, T, d) ? prefill_backward_tc_workspace_bytes(heads, T)
                                                    : (size_t)heads * T * sizeof(float4);
}

cudaError_t prefill_backward(const PrefillBackwardArgs &a, cudaStream_t stream) {
    if (prefill_backward_tc_applies(a.dtype, a.T, a.d)) return prefill_backward_tc(a, stream);
    const Args p{a.q, a.k, a.v, a.d_o, a.dq, a.dk, a.dv, static_cast<float4 *>(a.ws), a.T,
                 (a.T + kB - 1) / kB, a.eps};
    return a.dtype == 0 ? run_d<float>(p, a.heads, a.d, stream)
                        : run_d<__nv_bfloat16>(p, a.heads, a.d, stream);
}

}  // namespace kata
