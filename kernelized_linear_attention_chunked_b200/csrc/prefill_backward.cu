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
// This file: fp32 inputs, in split-tf32 products (mma_tf32.cuh), which keep fp32
// accuracy; bf16 inputs are prefill_backward_tc.cu's. Two launches: bwd_query (one CTA
// per ROWS queries: den and delta over the keys, then dQ) and bwd_key (one CTA
// per ROWS keys: dK, dV). bwd_query leaves den and delta of every row for
// bwd_key. ROWS is 64, or 32 where 64 would leave SMs idle.
//
// Rows with few keys need care: there delta_i is nearly dP_ij (row 0 has
// dP - delta = dP eps / den), and a score near zero enters as 1 / s^3. So delta
// is kept as two floats (hi + lo: dP - hi is exact when the two are close, and
// only then does lo matter) and summed in 64 bits, and the first sixteen
// queries' scores and dP are formed in 64 bits, the same in both kernels. From
// row 16 on a row's den is a sum over more than 16 keys.
//
// Measured on B200 at B1 H4 T643 d64: 67 + 50 us (84 CTAs; the longest walks 22
// steps); at B2 H8 T2048 d64 1.15 ms, 18.7 TFLOP/s of the five products per causal pair, of
// which nine are run in three tf32 parts (101 TFLOP/s of 288 in tf32). Bound by issue (50 %)
// and shared memory (61 to 67 %).
#include "delta.cuh"

namespace kata {
namespace {

using namespace tf;
using delta::cp_commit;
using delta::cp_wait_all;
using delta::load_tile;

constexpr int kB = 64;    // streamed rows per step
constexpr int kTS = 72;   // row stride of a ROWS x 64 product

struct Args {
    const void *q, *k, *v, *d_o;
    void *dq, *dk, *dv;
    float4 *stat;  // [heads * T]: 1 / den, 2 / den, delta hi, delta lo
    int T, tiles, steps;  // tokens; ROWS-row tiles and 64-row steps per head
    float eps;
};

// Four warps per 16 rows, each 16 columns of a ROWS x 64 product and ND 8-column
// tiles of a ROWS x D one.
template <int D, int ROWS>
struct BwdCfg {
    static constexpr int THREADS = ROWS / 16 * 128;
    static constexpr int ND = D >= 32 ? D / 32 : 1;
    static constexpr int RS = D + 8;
    static constexpr int OWN = ROWS * RS * 4, IN = kB * RS * 4;
    static constexpr int A0 = 0, A1 = OWN;     // the CTA's own rows: q, dO or k, v
    static constexpr int B0 = 2 * OWN;         // two stages of the other side's two tiles
    static constexpr int DS = B0 + 4 * IN;     // ROWS x 64 products
    static constexpr int P = DS + ROWS * kTS * 4;
    static constexpr int STAT = P + ROWS * kTS * 4;  // bwd_key: two stages of 64 float4
    static constexpr int RED = STAT + 2 * kB * 16;   // bwd_query: row sums of four column quarters
    static constexpr int BYTES = RED + 8 * ROWS * 8;
};

// s and dP in 64 bits for two rows (0, 8 on) of q, o against four columns (0, 1,
// 8, 9 on) of k, v, in the layout of two accumulator tiles.
template <int D>
__device__ __forceinline__ void dots64(const float *q, const float *o, const float *k, const float *v,
                                       double (&s)[2][4], double (&dp)[2][4]) {
    constexpr int RS = D + 8;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = dp[n][e] = 0.0;
#pragma unroll 2
    for (int c = 0; c < D; ++c) {
        double a[2], b[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            a[h] = q[8 * h * RS + c];
            b[h] = o[8 * h * RS + c];
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const double x = k[(8 * n + e) * RS + c], y = v[(8 * n + e) * RS + c];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s[n][2 * h + e] = fma(a[h], x, s[n][2 * h + e]);
                    dp[n][2 * h + e] = fma(b[h], y, dp[n][2 * h + e]);
                }
            }
    }
}

// Columns d0 .. of rows m0 .. of a tile that starts at row t0 of a [T, D] matrix
template <int D, int N>
__device__ __forceinline__ void store_rows(void *dst, size_t row0, int t0, int T,
                                           const float (&acc)[N][4], int m0, int d0, int gr, int t2) {
    float *o = static_cast<float *>(dst);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int t = t0 + m0 + gr + 8 * h;
        if (t >= T) continue;
#pragma unroll
        for (int nt = 0; nt < N; ++nt)
            *reinterpret_cast<float2 *>(o + (row0 + t) * (size_t)D + d0 + 8 * nt + t2) =
                make_float2(acc[nt][2 * h], acc[nt][2 * h + 1]);
    }
}

// One CTA per (head, ROWS queries). Two walks over the key tiles up to the
// diagonal: den and delta, then dQ.
template <int D, int ROWS>
__global__ void __launch_bounds__(BwdCfg<D, ROWS>::THREADS) bwd_query(Args p) {
    using L = BwdCfg<D, ROWS>;
    constexpr int RS = L::RS, ND = L::ND, TH = L::THREADS;
    extern __shared__ __align__(16) uint8_t sm[];
    float *sQ = reinterpret_cast<float *>(sm + L::A0), *sO = reinterpret_cast<float *>(sm + L::A1);
    float *sDS = reinterpret_cast<float *>(sm + L::DS);
    double *red = reinterpret_cast<double *>(sm + L::RED);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, t2 = 2 * (lane & 3);
    const int quarter = warp & 3, m0 = 16 * (warp >> 2), n0 = 16 * quarter, d0 = 8 * ND * quarter;
    const size_t head = blockIdx.x / p.tiles;
    const int q0 = (p.tiles - 1 - (int)(blockIdx.x % p.tiles)) * ROWS;  // the longest rows first
    const size_t row0 = head * (size_t)p.T;
    const int walk = (min(q0 + ROWS, p.T) + kB - 1) / kB;  // key tiles with a key that a query sees
    const bool few = q0 == 0 && m0 == 0;  // this warp's rows are the first sixteen queries

    auto tileK = [&](int u) { return reinterpret_cast<float *>(sm + L::B0 + (u & 1) * 2 * L::IN); };
    auto tileV = [&](int u) { return tileK(u) + kB * RS; };
    auto prefetch = [&](int u) {
        const int t = (u < walk ? u : u - walk) * kB;
        load_tile<float, D, TH>(tileK(u), RS, static_cast<const float *>(p.k), row0, t, p.T, D, 0, tid);
        load_tile<float, D, TH>(tileV(u), RS, static_cast<const float *>(p.v), row0, t, p.T, D, 0, tid);
        cp_commit();
    };
    if (tid == 0) sm100::launch_dependents();  // bwd_key: it waits for this grid's end
    load_tile<float, D, TH, ROWS>(sQ, RS, static_cast<const float *>(p.q), row0, q0, p.T, D, 0, tid);
    load_tile<float, D, TH, ROWS>(sO, RS, static_cast<const float *>(p.d_o), row0, q0, p.T, D, 0, tid);
    prefetch(0);
    cp_wait_all();
    __syncthreads();

    double den[2] = {0.0, 0.0}, num[2] = {0.0, 0.0};  // rows gr, gr + 8
    float inv2[2], dhi[2], dlo[2];
    float dq[ND][4];
    clear(dq);
    for (int u = 0; u < 2 * walk; ++u) {
        if (u + 1 < 2 * walk) prefetch(u + 1);
        const bool second = u >= walk;
        const int k0 = (second ? u - walk : u) * kB;
        const float *k = tileK(u), *v = tileV(u);
        if (u == walk) {  // the rows' sums are complete: join the lanes, then the column quarters
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int off = 1; off < 4; off <<= 1) {
                    den[h] += __shfl_xor_sync(0xffffffffu, den[h], off);
                    num[h] += __shfl_xor_sync(0xffffffffu, num[h], off);
                }
                if ((lane & 3) == 0) {
                    red[2 * quarter * ROWS + m0 + gr + 8 * h] = den[h];
                    red[(2 * quarter + 1) * ROWS + m0 + gr + 8 * h] = num[h];
                }
            }
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = m0 + gr + 8 * h;
                den[h] = (double)p.eps;
                num[h] = 0.0;
                for (int c = 0; c < 4; ++c) {
                    den[h] += red[2 * c * ROWS + i];
                    num[h] += red[(2 * c + 1) * ROWS + i];
                }
                const double delta = den[h] == 0.0 ? 0.0 : num[h] / den[h];
                inv2[h] = den[h] == 0.0 ? 0.f : (float)(2.0 / den[h]);
                dhi[h] = (float)delta;
                dlo[h] = (float)(delta - (double)dhi[h]);
                if (quarter == 0 && (lane & 3) == 0 && q0 + i < p.T)
                    p.stat[row0 + q0 + i] = make_float4(0.5f * inv2[h], inv2[h], dhi[h], dlo[h]);
            }
        }
        float s[2][4], dp[2][4];
        if (few && k0 == 0 && n0 == 0) {
            double s64[2][4], dp64[2][4];
            dots64<D>(sQ + gr * RS, sO + gr * RS, k + t2 * RS, v + t2 * RS, s64, dp64);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int h = e >> 1;
                    const bool seen = 8 * nt + t2 + (e & 1) <= gr + 8 * h;
                    const double x = seen ? s64[nt][e] : 0.0;
                    if (!second) {
                        den[h] = fma(x, x, den[h]);
                        if (seen) num[h] = fma(x * x, dp64[nt][e], num[h]);
                    } else {
                        s[nt][e] = seen ? (float)((double)inv2[h] * x *
                                                  ((dp64[nt][e] - (double)dhi[h]) - (double)dlo[h]))
                                        : 0.f;
                    }
                }
        } else {
            clear(s);
            clear(dp);
            gemm<2, 2, 2, 4>(
                s, 0, D / 16, [&](int m, int kk) { return quad<true>(sQ + m0 * RS, RS, m, kk); },
                [&](int n, int kk) { return quad<true>(k + n0 * RS, RS, n, kk); });
            gemm<2, 2, 2, 4>(
                dp, 0, D / 16, [&](int m, int kk) { return quad<true>(sO + m0 * RS, RS, m, kk); },
                [&](int n, int kk) { return quad<true>(v + n0 * RS, RS, n, kk); });
            float ds[2] = {0.f, 0.f}, ns[2] = {0.f, 0.f};
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int h = e >> 1;
                    const bool seen = k0 + n0 + 8 * nt + t2 + (e & 1) <= q0 + m0 + gr + 8 * h;
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
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2 *>(sDS + (m0 + gr + 8 * h) * kTS + n0 + 8 * nt + t2) =
                        make_float2(s[nt][2 * h], s[nt][2 * h + 1]);
            __syncthreads();
            if (d0 < D)
                gemm<2, 2, ND, 4>(
                    dq, 0, kB / 16,
                    [&](int m, int kk) { return quad<true>(sDS + m0 * kTS, kTS, m, kk); },
                    [&](int n, int kk) { return quad<false>(k + d0, RS, n, kk); });
        }
        cp_wait_all();
        __syncthreads();
    }
    if (d0 < D) store_rows<D>(p.dq, row0, q0, p.T, dq, m0, d0, gr, t2);
}

// One CTA per (head, ROWS keys): the query steps from the diagonal on. Rows of
// its ROWS x 64 tiles are keys: s^T = K Q^T, dP^T = V dO^T.
template <int D, int ROWS>
__global__ void __launch_bounds__(BwdCfg<D, ROWS>::THREADS) bwd_key(Args p) {
    using L = BwdCfg<D, ROWS>;
    constexpr int RS = L::RS, ND = L::ND, TH = L::THREADS;
    extern __shared__ __align__(16) uint8_t sm[];
    float *sK = reinterpret_cast<float *>(sm + L::A0), *sV = reinterpret_cast<float *>(sm + L::A1);
    float *sDS = reinterpret_cast<float *>(sm + L::DS), *sP = reinterpret_cast<float *>(sm + L::P);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, t2 = 2 * (lane & 3);
    const int quarter = warp & 3, m0 = 16 * (warp >> 2), n0 = 16 * quarter, d0 = 8 * ND * quarter;
    const size_t head = blockIdx.x / p.tiles;
    const int k0 = (int)(blockIdx.x % p.tiles) * ROWS;  // the keys that most queries see first
    const size_t row0 = head * (size_t)p.T;

    auto tileQ = [&](int u) { return reinterpret_cast<float *>(sm + L::B0 + (u & 1) * 2 * L::IN); };
    auto tileO = [&](int u) { return tileQ(u) + kB * RS; };
    auto stats = [&](int u) { return reinterpret_cast<float4 *>(sm + L::STAT) + (u & 1) * kB; };
    auto prefetch = [&](int u) {
        load_tile<float, D, TH>(tileQ(u), RS, static_cast<const float *>(p.q), row0, u * kB, p.T, D, 0, tid);
        load_tile<float, D, TH>(tileO(u), RS, static_cast<const float *>(p.d_o), row0, u * kB, p.T, D, 0,
                              tid);
        if (tid < kB) {
            const bool have = u * kB + tid < p.T;
            delta::cp16(stats(u) + tid, p.stat + row0 + (have ? u * kB + tid : 0), have);
        }
        cp_commit();
    };
    load_tile<float, D, TH, ROWS>(sK, RS, static_cast<const float *>(p.k), row0, k0, p.T, D, 0, tid);
    load_tile<float, D, TH, ROWS>(sV, RS, static_cast<const float *>(p.v), row0, k0, p.T, D, 0, tid);
    const int first = k0 / kB;
    sm100::grid_dependency_wait();  // bwd_query's statistics
    prefetch(first);
    cp_wait_all();
    __syncthreads();

    float dk[ND][4], dv[ND][4];
    clear(dk);
    clear(dv);
    for (int u = first; u < p.steps; ++u) {
        if (u + 1 < p.steps) prefetch(u + 1);
        const float *q = tileQ(u), *o = tileO(u);
        const float4 *st = stats(u);
        float s[2][4], dp[2][4];
        clear(s);
        clear(dp);
        gemm<2, 2, 2, 4>(
            s, 0, D / 16, [&](int m, int kk) { return quad<true>(sK + m0 * RS, RS, m, kk); },
            [&](int n, int kk) { return quad<true>(q + n0 * RS, RS, n, kk); });
        gemm<2, 2, 2, 4>(
            dp, 0, D / 16, [&](int m, int kk) { return quad<true>(sV + m0 * RS, RS, m, kk); },
            [&](int n, int kk) { return quad<true>(o + n0 * RS, RS, n, kk); });
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = k0 + m0 + gr + (e & 2 ? 8 : 0), i = n0 + 8 * nt + t2 + (e & 1);
                const bool seen = j <= u * kB + i;
                const float4 t = st[i];
                const float x = s[nt][e];
                s[nt][e] = seen ? t.y * x * ((dp[nt][e] - t.z) - t.w) : 0.f;
                dp[nt][e] = seen ? x * x * t.x : 0.f;
            }
        if (u == 0 && n0 == 0 && k0 + m0 == 0) {  // the first sixteen queries (and keys) in 64 bits
            double s64[2][4], dp64[2][4];
            dots64<D>(sK + gr * RS, sV + gr * RS, q + t2 * RS, o + t2 * RS, s64, dp64);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = gr + (e & 2 ? 8 : 0), i = 8 * nt + t2 + (e & 1);
                    const float4 t = st[i];
                    const double x = s64[nt][e];
                    if (j > i) continue;
                    s[nt][e] = (float)((double)t.y * x * ((dp64[nt][e] - (double)t.z) - (double)t.w));
                    dp[nt][e] = (float)(x * x * (double)t.x);
                }
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = (m0 + gr + 8 * h) * kTS + n0 + 8 * nt + t2;
                *reinterpret_cast<float2 *>(sDS + at) = make_float2(s[nt][2 * h], s[nt][2 * h + 1]);
                *reinterpret_cast<float2 *>(sP + at) = make_float2(dp[nt][2 * h], dp[nt][2 * h + 1]);
            }
        __syncthreads();
        if (d0 < D) {
            gemm<2, 2, ND, 4>(
                dk, 0, kB / 16,
                [&](int m, int kk) { return quad<true>(sDS + m0 * kTS, kTS, m, kk); },
                [&](int n, int kk) { return quad<false>(q + d0, RS, n, kk); });
            gemm<2, 2, ND, 4>(
                dv, 0, kB / 16,
                [&](int m, int kk) { return quad<true>(sP + m0 * kTS, kTS, m, kk); },
                [&](int n, int kk) { return quad<false>(o + d0, RS, n, kk); });
        }
        cp_wait_all();
        __syncthreads();
    }
    if (d0 < D) {
        store_rows<D>(p.dk, row0, k0, p.T, dk, m0, d0, gr, t2);
        store_rows<D>(p.dv, row0, k0, p.T, dv, m0, d0, gr, t2);
    }
}

template <int D, int ROWS>
cudaError_t run(Args p, long heads, cudaStream_t stream) {
    using L = BwdCfg<D, ROWS>;
    static_assert(L::BYTES <= 227 * 1024, "shared memory of one CTA");
    p.tiles = (p.T + ROWS - 1) / ROWS;
    cudaError_t e;
    if ((e = tc::set_smem_once<bwd_query<D, ROWS>>(L::BYTES)) != cudaSuccess) return e;
    if ((e = tc::set_smem_once<bwd_key<D, ROWS>>(L::BYTES)) != cudaSuccess) return e;
    const unsigned grid = (unsigned)(heads * p.tiles);
    bwd_query<D, ROWS><<<grid, L::THREADS, L::BYTES, stream>>>(p);
    if ((e = after_launch()) != cudaSuccess) return e;
    e = tc::launch_overlapped(bwd_key<D, ROWS>, grid, L::THREADS, L::BYTES, stream, p);
    return e != cudaSuccess ? e : after_launch();
}

// 32 rows per CTA where 64 would not give every SM two
template <int D>
cudaError_t run_rows(const Args &p, long heads, cudaStream_t stream) {
    const bool small = heads * ((p.T + 63) / 64) < 2 * 148;
    return small ? run<D, 32>(p, heads, stream) : run<D, 64>(p, heads, stream);
}

}  // namespace

size_t prefill_backward_workspace_bytes(int dtype, long heads, int T) {
    return dtype == 1 ? prefill_backward_tc_workspace_bytes(heads, T)
                      : (size_t)heads * T * sizeof(float4);
}

cudaError_t prefill_backward(const PrefillBackwardArgs &a, cudaStream_t stream) {
    if (a.dtype == 1) return prefill_backward_tc(a, stream);
    const Args p{a.q, a.k, a.v, a.d_o, a.dq, a.dk, a.dv, static_cast<float4 *>(a.ws), a.T, 0,
                 (a.T + kB - 1) / kB, a.eps};
    switch (a.d) {
        case 16: return run_rows<16>(p, a.heads, stream);
        case 32: return run_rows<32>(p, a.heads, stream);
        case 64: return run_rows<64>(p, a.heads, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kata
