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
// accuracy; bf16 inputs are prefill_backward_tc.cu's. Two launches: bwd_query (den and
// delta over the keys of ROWS queries, then their dQ) and bwd_key (dK, dV of ROWS
// keys). bwd_query leaves den and delta of every row for bwd_key. ROWS is 64, or 32
// where 64 would leave SMs idle. A tile of rows is one CTA's or, where tiles are few
// and walks are long, a cluster's: its CTAs take every n-th step, and their sums are
// joined through each other's shared memory in the CTAs' order.
//
// Rows with few keys need care: there delta_i is nearly dP_ij (row 0 has
// dP - delta = dP eps / den), and a score near zero enters as 1 / s^3. So delta
// is kept as two floats (hi + lo: dP - hi is exact when the two are close, and
// only then does lo matter) and summed in 64 bits, and the first sixteen
// queries' scores and dP are formed in 64 bits, the same in both kernels. From
// row 16 on a row's den is a sum over more than 16 keys.
//
// Measured on B200 at B1 H4 T643 d64: 54 us (four CTAs per tile; 103 with one each: 84
// CTAs, the longest walking 22 steps); at B1 H16 T2048 d64 1.00 ms, 21.5 TFLOP/s of the
// five products per causal pair, of which nine are run in three tf32 parts (116 TFLOP/s of
// 288 in tf32). Bound by issue (49 %), the tensor pipe (47 %) and the steps' dependent
// parts (8 warps per SM).
#include <float.h>

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
    static constexpr int RED = STAT + 2 * kB * 16;   // bwd_query: row sums of four column quarters, and theirs
    static constexpr int BYTES = RED + 10 * ROWS * 8;
};

// The first sixteen queries' scores and dP in 64 bits, in the layout of two accumulator
// tiles: rows (0, 8 on) of q, o against columns (0, 1, 8, 9 on) of k, v. Each of four
// warps (`quarter`) sums a quarter of the d terms into its 512 doubles of `buf`; after a
// barrier one of them joins those. (By one warp alone, in every pass, this was two thirds
// of a call of 64 tokens at d = 64.)
template <int D>
__device__ __forceinline__ void dots64(double *buf, int quarter, int lane, const float *q,
                                       const float *o, const float *k, const float *v) {
    constexpr int RS = D + 8;
    double s[2][4], dp[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = dp[n][e] = 0.0;
#pragma unroll 2
    for (int c = quarter * (D / 4); c < (quarter + 1) * (D / 4); ++c) {
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
    double *d = buf + 512 * quarter + lane;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            d[32 * (4 * n + e)] = s[n][e];
            d[32 * (8 + 4 * n + e)] = dp[n][e];
        }
}
// value x (0 .. 7 the scores, then dP) of this lane, joined
__device__ __forceinline__ double joined64(const double *buf, int lane, int x) {
    const double *d = buf + 32 * x + lane;
    return (d[0] + d[512]) + (d[1024] + d[1536]);
}

// The CTAs of a cluster share a tile of rows: each takes every n-th step of its walk.
struct Split {
    int rank, n;
    __device__ __forceinline__ Split() {
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    }
    __device__ __forceinline__ int steps(int all) const { return all > rank ? (all - rank + n - 1) / n : 0; }
    __device__ __forceinline__ void sync() const {
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                         : "memory");
    }
    // CTA `r`'s address of shared memory at `p`
    __device__ __forceinline__ uint32_t at(const void *p, int r) const {
        uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
        asm("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(r));
        return a;
    }
};
__device__ __forceinline__ double peer_f64(uint32_t a) {
    double x;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(x) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ float4 peer_f32x4(uint32_t a) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "r"(a)
                 : "memory");
    return x;
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

// The same of `part`, the sum over the cluster's CTAs (in their order: the same bits on
// every run), through `tile` (ROWS x D in shared memory that nobody else uses). Each CTA
// joins and writes its share of the rows. Ends with the reads done everywhere.
template <int D, int ROWS, int N, int M>
__device__ __forceinline__ void join_rows(void *const (&dst)[M], size_t row0, int t0, int T,
                                          const float (*const (&part)[M])[4], float *tile,
                                          const Split &cl, int m0, int d0, int gr, int t2) {
    constexpr int RS = D + 8;
#pragma unroll
    for (int x = 0; x < M; ++x)
        if (d0 < D) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nt = 0; nt < N; ++nt)
                    *reinterpret_cast<float2 *>(tile + (x * ROWS + m0 + gr + 8 * h) * RS + d0 + 8 * nt +
                                                t2) =
                        make_float2(part[x][nt][2 * h], part[x][nt][2 * h + 1]);
        }
    cl.sync();
    for (int i = cl.rank * blockDim.x + threadIdx.x; i < M * ROWS * (D / 4); i += cl.n * blockDim.x) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4)), t = t0 + r % ROWS;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < cl.n; ++p) {
            const float4 v = peer_f32x4(cl.at(tile + r * RS + c, p));
            sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
        }
        if (t < T)
            *reinterpret_cast<float4 *>(static_cast<float *>(dst[M == 1 ? 0 : r / ROWS]) +
                                        (row0 + t) * (size_t)D + c) = sum;
    }
    cl.sync();
}

// One cluster per (head, ROWS queries). Two walks over the key tiles up to the
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
    const Split cl;
    const unsigned id = blockIdx.x / cl.n;
    const size_t head = id / p.tiles;
    const int q0 = (p.tiles - 1 - (int)(id % p.tiles)) * ROWS;  // the longest rows first
    const size_t row0 = head * (size_t)p.T;
    // this CTA's key tiles with a key that a query sees
    const int walk = cl.steps((min(q0 + ROWS, p.T) + kB - 1) / kB);
    // step 0 holds the first sixteen queries' tile; it is one warp's
    const bool few = q0 == 0 && cl.rank == 0, mine = few && m0 == 0 && n0 == 0;
    double *buf = reinterpret_cast<double *>(sm + L::DS);

    auto tileK = [&](int u) { return reinterpret_cast<float *>(sm + L::B0 + (u & 1) * 2 * L::IN); };
    auto tileV = [&](int u) { return tileK(u) + kB * RS; };
    auto prefetch = [&](int u) {
        const int t = ((u < walk ? u : u - walk) * cl.n + cl.rank) * kB;
        load_tile<float, D, TH>(tileK(u), RS, static_cast<const float *>(p.k), row0, t, p.T, D, 0, tid);
        load_tile<float, D, TH>(tileV(u), RS, static_cast<const float *>(p.v), row0, t, p.T, D, 0, tid);
        cp_commit();
    };
    // After the wait for whatever the stream ran before: bwd_key reads inputs at once, and
    // only for the statistics waits for this grid's end.
    sm100::grid_dependency_wait();
    if (tid == 0) sm100::launch_dependents();
    load_tile<float, D, TH, ROWS>(sQ, RS, static_cast<const float *>(p.q), row0, q0, p.T, D, 0, tid);
    load_tile<float, D, TH, ROWS>(sO, RS, static_cast<const float *>(p.d_o), row0, q0, p.T, D, 0, tid);
    if (walk > 0) prefetch(0);
    cp_wait_all();
    __syncthreads();

    double den[2] = {0.0, 0.0}, num[2] = {0.0, 0.0};  // rows gr, gr + 8
    float inv2[2], dhi[2], dlo[2];
    float dq[ND][4];
    clear(dq);
    auto scores = [&](const float *k, const float *v, float(&s)[2][4], float(&dp)[2][4]) {
        clear(s);
        clear(dp);
        gemm<2, 2, 2, 4>(
            s, 0, D / 16, [&](int m, int kk) { return quad<true>(sQ + m0 * RS, RS, m, kk); },
            [&](int n, int kk) { return quad<true>(k + n0 * RS, RS, n, kk); });
        gemm<2, 2, 2, 4>(
            dp, 0, D / 16, [&](int m, int kk) { return quad<true>(sO + m0 * RS, RS, m, kk); },
            [&](int n, int kk) { return quad<true>(v + n0 * RS, RS, n, kk); });
    };
    // whether row gr + 8 h sees column 8 nt + t2 + (e & 1) of step u
    auto seen = [&](int u, int nt, int e) {
        return (u * cl.n + cl.rank) * kB + n0 + 8 * nt + t2 + (e & 1) <= q0 + m0 + gr + 8 * (e >> 1);
    };
    for (int u = 0; u < walk; ++u) {  // den and delta den
        prefetch(u + 1);
        const float *k = tileK(u), *v = tileV(u);
        if (few && u == 0) {
            if (m0 == 0)
                dots64<D>(buf, quarter, lane, sQ + gr * RS, sO + gr * RS, k + t2 * RS, v + t2 * RS);
            __syncthreads();
        }
        if (mine && u == 0) {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (seen(0, nt, e)) {
                        const double x = joined64(buf, lane, 4 * nt + e);
                        den[e >> 1] = fma(x, x, den[e >> 1]);
                        num[e >> 1] = fma(x * x, joined64(buf, lane, 8 + 4 * nt + e), num[e >> 1]);
                    }
        } else {
            float s[2][4], dp[2][4], ds[2] = {0.f, 0.f}, ns[2] = {0.f, 0.f};
            scores(k, v, s, dp);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool on = seen(u, nt, e);
                    const float w = on ? s[nt][e] * s[nt][e] : 0.f;
                    ds[e >> 1] += w;
                    ns[e >> 1] = fmaf(w, on ? dp[nt][e] : 0.f, ns[e >> 1]);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                den[h] += (double)ds[h];
                num[h] += (double)ns[h];
            }
        }
        cp_wait_all();
        __syncthreads();
    }
    // the rows' sums are complete: join the lanes, the column quarters, the CTAs
    {
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
        double *sum = red + 8 * ROWS;
        if (tid < 2 * ROWS) {
            double x = 0.0;
            for (int c = 0; c < 4; ++c) x += red[2 * c * ROWS + tid];
            sum[tid] = x;
        }
        cl.sync();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = m0 + gr + 8 * h;
            double d = (double)p.eps, n = 0.0;
            for (int r = 0; r < cl.n; ++r) {
                d += peer_f64(cl.at(sum + i, r));
                n += peer_f64(cl.at(sum + ROWS + i, r));
            }
            const bool none = d < (double)FLT_MIN;  // below it 2 / d may be infinite in fp32
            const double delta = none ? 0.0 : n / d;
            inv2[h] = none ? 0.f : (float)(2.0 / d);
            dhi[h] = (float)delta;
            dlo[h] = (float)(delta - (double)dhi[h]);
            if (cl.rank == 0 && quarter == 0 && (lane & 3) == 0 && q0 + i < p.T)
                p.stat[row0 + q0 + i] = make_float4(0.5f * inv2[h], inv2[h], dhi[h], dlo[h]);
        }
    }
    if (mine) {  // sDS takes the partial sums' place: keep the joined ones behind it
        double x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = joined64(buf, lane, i);
        __syncwarp();
        buf = reinterpret_cast<double *>(sm + L::P);
#pragma unroll
        for (int i = 0; i < 16; ++i) buf[32 * i + lane] = x[i];
    }
    if (few) __syncthreads();
    for (int u = 0; u < walk; ++u) {  // dQ
        if (u + 1 < walk) prefetch(walk + u + 1);
        const float *k = tileK(walk + u), *v = tileV(walk + u);
        float s[2][4];
        if (mine && u == 0) {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int h = e >> 1;
                    const double x = buf[32 * (4 * nt + e) + lane], y = buf[32 * (8 + 4 * nt + e) + lane];
                    s[nt][e] = seen(0, nt, e) ? (float)((double)inv2[h] * x *
                                                        ((y - (double)dhi[h]) - (double)dlo[h]))
                                              : 0.f;
                }
        } else {
            float dp[2][4];
            scores(k, v, s, dp);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int h = e >> 1;
                    s[nt][e] =
                        seen(u, nt, e) ? inv2[h] * s[nt][e] * ((dp[nt][e] - dhi[h]) - dlo[h]) : 0.f;
                }
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2 *>(sDS + (m0 + gr + 8 * h) * kTS + n0 + 8 * nt + t2) =
                    make_float2(s[nt][2 * h], s[nt][2 * h + 1]);
        __syncthreads();
        if (d0 < D)
            gemm<2, 2, ND, 4>(
                dq, 0, kB / 16, [&](int m, int kk) { return quad<true>(sDS + m0 * kTS, kTS, m, kk); },
                [&](int n, int kk) { return quad<false>(k + d0, RS, n, kk); });
        cp_wait_all();
        __syncthreads();
    }
    if (cl.n > 1)
        join_rows<D, ROWS, ND, 1>({p.dq}, row0, q0, p.T, {dq}, reinterpret_cast<float *>(sm + L::B0), cl,
                                  m0, d0, gr, t2);
    else if (d0 < D)
        store_rows<D>(p.dq, row0, q0, p.T, dq, m0, d0, gr, t2);
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
    const Split cl;
    const unsigned id = blockIdx.x / cl.n;
    const size_t head = id / p.tiles;
    const int k0 = (int)(id % p.tiles) * ROWS;  // the keys that most queries see first
    const size_t row0 = head * (size_t)p.T;

    const int first = k0 / kB + cl.rank, walk = cl.steps(p.steps - k0 / kB);  // this CTA's steps

    auto tileQ = [&](int j) { return reinterpret_cast<float *>(sm + L::B0 + (j & 1) * 2 * L::IN); };
    auto tileO = [&](int j) { return tileQ(j) + kB * RS; };
    auto stats = [&](int j) { return reinterpret_cast<float4 *>(sm + L::STAT) + (j & 1) * kB; };
    auto prefetch = [&](int j) {
        const int t = (first + j * cl.n) * kB;
        load_tile<float, D, TH>(tileQ(j), RS, static_cast<const float *>(p.q), row0, t, p.T, D, 0, tid);
        load_tile<float, D, TH>(tileO(j), RS, static_cast<const float *>(p.d_o), row0, t, p.T, D, 0, tid);
        if (tid < kB) {
            const bool have = t + tid < p.T;
            delta::cp16(stats(j) + tid, p.stat + row0 + (have ? t + tid : 0), have);
        }
        cp_commit();
    };
    load_tile<float, D, TH, ROWS>(sK, RS, static_cast<const float *>(p.k), row0, k0, p.T, D, 0, tid);
    load_tile<float, D, TH, ROWS>(sV, RS, static_cast<const float *>(p.v), row0, k0, p.T, D, 0, tid);
    sm100::grid_dependency_wait();  // bwd_query's statistics
    if (walk > 0) prefetch(0);
    cp_wait_all();
    __syncthreads();

    float dk[ND][4], dv[ND][4];
    clear(dk);
    clear(dv);
    for (int j = 0; j < walk; ++j) {
        if (j + 1 < walk) prefetch(j + 1);
        const int u = first + j * cl.n;
        const float *q = tileQ(j), *o = tileO(j);
        const float4 *st = stats(j);
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
        if (u == 0 && k0 == 0) {  // the first sixteen queries (and keys) in 64 bits
            double *buf = reinterpret_cast<double *>(sm + L::DS);
            if (m0 == 0) dots64<D>(buf, quarter, lane, sK + gr * RS, sV + gr * RS, q + t2 * RS, o + t2 * RS);
            __syncthreads();
            if (m0 == 0 && n0 == 0) {
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = gr + (e & 2 ? 8 : 0), i = 8 * nt + t2 + (e & 1);
                        const float4 t = st[i];
                        const double x = joined64(buf, lane, 4 * nt + e);
                        const double y = joined64(buf, lane, 8 + 4 * nt + e);
                        if (j > i) continue;
                        s[nt][e] = (float)((double)t.y * x * ((y - (double)t.z) - (double)t.w));
                        dp[nt][e] = (float)(x * x * (double)t.x);
                    }
            }
            __syncthreads();  // sDS and sP take the partial sums' place
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
    if (cl.n > 1) {
        join_rows<D, ROWS, ND, 2>({p.dk, p.dv}, row0, k0, p.T, {dk, dv},
                                  reinterpret_cast<float *>(sm + L::B0), cl, m0, d0, gr, t2);
    } else if (d0 < D) {
        store_rows<D>(p.dk, row0, k0, p.T, dk, m0, d0, gr, t2);
        store_rows<D>(p.dv, row0, k0, p.T, dv, m0, d0, gr, t2);
    }
}

template <int D, int ROWS>
cudaError_t run(Args p, long heads, int split, cudaStream_t stream) {
    using L = BwdCfg<D, ROWS>;
    static_assert(L::BYTES <= 227 * 1024, "shared memory of one CTA");
    p.tiles = (p.T + ROWS - 1) / ROWS;
    cudaError_t e;
    if ((e = tc::set_smem_once<bwd_query<D, ROWS>>(L::BYTES)) != cudaSuccess) return e;
    if ((e = tc::set_smem_once<bwd_key<D, ROWS>>(L::BYTES)) != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernels wait themselves
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(heads * p.tiles * split), 1, 1);
    cfg.blockDim = dim3(L::THREADS, 1, 1);
    cfg.dynamicSmemBytes = L::BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if ((e = cudaLaunchKernelEx(&cfg, bwd_query<D, ROWS>, p)) != cudaSuccess) return e;
    if ((e = after_launch()) != cudaSuccess) return e;
    e = cudaLaunchKernelEx(&cfg, bwd_key<D, ROWS>, p);
    return e != cudaSuccess ? e : after_launch();
}

// CTAs per tile of rows, for `tiles` of them whose longest walk has `steps`: doubled as
// long as all fit the SMs at once, or the longest walk keeps two steps (up to 512 CTAs)
// or four (up to 1024). Measured, for 1, 2, 4, 8 (us; fp32 d64, heads x T): 4 x 643: 95, 75,
// 55, 73; 1 x 2048: 257, 137, 104, 91; 4 x 2048: 405, 307, 267, 319; 16 x 1024: 315, 282,
// 307, 430; 48 x 300: 115, 127, 163, 299; 16 x 2048: 1080, 998, 1146, 1594; 64 x 1024:
// 1009, 1072, 1420, 2243.
int split_of(long tiles, int steps) {
    int n = 1;
    while (n < 8 && 2 * n <= steps) {
        const long ctas = 2 * n * tiles;
        if (!(ctas <= 148 || (ctas <= 512 && steps >= 4 * n) || (ctas <= 1024 && steps >= 8 * n))) break;
        n *= 2;
    }
    return n;
}

// 32 rows per CTA where 64 would not give every SM two
template <int D>
cudaError_t run_rows(const Args &p, long heads, cudaStream_t stream) {
    const long t64 = heads * ((p.T + 63) / 64), t32 = heads * ((p.T + 31) / 32);
    return t64 < 2 * 148 ? run<D, 32>(p, heads, split_of(t32, p.steps), stream)
                         : run<D, 64>(p, heads, split_of(t64, p.steps), stream);
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
