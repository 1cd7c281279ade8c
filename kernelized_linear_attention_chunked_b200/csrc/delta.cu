// The gated delta rule for serving: the chunked prefill (kernels and
// mathematics in delta.cuh) and the one-token step.
#include "delta.cuh"

namespace kata {
namespace {

using namespace delta;

// floats of scratch per chunk
constexpr size_t chunk_floats(int d) {
    return 2 * (size_t)kC * d + (size_t)kC * kC + kCoef;
}

Scratch carve(void *ws, size_t chunks, int d) {
    float *f = static_cast<float *>(ws);
    Scratch s;
    s.W = f;
    s.Y = s.W + chunks * kC * d;
    s.M = s.Y + chunks * kC * d;
    s.coef = s.M + chunks * kC * kC;
    return s;
}

template <typename Tin, int D>
cudaError_t prefill_d(const Args &p, const Scratch &w, long heads, cudaStream_t stream) {
    cudaError_t e = launch_prep<Tin, D, false>(p, w, Scratch{}, heads, stream);
    if (e != cudaSuccess) return e;
    return launch_chain<Tin, D>(p, w, heads, stream);
}

template <typename Tin>
cudaError_t prefill_t(const Args &p, const Scratch &w, long heads, int d, cudaStream_t stream) {
    switch (d) {
        case 16: return prefill_d<Tin, 16>(p, w, heads, stream);
        case 32: return prefill_d<Tin, 32>(p, w, heads, stream);
        case 64: return prefill_d<Tin, 64>(p, w, heads, stream);
        case 128: return prefill_d<Tin, 128>(p, w, heads, stream);
        default: return cudaErrorInvalidValue;
    }
}

// One token: S = a S + beta k (v - a S^T k)^T, o = scale S^T q, a = exp(g).
// Bound by reading and writing the state once. The state's columns are
// independent, and both sums over its rows can be taken on the state as read,
//     r = S^T k, p = S^T q:  e = v - a r,  o = scale (a p + (q.k) beta e),
// so one pass reads it into registers, one exchange joins the row sums, and the
// same registers are updated and written back. Measured (steps in a CUDA graph; states
// in turn, 0.7 to 0.8 GB of them, so that each comes from HBM): B64 H16 d128 bf16 21.7 us,
// 6.2 TB/s of state traffic, 95 % of the copy bandwidth; B37 H12 d128 fp32 10.8 us, 83 %;
// B64 H16 d64 bf16 7.9 us, 66 %. One state again and again stays in L2 where it fits:
// 14.7, 7.2 and 5.3 us. A call through Python takes 10 us of host time. A CTA takes CW
// columns of one head, a thread float4s of one column group, RPP rows apart.
template <typename Tin, int D>
struct StepCfg {
    static constexpr int CW = D < 64 ? D : 64;
    static constexpr int CG = CW / 4;
    static constexpr int THREADS = D * CG < 256 ? D * CG : 256;
    static constexpr int RPP = THREADS / CG;
    static constexpr int ROWS = D / RPP;  // rows per thread
    static constexpr int NW = THREADS / 32;
};

__device__ __forceinline__ float4 fma4(float a, float4 x, float4 y) {
    return make_float4(fmaf(a, x.x, y.x), fmaf(a, x.y, y.y), fmaf(a, x.z, y.z), fmaf(a, x.w, y.w));
}
__device__ __forceinline__ float4 add4(float4 x, float4 y) {
    return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
}
__device__ __forceinline__ float4 shfl4(float4 x, int off) {
    return make_float4(__shfl_xor_sync(0xffffffffu, x.x, off), __shfl_xor_sync(0xffffffffu, x.y, off),
                       __shfl_xor_sync(0xffffffffu, x.z, off), __shfl_xor_sync(0xffffffffu, x.w, off));
}

template <typename Tin, int D>
__global__ void __launch_bounds__(StepCfg<Tin, D>::THREADS)
    delta_step(const Tin *q, const Tin *k, const Tin *v, const float *g, const float *beta, float scale,
               float *S, Tin *o) {
    using L = StepCfg<Tin, D>;
    constexpr int PARTS = D / L::CW;
    __shared__ float4 redr[L::NW][L::CG], redp[L::NW][L::CG];
    __shared__ float redqk[L::NW];
    const int tid = threadIdx.x, cg = tid % L::CG, r0 = tid / L::CG;
    const int warp = tid >> 5, lane = tid & 31;
    const size_t head = blockIdx.x / PARTS;
    const int c0 = (int)(blockIdx.x % PARTS) * L::CW + 4 * cg;
    float *Sh = S + head * (size_t)(D * D) + c0;
    // Whatever the stream ran before may still be writing any of these tensors (q may be the
    // o of the step before): no __restrict__, which would allow loads ahead of the wait or
    // through the read-only cache.
    if (tid == 0) sm100::launch_dependents();
    sm100::grid_dependency_wait();
    float4 s[L::ROWS];
#pragma unroll
    for (int i = 0; i < L::ROWS; ++i)
        s[i] = __ldcs(reinterpret_cast<const float4 *>(Sh + (r0 + i * L::RPP) * D));
    float kr[L::ROWS];
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f), p = r;
    float qk = 0.f;
#pragma unroll
    for (int i = 0; i < L::ROWS; ++i) {
        const int row = r0 + i * L::RPP;
        kr[i] = to_f32(k[head * D + row]);
        const float qr = to_f32(q[head * D + row]);
        r = fma4(kr[i], s[i], r);
        p = fma4(qr, s[i], p);
        qk = fmaf(qr, kr[i], qk);
    }
    const float lg = g[head], a = expf(lg < kMinLog ? kMinLog : lg), b = beta[head];
    const float4 vv = make_float4(to_f32(v[head * D + c0]), to_f32(v[head * D + c0 + 1]),
                                  to_f32(v[head * D + c0 + 2]), to_f32(v[head * D + c0 + 3]));
    // lanes CG apart hold other rows of the same columns
#pragma unroll
    for (int off = L::CG; off < 32; off <<= 1) {
        r = add4(r, shfl4(r, off));
        p = add4(p, shfl4(p, off));
        qk += __shfl_xor_sync(0xffffffffu, qk, off);
    }
    if (lane < L::CG) {
        redr[warp][lane] = r;
        redp[warp][lane] = p;
    }
    if (lane == 0) redqk[warp] = qk;
    __syncthreads();
    r = redr[0][cg];
    p = redp[0][cg];
    qk = redqk[0];
#pragma unroll
    for (int w = 1; w < L::NW; ++w) {
        r = add4(r, redr[w][cg]);
        p = add4(p, redp[w][cg]);
        qk += redqk[w];
    }
    const float4 e = fma4(-a, r, vv);
    const float4 u = make_float4(b * e.x, b * e.y, b * e.z, b * e.w);
#pragma unroll
    for (int i = 0; i < L::ROWS; ++i) {
        const float4 n = fma4(kr[i], u, make_float4(a * s[i].x, a * s[i].y, a * s[i].z, a * s[i].w));
        __stcs(reinterpret_cast<float4 *>(Sh + (r0 + i * L::RPP) * D), n);
    }
    if (r0 == 0) {
        const float4 x = fma4(qk, u, make_float4(a * p.x, a * p.y, a * p.z, a * p.w));
        Tin *d = o + head * D + c0;
        if constexpr (sizeof(Tin) == 2) {
            reinterpret_cast<__nv_bfloat162 *>(d)[0] = __floats2bfloat162_rn(scale * x.x, scale * x.y);
            reinterpret_cast<__nv_bfloat162 *>(d)[1] = __floats2bfloat162_rn(scale * x.z, scale * x.w);
        } else {
            *reinterpret_cast<float4 *>(d) =
                make_float4(scale * x.x, scale * x.y, scale * x.z, scale * x.w);
        }
    }
}

template <typename Tin, int D>
cudaError_t step_d(const void *q, const void *k, const void *v, const float *g, const float *beta,
                   long heads, float scale, float *S, void *o, cudaStream_t stream) {
    using L = StepCfg<Tin, D>;
    const cudaError_t e = tc::launch_overlapped(
        delta_step<Tin, D>, (unsigned)(heads * (D / L::CW)), L::THREADS, 0, stream,
        static_cast<const Tin *>(q), static_cast<const Tin *>(k), static_cast<const Tin *>(v), g, beta,
        scale, S, static_cast<Tin *>(o));
    return e != cudaSuccess ? e : after_launch();
}

template <typename Tin>
cudaError_t step_t(const void *q, const void *k, const void *v, const float *g, const float *beta,
                   long heads, int d, float scale, float *S, void *o, cudaStream_t stream) {
    switch (d) {
        case 16: return step_d<Tin, 16>(q, k, v, g, beta, heads, scale, S, o, stream);
        case 32: return step_d<Tin, 32>(q, k, v, g, beta, heads, scale, S, o, stream);
        case 64: return step_d<Tin, 64>(q, k, v, g, beta, heads, scale, S, o, stream);
        case 128: return step_d<Tin, 128>(q, k, v, g, beta, heads, scale, S, o, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

size_t delta_prefill_workspace_bytes(long heads, int T, int d) {
    return (size_t)heads * delta::chunks_of(T) * chunk_floats(d) * sizeof(float);
}

cudaError_t delta_prefill(const DeltaArgs &a, cudaStream_t stream) {
    const int nc = delta::chunks_of(a.T);
    Args p{};
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.g = a.g;
    p.beta = a.beta;
    p.S_in = a.S_in;
    p.S_out = a.S_out;
    p.o = a.o;
    p.T = a.T;
    p.nc = nc;
    p.scale = a.scale;
    const Scratch w = carve(a.ws, (size_t)a.heads * nc, a.d);
    return a.dtype == 0 ? prefill_t<float>(p, w, a.heads, a.d, stream)
                        : prefill_t<__nv_bfloat16>(p, w, a.heads, a.d, stream);
}

cudaError_t delta_decode_step(const void *q, const void *k, const void *v, int dtype,
                              const float *g, const float *beta, long heads, int d, float scale,
                              float *S, void *o, cudaStream_t stream) {
    return dtype == 0 ? step_t<float>(q, k, v, g, beta, heads, d, scale, S, o, stream)
                      : step_t<__nv_bfloat16>(q, k, v, g, beta, heads, d, scale, S, o, stream);
}

}  // namespace kata
