// Gradients of the causal kernelized prefill on the tcgen05 tensor cores, for
// bf16 inputs and any T. The formulas are in
// prefill_backward.cu; this file is about how the products are fed.
//
// One kernel in two modes, two launches:
//   queries  one CTA per (head, 128 queries). Walks the 64-key steps up to the
//            diagonal twice: first S = Q K^T and dP = dO V^T for the rows' den
//            and delta, then the same again for dS and dQ += dS K.
//   keys     one CTA per (head, 128 keys). Walks the 64-query steps from the
//            diagonal on: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO,
//            dK += dS^T Q, with each query's 1 / den and delta from the first.
// In both the CTA's own 128 rows are the A operands of the score products
// (tensor-memory lane = row) and the other side's 64 rows stream by TMA.
//
// Tensor memory (512 columns, one CTA per SM): three buffers of S (64 fp32
// columns) and dP (64), then the accumulators. The workers overwrite S with P
// and dP with dS as bf16 pairs, in place, sixteen columns with eight of upper parts and
// eight of lower ones, and the output products take them from there as A operands. A
// streamed tile serves both products it is needed in: [64 rows, d] in rows of 2 d bytes,
// swizzled by that width, is a K-major operand for the scores and an MN-major one for the
// outputs.
//
// Warp roles: two sets of workers on alternate steps, each two groups of four
// warps with half the step's columns (thread = row), two issuers of the score products (alternate steps: one
// thread needs longer for a step's waits and MMAs than the tensor pipe), one of the
// output products, a TMA producer. Every wait is bounded.
//
// Rounding: scores, dP, den and delta are fp32 or wider. P and dS go in as two bf16
// parts each (16 bits), so that the gradients are off by little more than their last
// rounding, 1.66e-3 of their norm. With one part dV was off by 2.3e-3, and dQ and dK, whose
// terms cancel, by up to 3.1e-3 (the second part of P costs 6 % of the time, that of dS
// 12 %). The rows of the first 128 queries sum den and delta in 64 bits, and delta is two
// floats: with few keys dP - delta is a small difference. It stays exact because
// S and dP come out of the same products with the same bits in both modes and
// both walks.
//
// Measured on B200 at B2 H8 T8192 d64 (344 GFLOP as five products per causal
// pair; twelve are run: six in either mode, P and dS counting twice): 987 to 1029 us a call
// (power), 334 to 348 TFLOP/s of the five; queries 534 us, keys 503 us by themselves under ncu. At T4096 ncu
// shows the tensor pipe at 36 % (queries) and 38 % (keys) of its cycles, issue at 56 and
// 63 %, shared memory at 42 and 53 %. What bounds it: the steps' hand-offs, the keys'
// workers, which read two statistics per column from shared memory and cut P and dS
// (without P's second part they took 451 us), and for the queries the single threads that
// issue the products (66 cycles per MMA against 48 for the operands' shared-memory reads).
#include <float.h>

#include "kata_internal.h"
#include "tc_tiles.cuh"

namespace kata {
namespace {

using namespace tc;

constexpr int kStep = 64;    // streamed rows per step
constexpr int kBufs = 3;     // S | dP buffers
constexpr int kStages = 6;   // streamed tiles in flight, a multiple of kBufs and kSets
constexpr int kSets = 2;     // sets of workers, on alternate steps
constexpr int kGroups = 2 * kSets;  // a set is two groups of four warps, half the columns each
constexpr int kWorkerWarps = 4 * kGroups;
static_assert(kStages == 2 * kBufs && kStages % kSets == 0, "slots of a step");
constexpr int kThreads = 32 * (kWorkerWarps + 4);
// Sixteen columns of S (dP) become the upper parts of P (dS) and, eight columns on, the lower.
constexpr uint32_t kLower = 8;

constexpr uint32_t kSwizzle32 = 6;  // rows of 32 bytes, 16-byte chunks swapped every four rows

struct BwdParams {
    int T, heads, tiles, steps;  // tokens; 128-row tiles and 64-row steps per head
    long pitch;           // rows per head of the statistics: 128 * tiles
    float eps;
    float *inv, *dhi, *dlo;  // [heads][pitch]: 1 / den, -delta as two floats
    __nv_bfloat16 *out0, *out1;  // queries: dQ; keys: dV, dK
    unsigned int *err;
};

enum BwdBar {
    kOwn = 0,                     // the CTA's own tiles landed
    // one per stage, step s using stage s % kStages in phase s / kStages:
    kTileFull = 1,                 // its tiles (and statistics) landed
    kSFull = kTileFull + kStages,  // S and dP are in tensor memory
    kOver = kSFull + kStages,      // its tiles and its buffer are free (9 arrivals)
    kPFull = kOver + kStages,      // second walk: P and dS are written (8 arrivals)
    kOutDone = kPFull + kStages,
    kSDrain,                   // two issuers
    kODrain = kSDrain + kSets,
    kBars
};

template <int DH, bool KEYS>
struct BwdCfg {
    static constexpr int ROW = 2 * DH;                       // bytes per row, one swizzle atom
    static constexpr uint32_t SW = DH == 64 ? kSwizzle128 : DH == 32 ? kSwizzle64 : kSwizzle32;
    static constexpr int OWN = 128 * ROW;                    // one own tile
    static constexpr int TILE = kStep * ROW;                 // one streamed tile
    static constexpr int STATS = 2 * TILE;                   // keys: inv, dhi, dlo of a step
    static constexpr int STAGE = 2 * TILE + 1024;
    static constexpr int STREAM = 2 * OWN;
    static constexpr int RED = STREAM + kStages * STAGE;     // queries: row sums of the two groups
    static constexpr int BAR = RED + kGroups * 2 * 128 * 8;
    static constexpr int SLOT = BAR + kBars * 8;
    static constexpr int NEED = SLOT + 16 + 1024;
    // over half an SM's shared memory: a second CTA could not have tensor memory
    static constexpr int BYTES = NEED > 118 * 1024 ? NEED : 118 * 1024;
    static constexpr uint32_t ACC = 128 * kBufs;             // first accumulator column
    static_assert(ACC + 2 * DH <= 512, "tensor-memory budget");
    static_assert(SLOT % 8 == 0 && BAR % 8 == 0, "barriers");
    static constexpr int S_WARP = kWorkerWarps, O_WARP = S_WARP + kSets, TMA_WARP = O_WARP + 1;
};

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Two fp32 values per instruction.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ F2 f2(uint32_t x, uint32_t y) {
    return f2(__uint_as_float(x), __uint_as_float(y));
}
__device__ __forceinline__ float2 un(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// Two values as bf16 pairs: rounded, and what the rounding left.
__device__ __forceinline__ void cut2(F2 x, uint32_t &up, uint32_t &low) {
    const float2 v = un(x);
    up = pack_bf16x2(v.x, v.y);
    low = pack_bf16x2(v.x - __uint_as_float(up << 16), v.y - __uint_as_float(up & 0xFFFF0000u));
}

template <int DH, bool KEYS>
__global__ void __launch_bounds__(kThreads, 1)
    backward_kernel(const __grid_constant__ CUtensorMap own0, const __grid_constant__ CUtensorMap own1,
                    const __grid_constant__ CUtensorMap str0, const __grid_constant__ CUtensorMap str1,
                    BwdParams p) {
    using L = BwdCfg<DH, KEYS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::BAR);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + L::SLOT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.x % p.heads;
    // the longest walks launch first: the last queries, the first keys
    const int at = blockIdx.x / p.heads, tile = KEYS ? at : p.tiles - 1 - at;
    const ErrCtx err{p.err};
    // steps of one walk: keys up to the diagonal, or queries from it on
    const int first = KEYS ? 2 * tile : 0;
    const int walk = KEYS ? p.steps - first : min(2 * tile + 2, p.steps);
    const int n1 = KEYS ? 0 : walk;  // steps of the first (statistics) walk
    const int n = n1 + walk;
    auto step_of = [&](int s) { return first + (s < n1 ? s : s - n1); };
    // step s is over: the workers have read its S and dP and, in the second walk,
    // the output products have completed
    auto wait_over = [&](int st, int par, unsigned int code) {
        return mbar_wait(&bar[kOver + st], par, err, code);
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) {
            const bool over = i >= kOver && i < kOver + kStages;
            const bool full = i >= kPFull && i < kPFull + kStages;
            mbar_init(&bar[i], over ? 9 : full ? 8 : 1);
        }
        cta_abort_clear();
        fence_barrier_init();
    }
    // Whatever the stream ran before, ahead of taking tensor memory that it may still want.
    // (The keys' kernel starts once every CTA of this one has its own and is past this.)
    if (!KEYS) grid_dependency_wait();
    if (warp == L::S_WARP) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;

    if (warp == L::TMA_WARP) {
        if (lane == 0) {
            prefetch_tensormap(&own0);
            prefetch_tensormap(&own1);
            prefetch_tensormap(&str0);
            prefetch_tensormap(&str1);
            mbar_arrive_expect_tx(&bar[kOwn], 2 * L::OWN);
            for (int h = 0; h < 2; ++h) {  // boxes are 64 rows high
                tma_load_3d(sm + h * L::TILE, &own0, 0, tile * 128 + h * kStep, head, &bar[kOwn]);
                tma_load_3d(sm + L::OWN + h * L::TILE, &own1, 0, tile * 128 + h * kStep, head,
                            &bar[kOwn]);
            }
            // the keys start on their own tiles while the last queries finish
            if (KEYS)
                grid_dependency_wait();
            else
                launch_dependents();
            int issued = 0;
            for (int s = 0, st = 0, par = 1; s < n; ++s) {
                if (s >= kStages && !wait_over(st, par, 0x801)) break;
                uint8_t *d = sm + L::STREAM + st * L::STAGE;
                const int y = step_of(s) * kStep;
                mbar_arrive_expect_tx(&bar[kTileFull + st], 2 * L::TILE + (KEYS ? 3 * 4 * kStep : 0));
                tma_load_3d(d, &str0, 0, y, head, &bar[kTileFull + st]);
                tma_load_3d(d + L::TILE, &str1, 0, y, head, &bar[kTileFull + st]);
                if (KEYS) {
                    const size_t at = (size_t)head * p.pitch + y;
                    bulk_load(d + L::STATS, p.inv + at, 4 * kStep, &bar[kTileFull + st]);
                    bulk_load(d + L::STATS + 4 * kStep, p.dhi + at, 4 * kStep, &bar[kTileFull + st]);
                    bulk_load(d + L::STATS + 8 * kStep, p.dlo + at, 4 * kStep, &bar[kTileFull + st]);
                }
                ++issued;
                if (++st == kStages) st = 0, par ^= 1;
            }
            // no copy may be in flight when the CTA exits: the last one on each barrier
            mbar_drain(&bar[kOwn], 0, err, 0x802);
            for (int s = issued - kStages < 0 ? 0 : issued - kStages; s < issued; ++s)
                mbar_drain(&bar[kTileFull + s % kStages], (s / kStages) & 1, err, 0x803);
        }
    } else if (warp >= L::S_WARP && warp < L::S_WARP + kSets) {
        if (lane == 0) {
            // S = own0 str0^T and dP = own1 str1^T into buffer s % kBufs, every kSets-th step
            const int me = warp - L::S_WARP;
            const uint32_t id = idesc_bf16(128, kStep, 0, 0);
            const uint32_t own = smem_u32(sm);
            const uint64_t a0 = smem_desc(own, 16, 8 * L::ROW, L::SW);
            const uint64_t a1 = smem_desc(own + L::OWN, 16, 8 * L::ROW, L::SW);
            const uint64_t db = smem_desc(own + L::STREAM, 16, 8 * L::ROW, L::SW);
            bool ok = mbar_wait(&bar[kOwn], 0, err, 0x810);
            for (int s = me, st = me, par = 0; ok && s < n; s += kSets) {
                const bool up = st >= kBufs;  // step s - kBufs used the buffer last
                ok = (s < kBufs || wait_over(up ? st - kBufs : st + kBufs, up ? par : par ^ 1, 0x811)) &&
                     mbar_wait(&bar[kTileFull + st], par, err, 0x812);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + 128 * (up ? st - kBufs : st);
                const uint64_t t0 = db + (uint32_t)(st * (L::STAGE >> 4)), t1 = t0 + (L::TILE >> 4);
#pragma unroll
                for (int kk = 0; kk < DH / 16; ++kk)  // 16 columns = 32 bytes on
                    mma_ss(d, a0 + 2 * kk, t0 + 2 * kk, id, kk > 0);
#pragma unroll
                for (int kk = 0; kk < DH / 16; ++kk)
                    mma_ss(d + 64, a1 + 2 * kk, t1 + 2 * kk, id, kk > 0);
                mma_commit(&bar[kSFull + st]);
                if (s < n1) mbar_arrive(&bar[kOver + st]);  // in the output products' place
                if ((st += kSets) >= kStages) st -= kStages, par ^= 1;
            }
            mma_commit(&bar[kSDrain + me]);
            mbar_drain(&bar[kSDrain + me], 0, err, 0x814);
        }
    } else if (warp == L::O_WARP) {
        if (lane == 0) {
            // queries: dQ += dS K;  keys: dK += dS^T Q and dV += P^T dO
            const uint32_t id = idesc_bf16(128, DH, 0, 1);
            const uint64_t db = smem_desc(smem_u32(sm) + L::STREAM, 16, 8 * L::ROW, L::SW);
            bool ok = true;
            uint32_t phases = 0;  // a bit per stage: kPFull is used in the second walk only
            for (int s = n1, st = n1 % kStages; s < n; ++s) {
                ok = mbar_wait(&bar[kPFull + st], (phases >> st) & 1, err, 0x820);
                if (!ok) break;
                phases ^= 1u << st;
                tc_fence_after();
                const uint64_t t0 = db + (uint32_t)(st * (L::STAGE >> 4)), t1 = t0 + (L::TILE >> 4);
                const uint32_t buf = tmem + 128 * (st >= kBufs ? st - kBufs : st);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {  // 16 rows on; the lower parts first
                    const uint32_t a = buf + 16 * kk + 64;
                    mma_ts(tmem + L::ACC, a + kLower, t0 + kk * L::ROW, id, s > n1 || kk > 0);
                    mma_ts(tmem + L::ACC, a, t0 + kk * L::ROW, id, 1);
                }
                if (KEYS) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t a = buf + 16 * kk;
                        mma_ts(tmem + L::ACC + DH, a + kLower, t1 + kk * L::ROW, id, s > n1 || kk > 0);
                        mma_ts(tmem + L::ACC + DH, a, t1 + kk * L::ROW, id, 1);
                    }
                }
                mma_commit(&bar[kOver + st]);
                if (++st == kStages) st = 0;
            }
            if (ok) mma_commit(&bar[kOutDone]);
            mma_commit(&bar[kODrain]);
            mbar_drain(&bar[kODrain], 0, err, 0x821);
        }
    } else if (warp < kWorkerWarps) {
        // ---------------- workers: thread = own row = tensor-memory lane ----------------
        const int group = warp >> 2, i = threadIdx.x & 127, row = tile * 128 + i;
        const int set = group >> 1, half = 32 * (group & 1);  // this group's columns
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        bool ok = true;
        float inv = 0.f, dhi = 0.f, dlo = 0.f;
        int s = set, st = set, par = 0;  // this set's steps
        auto next = [&] {
            s += kSets;
            if ((st += kSets) >= kStages) st -= kStages, par ^= 1;
        };

        // columns c .. c + 15 of S and dP (complete after tmem_ld_wait)
        auto load = [&](int b, int c, uint32_t (&s)[16], uint32_t (&dp)[16]) {
            tmem_ld16(lanes + 128 * b + c, s);
            tmem_ld16(lanes + 128 * b + 64 + c, dp);
        };
        // waits for the loads; ties the values to the wait, so that nothing that uses them moves above it
        auto arrived = [&](uint32_t (&s)[16], uint32_t (&dp)[16]) {
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(s[e]), "+r"(dp[e]));
        };
        // columns a row does not see count as a score of zero
        auto mask = [&](int col0, uint32_t (&s)[16]) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (KEYS ? col0 + e < row : col0 + e > row) s[e] = 0u;
        };
        auto on_diagonal = [&](int step) {
            return KEYS ? step < 2 * tile + 2 : step >= 2 * tile;
        };

        if (!KEYS) {
            double den = 0.0, num = 0.0;
            for (; s < n1; next()) {
                const int b = st >= kBufs ? st - kBufs : st, step = step_of(s);
                if (!(ok = warp_wait(&bar[kSFull + st], par, err, 0x830))) break;
                tc_fence_after();
                F2 d2 = f2(0.f, 0.f), n2 = d2;
                uint32_t sv[2][16], dv[2][16];
                load(b, half, sv[0], dv[0]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {  // the next columns load while these are summed
                    uint32_t(&x)[16] = sv[c & 1];
                    uint32_t(&y)[16] = dv[c & 1];
                    arrived(x, y);
                    if (c == 0) load(b, half + 16, sv[1], dv[1]);
                    if (on_diagonal(step)) mask(step * kStep + half + 16 * c, x);
                    if (tile == 0) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const double v = __uint_as_float(x[e]), w = v * v;
                            den += w;
                            num = ::fma(w, (double)__uint_as_float(y[e]), num);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const F2 v = f2(x[e], x[e + 1]), w = mul(v, v);
                            d2 = add(d2, w);
                            n2 = fma(w, f2(y[e], y[e + 1]), n2);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kOver + st]);
                const float2 a = un(d2), c = un(n2);
                den += (double)a.x + (double)a.y;
                num += (double)c.x + (double)c.y;
            }
            // join the two groups' sums
            double *red = reinterpret_cast<double *>(sm + L::RED);
            red[group * 256 + i] = den;
            red[group * 256 + 128 + i] = num;
            ok = bar_sync_and(1, 32 * kWorkerWarps, ok);
            den = (double)p.eps;
            num = 0.0;
            for (int g = 0; g < kGroups; ++g) {
                den += red[g * 256 + i];
                num += red[g * 256 + 128 + i];
            }
            if (!(den < (double)FLT_MIN)) {  // below it 1 / den may be infinite in fp32
                const double minus = -num / den;
                inv = (float)(1.0 / den);
                dhi = (float)minus;
                dlo = (float)(minus - (double)dhi);
            }
            if (ok && group == 0) {  // rows from T on: zeros, which make their keys' terms zero
                const size_t at = (size_t)head * p.pitch + row;
                const bool have = row < p.T;
                p.inv[at] = have ? inv : 0.f;
                p.dhi[at] = have ? dhi : 0.f;
                p.dlo[at] = have ? dlo : 0.f;
            }
        }
        // dS / 2 = (s / den) (dP - delta), P = s (s / den); the factor 2 comes at the end
        for (; ok && s < n; next()) {
            const int b = st >= kBufs ? st - kBufs : st, step = step_of(s);
            if (!(ok = warp_wait(&bar[kSFull + st], par, err, 0x831))) break;
            tc_fence_after();
            // the statistics arrived with the step's tiles, before its products
            if (KEYS && !(ok = warp_wait(&bar[kTileFull + st], par, err, 0x832))) break;
            const float *stats = reinterpret_cast<const float *>(sm + L::STREAM + st * L::STAGE + L::STATS);
            const bool few = KEYS ? step < 2 : tile == 0;  // rows that may see few keys
            uint32_t sv[2][16], dv[2][16];
            load(b, half, sv[0], dv[0]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t(&x)[16] = sv[c & 1];
                uint32_t(&y)[16] = dv[c & 1];
                arrived(x, y);
                if (c == 0) load(b, half + 16, sv[1], dv[1]);
                if (on_diagonal(step)) mask(step * kStep + half + 16 * c, x);
                uint32_t pu[8], pl[8], du[8], dl_[8];  // upper and lower parts of P and dS
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float4 iv = make_float4(inv, inv, inv, inv), dh = make_float4(dhi, dhi, dhi, dhi);
                    float4 dl = make_float4(dlo, dlo, dlo, dlo);
                    if (KEYS) {
                        const float *at = stats + half + 16 * c + e;
                        iv = *reinterpret_cast<const float4 *>(at);
                        dh = *reinterpret_cast<const float4 *>(at + kStep);
                        if (few) dl = *reinterpret_cast<const float4 *>(at + 2 * kStep);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const F2 v = f2(x[e + 2 * h], x[e + 2 * h + 1]);
                        const F2 w = mul(v, h ? f2(iv.z, iv.w) : f2(iv.x, iv.y));
                        F2 t = add(f2(y[e + 2 * h], y[e + 2 * h + 1]),
                                   h ? f2(dh.z, dh.w) : f2(dh.x, dh.y));
                        if (few) t = add(t, h ? f2(dl.z, dl.w) : f2(dl.x, dl.y));
                        cut2(mul(w, t), du[e / 2 + h], dl_[e / 2 + h]);
                        if (KEYS) cut2(mul(v, w), pu[e / 2 + h], pl[e / 2 + h]);
                    }
                }
                // over the sixteen columns of S and of dP that these come from
                const uint32_t at = lanes + 128 * b + half + 16 * c;
                if (KEYS) {
                    tmem_st8(at, pu);
                    tmem_st8(at + kLower, pl);
                }
                tmem_st8(at + 64, du);
                tmem_st8(at + 64 + kLower, dl_);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar[kPFull + st]);
                mbar_arrive(&bar[kOver + st]);
            }
        }
        // half of the columns each (sixteen at least): set 0 those of dQ or dK, set 1
        // (keys) those of dV
        constexpr int COLS = DH >= 32 ? DH / 2 : DH;
        if (ok)
            ok = (KEYS || set == 0) && (DH >= 32 || (group & 1) == 0) &&
                 warp_wait(&bar[kOutDone], 0, err, 0x833);
        tc_fence_after();
        const uint32_t col0 = L::ACC + set * DH + (group & 1) * COLS;
        const float scale = set == 0 ? 2.f : 1.f;
        __nv_bfloat16 *out = set == 0 ? p.out0 : p.out1;
        uint4 *dst = reinterpret_cast<uint4 *>(out + ((size_t)head * p.T + row) * DH +
                                               (group & 1) * COLS);
#pragma unroll
        for (int c = 0; c < COLS; c += 16) {
            if (!ok) break;
            uint32_t r[16];
            tmem_ld16(lanes + col0 + c, r);
            tmem_ld_wait();
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = pack_bf16x2(scale * __uint_as_float(r[2 * e]),
                                   scale * __uint_as_float(r[2 * e + 1]));
            if (row < p.T) {
                dst[c / 8] = make_uint4(o[0], o[1], o[2], o[3]);
                dst[c / 8 + 1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == L::S_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// [heads, T, d] in boxes of 64 rows x d columns; rows past T are zero-filled.
bool map_rows(CUtensorMap *m, const void *base, int d, int T, long heads) {
    auto enc = get_encode();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)T * d * 2};
    cuuint32_t box[3] = {(cuuint32_t)d, (cuuint32_t)kStep, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               d == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
               : d == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                         : CU_TENSOR_MAP_SWIZZLE_32B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DH>
cudaError_t launch(const PrefillBackwardArgs &a, cudaStream_t stream) {
    CUtensorMap mq, mk, mv, mo;
    if (!map_rows(&mq, a.q, DH, a.T, a.heads) || !map_rows(&mk, a.k, DH, a.T, a.heads) ||
        !map_rows(&mv, a.v, DH, a.T, a.heads) || !map_rows(&mo, a.d_o, DH, a.T, a.heads))
        return cudaErrorInvalidValue;
    BwdParams p;
    p.T = a.T;
    p.heads = (int)a.heads;
    p.tiles = (a.T + 127) / 128;
    p.steps = (a.T + kStep - 1) / kStep;
    p.pitch = 128L * p.tiles;
    p.eps = a.eps;
    p.inv = static_cast<float *>(a.ws);
    p.dhi = p.inv + a.heads * p.pitch;
    p.dlo = p.dhi + a.heads * p.pitch;
    p.err = a.err;
    const unsigned grid = (unsigned)(a.heads * p.tiles);
    cudaError_t e;
    using Q = BwdCfg<DH, false>;
    using K = BwdCfg<DH, true>;
    if ((e = set_smem_once<backward_kernel<DH, false>>(Q::BYTES)) != cudaSuccess) return e;
    if ((e = set_smem_once<backward_kernel<DH, true>>(K::BYTES)) != cudaSuccess) return e;
    p.out0 = static_cast<__nv_bfloat16 *>(a.dq);
    p.out1 = nullptr;
    e = launch_overlapped(backward_kernel<DH, false>, grid, kThreads, Q::BYTES, stream, mq, mo, mk, mv, p);
    if (e != cudaSuccess || (e = after_launch()) != cudaSuccess) return e;
    p.out0 = static_cast<__nv_bfloat16 *>(a.dk);
    p.out1 = static_cast<__nv_bfloat16 *>(a.dv);
    e = launch_overlapped(backward_kernel<DH, true>, grid, kThreads, K::BYTES, stream, mk, mv, mq, mo, p);
    return e != cudaSuccess ? e : after_launch();
}

}  // namespace

size_t prefill_backward_tc_workspace_bytes(long heads, int T) {
    return (size_t)heads * ((T + 127) / 128) * 128 * 3 * sizeof(float);
}

cudaError_t prefill_backward_tc(const PrefillBackwardArgs &a, cudaStream_t stream) {
    switch (a.d) {
        case 16: return launch<16>(a, stream);
        case 32: return launch<32>(a, stream);
        case 64: return launch<64>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kata
