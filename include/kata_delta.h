/*
 * kata_delta.h -- the gated delta rule in libkata.so: chunked prefill,
 * one-token step and gradients, on NVIDIA B200 (sm_100a).
 *
 * The conventions are those of kata.h (row-major, 16-byte aligned device
 * pointers, caller-owned buffers, asynchronous on `stream`, arguments
 * validated on the host before any launch, kata_status returned and
 * kata_last_error() set), with these differences of this family:
 *   - the state is S [B, H, d, d] fp32, key rows and value columns (no packed
 *     feature, no normaliser);
 *   - o and the gradients of q, k, v have the dtype of q, k, v: what the next
 *     layer's product reads. g, beta, their gradients and the states are fp32;
 *   - d may be 16, 32, 64 or 128, and T any positive number;
 *   - g, beta, dg and dbeta need 4-byte alignment only.
 *
 * Per (b, h), token by token:
 *   e_t = v_t - exp(g_t) S_{t-1}^T k_t
 *   S_t = exp(g_t) S_{t-1} + beta_t k_t e_t^T
 *   o_t = scale S_t^T q_t
 * g_t is the log of the decay, <= 0 in use (values below -200 count as -200:
 * exp of either is 0 in fp32; minus infinity starts the state anew, from values
 * that are finite themselves: 0 times an infinity or a NaN is a NaN); beta_t is
 * the writing strength. Keys are used as given: callers that want unit keys
 * normalise them. A token with beta = 0 and g = 0 leaves the state as it is,
 * so shorter sequences of a padded batch are padded with such tokens (with
 * finite q, k and v: a NaN or an infinity reaches the whole 64-token chunk it
 * lies in, and the state).
 */
#ifndef KATA_DELTA_H
#define KATA_DELTA_H

#include "kata.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device workspace bytes kata_delta_prefill needs (0: invalid sizes): 4 (128 d +
 * 4352) for each 64 tokens of a head, 50 KB at d = 64. */
KATA_API size_t kata_delta_prefill_workspace_bytes(int B, int H, int T, int d, int dtype);

/*
 * The rule over T tokens, in chunks of 64 (the chunked form is exact).
 *   q, k, v   [B, H, T, d], dtype KATA_F32 or KATA_BF16.
 *   g, beta   [B, H, T] fp32.
 *   S_in      [B, H, d, d] first state; NULL = zero.
 *   o         [B, H, T, d], dtype of q; NULL: not computed.
 *   S_out     [B, H, d, d] last state; NULL: not written; may be S_in. One of
 *             o and S_out at least.
 *   workspace device scratch of at least
 *             kata_delta_prefill_workspace_bytes(); calls that may run at the
 *             same time need one each.
 * Buffers that overlap otherwise are refused.
 */
KATA_API int kata_delta_prefill(const void *q, const void *k, const void *v, int dtype,
                                const float *g, const float *beta, int B, int H, int T, int d,
                                float scale, const float *S_in, void *o, float *S_out,
                                void *workspace, size_t ws_bytes, void *stream);

/*
 * One token per (b, h): the state is updated IN PLACE, then read out.
 *   q, k, v  [B, H, d]; g, beta [B, H] fp32; S [B, H, d, d] fp32, read and
 *   written; o [B, H, d], dtype of q. S and o that overlap each other or
 *   another buffer are refused.
 */
KATA_API int kata_delta_decode_step(const void *q, const void *k, const void *v, int dtype,
                                    const float *g, const float *beta, int B, int H, int d,
                                    float scale, float *S, void *o, void *stream);

/* Device workspace bytes kata_delta_backward needs (0: invalid sizes): 8 (192 d +
 * d d + 256) for each 64 tokens of a head, 133 KB at d = 64 and 330 KB at d = 128
 * (1.1 GB for B = 2, H = 16, T = 16384, d = 64). */
KATA_API size_t kata_delta_backward_workspace_bytes(int B, int H, int T, int d, int dtype);

/*
 * Gradients of kata_delta_prefill. The states are recomputed from the inputs;
 * nothing of the forward call is needed.
 *   q, k, v, g, beta, S_in, scale   as given to kata_delta_prefill.
 *   d_o       [B, H, T, d] gradient of o, dtype of q.
 *   dS_out    [B, H, d, d] fp32 gradient of the last state; NULL = zero.
 *   dq, dk, dv  [B, H, T, d], dtype of q; dg, dbeta [B, H, T] fp32.
 *   dS_in     [B, H, d, d] fp32 gradient of the first state; NULL: not
 *             written; may be dS_out.
 * Buffers that overlap otherwise are refused. Deterministic. The
 * gradient of a g below -200 is that of -200 (0 to fp32 rounding of its
 * neighbours).
 */
KATA_API int kata_delta_backward(const void *q, const void *k, const void *v, int dtype,
                                 const float *g, const float *beta, int B, int H, int T, int d,
                                 float scale, const float *S_in, const void *d_o,
                                 const float *dS_out, void *dq, void *dk, void *dv, float *dg,
                                 float *dbeta, float *dS_in, void *workspace, size_t ws_bytes,
                                 void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KATA_DELTA_H */
