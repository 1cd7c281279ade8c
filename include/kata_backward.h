/*
 * kata_backward.h -- gradients of kata_prefill in libkata.so, on NVIDIA B200
 * (sm_100a). The conventions are those of kata.h.
 */
#ifndef KATA_BACKWARD_H
#define KATA_BACKWARD_H

#include "kata.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device workspace bytes kata_prefill_backward needs (0: invalid sizes): 16
 * for each token of a head in fp32, 12 in bf16 with T rounded up to 128. */
KATA_API size_t kata_prefill_backward_workspace_bytes(int B, int H, int T, int d, int dtype);

/*
 * Gradients of the output of kata_prefill from a zero state,
 *   o_i = sum_{j<=i} (q_i.k_j)^2 v_j / (sum_{j<=i} (q_i.k_j)^2 + eps),
 * with respect to q, k and v. The weights are recomputed from q and k; nothing
 * of the forward call is needed, o included. Work is quadratic in T.
 *   q, k, v      [B, H, T, d], dtype KATA_F32 or KATA_BF16; d 16, 32 or 64;
 *                T any positive number (no multiple is asked for).
 *   d_o          [B, H, T, d] gradient of o, in the dtype of q.
 *   dq, dk, dv   [B, H, T, d], dtype of q. Outputs or a workspace that overlap
 *                each other or an input are refused.
 *   workspace    device scratch of at least
 *                kata_prefill_backward_workspace_bytes(); calls that may run
 *                at the same time need one each.
 * Deterministic. Inputs are expected finite, up to the last token, and so are the
 * scores' squares in fp32: a NaN or an infinity reaches the whole 64- or 128-token
 * tile it lies in. A row whose denominator is below 2^-126, fp32's smallest normal
 * number (eps = 0, and every score next to 0), has no defined output; its
 * gradients are taken as 0.
 */
KATA_API int kata_prefill_backward(const void *q, const void *k, const void *v, int dtype, int B,
                                   int H, int T, int d, float eps, const void *d_o, void *dq,
                                   void *dk, void *dv, void *workspace, size_t ws_bytes,
                                   void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KATA_BACKWARD_H */
