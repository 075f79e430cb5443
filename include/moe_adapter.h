/*
 * moe_adapter.h - C ABI of the projection of libmoe_route with the low-rank
 * adapters of many requests beside it, for serving them together (a token has
 * the adapter of its request) and for training several of them at once.
 *
 *   moe_adapter_linear           y = x W^T + bias + s B_a^T + residual, s = c_a x A_a^T
 *   moe_adapter_linear_backward  dx, dA, dB
 *
 * Conventions: those of moe_ffn.h (device pointers owned by the caller,
 * asynchronous on `stream`, arguments checked on the host before anything is
 * launched, deterministic results, no allocation; bf16 or fp16, one type a
 * call, fp32 sums, one rounding of each output; any ld from the columns up to
 * MOE_FFN_MAX_LD and any element alignment; workspaces without initial
 * contents).
 */
#ifndef MOE_ADAPTER_H
#define MOE_ADAPTER_H

#include "moe_ffn.h" /* moe_dtype, moe_matrix */

#ifdef __cplusplus
extern "C" {
#endif

/* Envelope, beside MOE_FFN_MAX_WIDTH, MOE_FFN_MAX_ROWS and MOE_FFN_MAX_LD: what
 * lies beyond is refused with MOE_ERR_UNSUPPORTED. */
#define MOE_ADAPTER_MAX_RANK 128
#define MOE_ADAPTER_MAX 4096

/*
 * Linear product with a low-rank adapter for each token, and its backward pass.
 *   x [tokens, in], w [out, in], bias [out] and residual [tokens, out] (NULL:
 *   none) as moe_linear's without an activation;
 *   a [rank, in] and b [out, rank] of each of the `adapters`, stride elements
 *   apart; scale [adapters] fp32 (NULL: 1);
 *   ids [tokens]: the token's adapter; a number outside 0 .. adapters-1: none.
 *   s [tokens, rank] fp32, contiguous = scale[id] x A_id^T, 0 without an adapter
 *       (NULL: kept in the workspace; the backward pass reads it);
 *   y [tokens, out] = x W^T + bias + s B_id^T + residual.
 * Backward: u = scale[id] dy B_id,
 *   dx [tokens, in] = dy W + u A_id,
 *   da [rank, in] and db [out, rank] of each adapter = sum over its tokens of
 *       u^T x and of dy^T s, zeros for one without tokens.
 * W has no gradient here (moe_linear_backward computes it). Any of dx, da and db
 * may be left out (p NULL). The workspace holds a transposed copy of A and B for as many
 * adapters as there are tokens at most, and sums of a size that does not grow with the
 * adapters beyond that.
 * s and u are fp32, and so is what is multiplied with them, or the matrix cores take
 * them in three parts of the type, which hold all of their bits (in fp16, at a power of
 * two of their own, down to 2^-38 of the largest of 32 values).
 */
typedef struct moe_adapter_linear_args {
  int32_t dtype, rank;
  int64_t tokens;
  int32_t in, out;
  int32_t adapters, reserved; /* 0 */
  moe_matrix x, w, a, b, bias, residual, y;
  const int32_t *ids;
  const float *scale;
  float *s; /* written by the forward pass, read by the backward pass */
  moe_matrix dy, dx, da, db; /* backward only */
} moe_adapter_linear_args;

int64_t moe_adapter_linear_workspace_bytes(const moe_adapter_linear_args *a, int32_t backward);
int moe_adapter_linear(const moe_adapter_linear_args *a, void *workspace, size_t workspace_bytes,
                       void *stream);
int moe_adapter_linear_backward(const moe_adapter_linear_args *a, void *workspace,
                                size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ADAPTER_H */
