/*
 * moe_block.h - C ABI of the operators around the feed-forward block of
 * libmoe_route: the norm in front of the router and the experts, and dropout
 * of a sub-layer's output.
 *
 *   moe_rms_norm              h = residual + drop(x), y = h rstd weight, in 16
 *                             bits or as MXFP8
 *   moe_rms_norm_backward     dx, dresidual, dweight
 *   moe_dropout               out = residual + drop(x), and the backward pass
 *   moe_mxfp8_values          the values that MXFP8 codes and scales stand for
 *
 * Conventions: those of moe_ffn.h (device pointers owned by the caller,
 * asynchronous on `stream`, arguments checked on the host before anything is
 * launched, deterministic results, no allocation; bf16 or fp16, one type a
 * call, fp32 sums, one rounding of each output; any ld from the columns up to
 * MOE_FFN_MAX_LD and any element alignment; workspaces without initial
 * contents). An output may be one of the call's own inputs, the same elements
 * at the same places, in the norm and in dropout (h on residual, y on x).
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_ffn.h" /* moe_dtype, moe_matrix */

#ifdef __cplusplus
extern "C" {
#endif

/* Envelope, beside MOE_FFN_MAX_ROWS and MOE_FFN_MAX_LD: what lies beyond is
 * refused with MOE_ERR_UNSUPPORTED. */
#define MOE_NORM_MAX_WIDTH 32768
#define MOE_DROPOUT_MAX_SITE 32768

/*
 * Dropout: drop(v) of element (t, c) of a matrix is 0 where its 16-bit number is
 * below `level`, and v 2^16 / (2^16 - level) elsewhere: it is dropped with
 * probability level / 2^16. `level` 0: drop(v) = v, nothing is read; 2^16: all
 * are dropped. What is dropped has no effect, NaN and infinities too.
 * The numbers are those of Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
 * "Parallel random numbers: as easy as 1, 2, 3", 2011) with the key state[0]
 * and the counter (c / 8 + 2^17 site, t, state[1]), low words first: eight of
 * them, low halves first, for the elements 8 (c / 8) .. 8 (c / 8) + 7 of row t.
 * They depend on nothing else, so a backward pass with the same state and site
 * drops the same elements, and nothing is stored. `state` lies on the device:
 * a program adds to state[1] between its steps, in a captured graph too, and
 * tells its dropouts of one step apart by `site` (0 .. MOE_DROPOUT_MAX_SITE-1).
 */
typedef struct moe_dropout_spec {
  const uint64_t *state; /* [2] seed and offset; NULL allowed with level 0 */
  uint32_t level;        /* 0 .. 65536                                     */
  int32_t site;
} moe_dropout_spec;

/*
 * Root-mean-square norm with the residual's addition, and its backward pass.
 *   x, residual [tokens, width] (residual.p NULL: none), weight [width];
 *   h [tokens, width] = residual + drop(x), rounded to the type. Without a
 *       residual and without dropout h is x: h.p may be NULL, and has to be
 *       given in every other case;
 *   rstd [tokens] fp32 = 1 / sqrt(mean of the row's h^2 + eps) of the rounded
 *       h (NULL: not written; the backward pass reads it), also where the
 *       squares pass fp32's range. It is infinite, and y no number, where the mean
 *       plus eps is 0 or below 2^-256 (eps of 0 alone);
 *   y [tokens, width] = h rstd weight (p NULL: not written);
 *   q [tokens, width] E4M3 codes and q_scale [tokens, width / 32] E8M0 codes
 *       (both NULL: not written; width a multiple of 32) of the unrounded
 *       h rstd weight, in the form that moe_route_quant_local writes: scale
 *       2^s, s = max(floor(log2(largest of the 32)) - 8, -127), elements rounded
 *       to nearest even and saturating at +-448. A NaN gets the code of NaN.
 * At least one of y and q has to be written.
 * Backward: g = dy weight, n = h rstd,
 *   dtotal = dh + rstd (g - n mean(g n))  with dh (p NULL: 0) the gradient that
 *       reaches h from behind,
 *   dresidual [tokens, width] = dtotal (p NULL: not written), dx = drop(dtotal)
 *       (p NULL: not written; without dropout both are the same),
 *   dweight [width] = sum over the tokens of dy n (NULL: not computed).
 */
typedef struct moe_rms_norm_args {
  int32_t dtype, width;
  int64_t tokens;
  float eps;
  int32_t reserved; /* 0 */
  moe_dropout_spec drop;
  moe_matrix x, residual, h, y;
  const void *weight;
  float *rstd; /* written by the forward pass, read by the backward pass */
  uint8_t *q, *q_scale;
  moe_matrix dy, dh, dx, dresidual; /* backward only */
  void *dweight;                    /* backward only */
} moe_rms_norm_args;

int moe_rms_norm(const moe_rms_norm_args *a, void *stream);
/* Bytes of workspace of the backward pass (0 without dweight), or -1 for
 * arguments that it refuses. */
int64_t moe_rms_norm_backward_workspace_bytes(const moe_rms_norm_args *a, int32_t backward);
int moe_rms_norm_backward(const moe_rms_norm_args *a, void *workspace, size_t workspace_bytes,
                          void *stream);

/* out [tokens, width] = residual (p NULL: 0) + drop(x). The gradient of x is
 * the same call on the gradient of out without a residual; the residual's is
 * the gradient of out itself. Widths up to MOE_FFN_MAX_WIDTH. */
typedef struct moe_dropout_args {
  int32_t dtype, width;
  int64_t tokens;
  moe_dropout_spec drop;
  moe_matrix x, residual, out;
} moe_dropout_args;

int moe_dropout(const moe_dropout_args *a, void *stream);

/* values [count] (dtype) of count = 32 n E4M3 codes q and n E8M0 codes q_scale:
 * q 2^(q_scale - 127), rounded to the type (bf16 holds them all but for those
 * below its smallest). The scale code 255 and the element codes 0x7F and 0xFF
 * are NaN. */
int moe_mxfp8_values(const uint8_t *q, const uint8_t *q_scale, int64_t count, int32_t dtype,
                     void *values, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
