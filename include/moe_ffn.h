/*
 * moe_ffn.h - C ABI of the feed-forward operators of libmoe_route: what runs
 * on the rows that the routing calls of moe_route.h lay out, and on the
 * tokens themselves (shared experts, dense blocks).
 *
 *   moe_gated_ffn             h = act(x Wg^T) * (x Wu^T), one kernel
 *   moe_gated_ffn_backward    dx, dWg, dWu from dh and the pre-activations
 *   moe_linear                y = act(x W^T + bias) + residual, one kernel
 *   moe_linear_backward       dx, dW, dbias from dy (and the pre-activations)
 *   moe_combine               out[t] = residual[t] + sum_k w[t,k] y[row(t,k)]
 *   moe_combine_backward      dy and dw from dout
 *
 * Conventions, beside those of moe_route.h (device pointers owned by the
 * caller, asynchronous on `stream`, arguments checked on the host before
 * anything is launched, deterministic results, no allocation):
 *  - Matrices hold bf16 or fp16 (moe_dtype), all of a call the same; sums are
 *    fp32 and each output is rounded once. Inside moe_gated_ffn_backward and
 *    moe_linear_backward the gradient of the pre-activations (dg and du, or dz)
 *    is rounded once to the matrices' type before the two products that take
 *    it, so it has that type's range too: with fp16 one above 65504 becomes
 *    infinite, and its row of dx and its column's dw with it, and one below
 *    3e-8 is lost before the sums (a loss scale has to leave room for
 *    dh * u * act'). Bf16 has the range of fp32. Linear calls without an
 *    activation have nothing to round, and weight gradients of up to 8 rows,
 *    or rows an expert, take it unrounded and in fp32's range.
 *  - A moe_matrix has contiguous columns and rows `ld` elements apart; a
 *    stack of one matrix per expert has them `stride` elements apart. Any ld
 *    from the columns up to MOE_FFN_MAX_LD (rows that lie further apart are
 *    copied by the caller), any stride and any element alignment works.
 *    The matrix cores read 16-byte pieces: an operand of a product whose
 *    pointer, ld, stride or columns are no multiple of 8 elements is first
 *    copied into the workspace with its rows padded (but for forward
 *    products over experts with few rows, which read them in place).
 *  - Dense form: rows.num_experts = 0, the rows are the tokens.
 *  - Expert form: rows.num_experts = n experts with weights, ids 0 .. n-1 of
 *    a grouped layout (moe_grouped_layout, moe_route_local_grouped). A row r
 *    belongs to expert m_indices[r]. Every row of an output is written: one
 *    that is padding, or whose id is n or above (an expert of another rank),
 *    with zeros. The layout's rows end with the other ranks' entries, so a
 *    call may be given fewer rows than the layout has (a prefix of m_indices
 *    and row_entry); entries beyond it are left out of every operator.
 *  - Nothing reads the contents of rows without an entry, so they may hold
 *    anything.
 *  - Workspaces need no initial contents and nothing in them lasts.
 */
#ifndef MOE_FFN_H
#define MOE_FFN_H

#include <stddef.h>
#include <stdint.h>

#include "moe_route.h" /* moe_status */

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_dtype { MOE_BF16 = 0, MOE_F16 = 1 } moe_dtype;

/* silu: z / (1 + e^-z). gelu: z (1 + erf(z / sqrt 2)) / 2. */
typedef enum moe_activation { MOE_ACT_NONE = 0, MOE_ACT_SILU = 1, MOE_ACT_GELU = 2 } moe_activation;

/* Envelope: widths (hidden, inter, out) 1 .. 2^20, tokens and rows up to 2^30,
 * ld up to 2^22 elements, at most 4096 experts, tile_m a multiple of 16 up to
 * MOE_GROUPED_MAX_TILE. What lies beyond is refused with MOE_ERR_UNSUPPORTED. */
#define MOE_FFN_MAX_WIDTH (1 << 20)
#define MOE_FFN_MAX_ROWS (1 << 30)
#define MOE_FFN_MAX_LD (1 << 22)
#define MOE_FFN_MAX_EXPERTS 4096

typedef struct moe_matrix {
  void *p;        /* element type moe_dtype; NULL where a matrix is optional */
  int64_t ld;     /* elements from one row to the next                      */
  int64_t stride; /* elements from one expert's matrix to the next          */
} moe_matrix;

typedef struct moe_expert_rows {
  const int32_t *counts;         /* [>= num_experts] entries of each expert;
                                    read by the backward passes                */
  const int32_t *padded_offsets; /* [>= num_experts + 1] first row of each     */
  const int32_t *m_indices;      /* [rows] expert of each row, -1 on padding   */
  const int32_t *row_entry;      /* [rows] entry t * top_k + k of each row, -1;
                                    NULL: moe_gated_ffn's x has a row per row  */
  int64_t rows;                  /* rows of the row-wise matrices of this call */
  int32_t num_experts;           /* experts with weights; 0: dense             */
  int32_t tile_m;                /* the layout's row alignment                 */
  int32_t top_k;                 /* entries per token                          */
} moe_expert_rows;

/*
 * Gated feed-forward block, and its backward pass.
 *   x [tokens, hidden]: token rows, gathered through row_entry in the expert
 *       form; with row_entry NULL, or dense, row r of x belongs to row r;
 *   w_gate, w_up [inter, hidden] per expert;
 *   h [rows, inter] = act(g) * u with g = x Wg^T, u = x Wu^T;
 *   pre [rows, 2 inter] (p NULL: not written): g in the first inter columns,
 *       u in the others, what the backward pass reads.
 * Backward: dg = dh u act'(g), du = dh act(g),
 *   dx [rows, hidden] = dg Wg + du Wu: one row per ROW, also where x is
 *       gathered (moe_combine with unit weights sums them into tokens);
 *   dw_gate, dw_up [inter, hidden] per expert = dg^T x, du^T x (zeros for an
 *       expert without rows).
 * Any of dx and the pair (dw_gate, dw_up) may be left out (p NULL).
 */
typedef struct moe_gated_ffn_args {
  int32_t dtype, activation;
  int64_t tokens; /* rows of x */
  int32_t hidden, inter;
  moe_expert_rows rows;
  moe_matrix x, w_gate, w_up, h, pre;
  moe_matrix dh, dx, dw_gate, dw_up; /* backward only */
} moe_gated_ffn_args;

/* Bytes of workspace a call needs (0 where it needs none), or -1 for
 * arguments that the call refuses. */
int64_t moe_gated_ffn_workspace_bytes(const moe_gated_ffn_args *a, int32_t backward);
int moe_gated_ffn(const moe_gated_ffn_args *a, void *workspace, size_t workspace_bytes,
                  void *stream);
int moe_gated_ffn_backward(const moe_gated_ffn_args *a, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * Linear product with its epilogue, and its backward pass.
 *   x [rows, in], w [out, in] per expert, bias [out] per expert (bias.stride
 *   apart; p NULL: none), residual [rows, out] (p NULL: none);
 *   z = x W^T + bias, y [rows, out] = act(z) + residual,
 *   pre [rows, out] (p NULL: not written): z, what the backward pass reads
 *       when there is an activation.
 * Backward: dz = dy act'(pre), or dy without an activation;
 *   dx [rows, in] = dz W, dw [out, in] = dz^T x, dbias [out] = sum of dz's
 *   rows, per expert. The gradient of the residual is dy itself (on rows
 *   with an entry: the others' y is zero whatever the residual holds). Any of
 *   dx, dw and dbias may be left out (p NULL).
 */
typedef struct moe_linear_args {
  int32_t dtype, activation;
  int64_t tokens; /* rows in the dense form */
  int32_t in, out;
  moe_expert_rows rows; /* row_entry and top_k are not used */
  moe_matrix x, w, bias, residual, y, pre;
  moe_matrix dy, dx, dw, dbias; /* backward only */
} moe_linear_args;

int64_t moe_linear_workspace_bytes(const moe_linear_args *a, int32_t backward);
int moe_linear(const moe_linear_args *a, void *workspace, size_t workspace_bytes, void *stream);
int moe_linear_backward(const moe_linear_args *a, void *workspace, size_t workspace_bytes,
                        void *stream);

/*
 * The experts' rows summed into their tokens, and the backward pass.
 *   y [rows, width]; packed, inv_perm [tokens, top_k], offsets and
 *   padded_offsets of the routing call: entry (t, k) has id e = packed >> 16
 *   and row inv_perm - offsets[e] + padded_offsets[e]. Entries whose id is
 *   num_experts or above, or whose row is rows or above, are left out.
 *   weights [tokens, top_k] fp32 (NULL: unit weights)
 *   out [tokens, width] = residual (p NULL: zeros) + sum over k of w y,
 *   summed in fp32 in the order of k.
 * Backward: dy [rows, width]: weight times dout of the row's token, zeros on
 *   rows without an entry; dweights [tokens, top_k] fp32 (NULL: not
 *   computed) = <dout[t], y[row]>, 0 for entries left out. It walks the rows
 *   through m_indices and row_entry. The gradient of the residual is dout.
 */
typedef struct moe_combine_args {
  int32_t dtype, width;
  int64_t tokens, rows;
  int32_t top_k, num_experts;
  int32_t num_ids; /* ids of the routing call: offsets has num_ids + 1 elements */
  const int32_t *packed, *inv_perm, *offsets, *padded_offsets;
  const int32_t *m_indices, *row_entry; /* backward only */
  const float *weights;
  moe_matrix y, residual, out;
  moe_matrix dout, dy; /* backward only */
  float *dweights;     /* backward only */
} moe_combine_args;

int moe_combine(const moe_combine_args *a, void *stream);
int moe_combine_backward(const moe_combine_args *a, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FFN_H */
