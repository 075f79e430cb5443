// block.hip - the C entry points of the norm, dropout and the MXFP8 values.
#include <math.h>

#include "block_rows.hpp"
#include "ffn_host.hpp"

namespace moe_block {

static int check_drop(const moe_dropout_spec &d) {
  if (d.level > 65536 || d.site < 0) return MOE_ERR_SHAPE;
  if (d.site >= MOE_DROPOUT_MAX_SITE) return MOE_ERR_UNSUPPORTED;
  if (d.level == 0) return MOE_OK;
  if (!d.state) return MOE_ERR_NULL;
  return (uintptr_t)d.state % 8 ? MOE_ERR_SHAPE : MOE_OK;
}
static Drop drop_of(const moe_dropout_spec &d) {
  const float times = d.level < 65536 ? (float)(65536.0 / (65536 - (int)d.level)) : 0.f;
  return {d.state, d.level, (uint32_t)d.site, times};
}

static int check_norm(const moe_rms_norm_args *a, bool backward) {
  if (!a) return MOE_ERR_NULL;
  if (a->dtype != MOE_BF16 && a->dtype != MOE_F16) return MOE_ERR_UNSUPPORTED;
  if (a->tokens < 0 || a->width <= 0 || a->reserved != 0) return MOE_ERR_SHAPE;
  if (a->width > MOE_NORM_MAX_WIDTH || a->tokens > MAX_ROWS) return MOE_ERR_UNSUPPORTED;
  if (!backward && !(a->eps >= 0.f && a->eps <= 3.4e38f)) return MOE_ERR_SHAPE;
  MOE_TRY(check_drop(a->drop));
  const int64_t T = a->tokens;
  const int W = a->width;
  if (!a->weight) return MOE_ERR_NULL;
  if ((uintptr_t)a->weight % 2 || (uintptr_t)a->rstd % 4) return MOE_ERR_SHAPE;
  if (!backward) {
    MOE_TRY(check_matrix(a->x, T, W, 1, false));
    MOE_TRY(check_matrix(a->residual, T, W, 1, true));
    MOE_TRY(check_matrix(a->h, T, W, 1, !a->residual.p && a->drop.level == 0));
    MOE_TRY(check_matrix(a->y, T, W, 1, a->q != nullptr));
    if (!a->q != !a->q_scale) return MOE_ERR_NULL;
    return a->q && W % 32 != 0 ? MOE_ERR_SHAPE : MOE_OK;
  }
  if (T > 0 && !a->rstd) return MOE_ERR_NULL;
  if ((uintptr_t)a->dweight % 2) return MOE_ERR_SHAPE;
  MOE_TRY(check_matrix(a->dy, T, W, 1, false));
  MOE_TRY(check_matrix(a->h, T, W, 1, false));
  MOE_TRY(check_matrix(a->dh, T, W, 1, true));
  MOE_TRY(check_matrix(a->dx, T, W, 1, true));
  return check_matrix(a->dresidual, T, W, 1, true);
}

static NormArgs norm_args(const moe_rms_norm_args *a) {
  NormArgs n = {};
  n.x = (const uint16_t *)a->x.p, n.ld_x = a->x.ld;
  n.res = (const uint16_t *)a->residual.p, n.ld_res = a->residual.ld;
  n.h = (uint16_t *)a->h.p, n.ld_h = a->h.ld;
  n.y = (uint16_t *)a->y.p, n.ld_y = a->y.ld;
  n.dy = (const uint16_t *)a->dy.p, n.ld_dy = a->dy.ld;
  n.dh = (const uint16_t *)a->dh.p, n.ld_dh = a->dh.ld;
  n.dx = (uint16_t *)a->dx.p, n.ld_dx = a->dx.ld;
  n.dres = (uint16_t *)a->dresidual.p, n.ld_dres = a->dresidual.ld;
  n.weight = (const uint16_t *)a->weight;
  n.rstd = a->rstd, n.q = a->q, n.q_scale = a->q_scale;
  n.tokens = a->tokens, n.width = a->width, n.eps = a->eps;
  n.drop = drop_of(a->drop);
  return n;
}

// Blocks that go down `tokens` rows, ROWS of them at a time.
static int64_t row_blocks(int64_t tokens, int rows, int64_t most) {
  const int64_t n = (tokens + rows - 1) / rows;
  return n < most ? n : most;
}

// f with the least shape that holds the width.
template <class F>
static int with_shape(int width, F &&f) {
  if (width <= 128) return f(RowShape<16, 1>());
  if (width <= 256) return f(RowShape<16, 2>());
  if (width <= 512) return f(RowShape<64, 1>());
  if (width <= 1024) return f(RowShape<64, 2>());
  if (width <= 2048) return f(RowShape<64, 4>());
  if (width <= 4096) return f(RowShape<256, 2>());
  if (width <= 8192) return f(RowShape<256, 4>());
  if (width <= 16384) return f(RowShape<512, 4>());
  return f(RowShape<512, 8>());
}

template <class D>
static int run_norm(const moe_rms_norm_args *a, hipStream_t st) {
  const NormArgs n = norm_args(a);
  return with_shape(a->width, [&](auto shape) {
    typedef decltype(shape) S;
    const int64_t blocks = row_blocks(a->tokens, S::ROWS, 256 * (2048 / S::THREADS));
    norm_kernel<D, S><<<(uint32_t)blocks, S::THREADS, 0, st>>>(n);
    return hip_status();
  });
}

// Blocks of the backward pass: each has a row of partial sums of dweight.
template <class S>
static int64_t backward_blocks(int64_t tokens) {
  return row_blocks(tokens, S::ROWS, S::ROWS > 1 ? 1024 : S::THREADS == 256 ? 512 : 256);
}
template <class D>
static int run_norm_backward_of(const moe_rms_norm_args *a, Arena &ws, hipStream_t st) {
  NormArgs n = norm_args(a);
  return with_shape(a->width, [&](auto shape) {
    typedef decltype(shape) S;
    const int64_t blocks = backward_blocks<S>(a->tokens);
    if (a->dweight && blocks > 0)
      n.part = reinterpret_cast<float *>(ws.take((size_t)blocks * a->width * sizeof(float)));
    if (ws.dry) return (int)MOE_OK;
    if (blocks > 0 && (a->dweight || a->dx.p || a->dresidual.p)) {
      norm_backward_kernel<D, S><<<(uint32_t)blocks, S::THREADS, 0, st>>>(n);
      MOE_TRY(hip_status());
    }
    if (a->dweight) {
      norm_weight_kernel<D><<<(a->width + 63) / 64, dim3(64, NORM_SUM_ROWS), 0, st>>>(
          n.part, (int)blocks, a->width, (uint16_t *)a->dweight);
      return hip_status();
    }
    return (int)MOE_OK;
  });
}
static int run_norm_backward(const moe_rms_norm_args *a, Arena &ws, hipStream_t st) {
  return a->dtype == MOE_BF16 ? run_norm_backward_of<Bf16>(a, ws, st)
                              : run_norm_backward_of<F16>(a, ws, st);
}

static int check_dropout(const moe_dropout_args *a) {
  if (!a) return MOE_ERR_NULL;
  if (a->dtype != MOE_BF16 && a->dtype != MOE_F16) return MOE_ERR_UNSUPPORTED;
  if (a->tokens < 0 || a->width <= 0) return MOE_ERR_SHAPE;
  if (a->width > MOE_FFN_MAX_WIDTH || a->tokens > MAX_ROWS) return MOE_ERR_UNSUPPORTED;
  MOE_TRY(check_drop(a->drop));
  MOE_TRY(check_matrix(a->x, a->tokens, a->width, 1, false));
  MOE_TRY(check_matrix(a->residual, a->tokens, a->width, 1, true));
  return check_matrix(a->out, a->tokens, a->width, 1, false);
}

}  // namespace moe_block

extern "C" {

int moe_rms_norm(const moe_rms_norm_args *a, void *stream) {
  using namespace moe_block;
  MOE_TRY(check_norm(a, false));
  if (a->tokens == 0) return MOE_OK;
  return a->dtype == MOE_BF16 ? run_norm<Bf16>(a, (hipStream_t)stream)
                              : run_norm<F16>(a, (hipStream_t)stream);
}
int64_t moe_rms_norm_backward_workspace_bytes(const moe_rms_norm_args *a, int32_t backward) {
  using namespace moe_block;
  return backward ? sized(a, check_norm(a, true), run_norm_backward) : 0;
}
int moe_rms_norm_backward(const moe_rms_norm_args *a, void *workspace, size_t workspace_bytes,
                          void *stream) {
  using namespace moe_block;
  return checked_run(a, check_norm(a, true), run_norm_backward, workspace, workspace_bytes, stream);
}

int moe_dropout(const moe_dropout_args *a, void *stream) {
  using namespace moe_block;
  MOE_TRY(check_dropout(a));
  if (a->tokens == 0) return MOE_OK;
  DropoutArgs d = {};
  d.x = (const uint16_t *)a->x.p, d.ld_x = a->x.ld;
  d.res = (const uint16_t *)a->residual.p, d.ld_res = a->residual.ld;
  d.out = (uint16_t *)a->out.p, d.ld_out = a->out.ld;
  d.tokens = a->tokens, d.width = a->width, d.drop = drop_of(a->drop);
  const int chunks = (a->width + 7) / 8;
  int lanes = 1;  // of a row in a block
  while (lanes < chunks && lanes < 256) lanes *= 2;
  const int rows = 256 / lanes, across = (chunks + lanes - 1) / lanes;
  // some 16 blocks for each compute unit
  const int64_t most = (4096 + across - 1) / across;
  const dim3 grid(across, (uint32_t)row_blocks(a->tokens, rows, most));
  const auto kernel = a->dtype == MOE_BF16 ? dropout_kernel<Bf16> : dropout_kernel<F16>;
  kernel<<<grid, dim3(lanes, rows), 0, (hipStream_t)stream>>>(d);
  return hip_status();
}

int moe_mxfp8_values(const uint8_t *q, const uint8_t *q_scale, int64_t count, int32_t dtype,
                     void *values, void *stream) {
  using namespace moe_block;
  if (dtype != MOE_BF16 && dtype != MOE_F16) return MOE_ERR_UNSUPPORTED;
  if (count < 0 || count % 32 != 0) return MOE_ERR_SHAPE;
  if (count == 0) return MOE_OK;
  if (!q || !q_scale || !values) return MOE_ERR_NULL;
  if ((uintptr_t)values % 2) return MOE_ERR_SHAPE;
  if (count / 8 > MAX_ROWS * (MOE_FFN_MAX_WIDTH / 8)) return MOE_ERR_UNSUPPORTED;
  const int64_t blocks = row_blocks(count / 8, 256, 4096);
  const auto kernel = dtype == MOE_BF16 ? mx_values_kernel<Bf16> : mx_values_kernel<F16>;
  kernel<<<(uint32_t)blocks, 256, 0, (hipStream_t)stream>>>(q, q_scale, count / 8,
                                                           (uint16_t *)values);
  return hip_status();
}

}  // extern "C"
