// adapters.hip - the C entry points of the product with the low-rank adapters of
// many requests beside it.
#include "adapter_rows.hpp"
#include "ffn_host.hpp"

namespace moe_adapter {

static int check(const moe_adapter_linear_args *a, bool backward) {
  if (!a) return MOE_ERR_NULL;
  if (a->dtype != MOE_BF16 && a->dtype != MOE_F16) return MOE_ERR_UNSUPPORTED;
  if (a->tokens < 0 || a->in <= 0 || a->out <= 0 || a->rank <= 0 || a->adapters <= 0 ||
      a->reserved != 0)
    return MOE_ERR_SHAPE;
  if (a->in > MOE_FFN_MAX_WIDTH || a->out > MOE_FFN_MAX_WIDTH || a->tokens > MAX_ROWS ||
      a->rank > MOE_ADAPTER_MAX_RANK || a->adapters > MOE_ADAPTER_MAX)
    return MOE_ERR_UNSUPPORTED;
  const int64_t T = a->tokens;
  const int I = a->in, O = a->out, R = a->rank, n = a->adapters;
  const bool u = !backward || a->dx.p || a->da.p;  // whether B (or A and B) is read
  MOE_TRY(check_matrix(a->x, T, I, 1, backward && !a->da.p));
  MOE_TRY(check_matrix(a->w, O, I, 1, backward && !a->dx.p));
  MOE_TRY(check_matrix(a->a, R, I, n, backward && !a->dx.p));
  MOE_TRY(check_matrix(a->b, O, R, n, !u));
  if (T > 0 && !a->ids) return MOE_ERR_NULL;
  if ((uintptr_t)a->ids % 4 || (uintptr_t)a->scale % 4 || (uintptr_t)a->s % 4) return MOE_ERR_SHAPE;
  if (!backward) {
    MOE_TRY(check_matrix(a->bias, 1, O, 1, true));
    MOE_TRY(check_matrix(a->residual, T, O, 1, true));
    return check_matrix(a->y, T, O, 1, false);
  }
  if (T > 0 && a->db.p && !a->s) return MOE_ERR_NULL;
  MOE_TRY(check_matrix(a->dy, T, O, 1, false));
  MOE_TRY(check_matrix(a->dx, T, I, 1, true));
  MOE_TRY(check_matrix(a->da, R, I, n, true));
  return check_matrix(a->db, O, R, n, true);
}

template <class D, int MT, int RB, int WAVES>
static int shrink_as(const ShrinkArgs &g, int turns, hipStream_t st) {
  const dim3 grid((uint32_t)((g.M + 16 * MT - 1) / (16 * MT)), (uint32_t)turns);
  shrink_kernel<D, MT, RB, WAVES><<<grid, 64 * WAVES, 0, st>>>(g);
  return hip_status();
}
// Few rows: 16 a block, and blocks of their own for the adapters among them, of which
// a decode batch has up to 16. More: 32, so that A is read half as often.
template <class D>
static int shrink_of(const ShrinkArgs &g, hipStream_t st) {
  const int distinct = g.n < 16 ? g.n : 16;
  const int turns = g.M <= 1024 ? distinct : g.M <= 4096 ? (distinct < 4 ? distinct : 4) : 1;
  const int rb = (g.rank + 15) / 16;
  if (g.M <= 4096) {
    if (rb == 1) return shrink_as<D, 1, 1, 16>(g, turns, st);
    if (rb == 2) return shrink_as<D, 1, 2, 16>(g, turns, st);
    if (rb <= 4) return shrink_as<D, 1, 4, 8>(g, turns, st);
    return shrink_as<D, 1, 8, 8>(g, turns, st);
  }
  if (rb == 1) return shrink_as<D, 2, 1, 8>(g, 1, st);
  if (rb == 2) return shrink_as<D, 2, 2, 8>(g, 1, st);
  if (rb <= 4) return shrink_as<D, 2, 4, 8>(g, 1, st);
  return shrink_as<D, 1, 8, 8>(g, 1, st);
}
static int shrink(int dtype, const ShrinkArgs &g, hipStream_t st) {
  return dtype == MOE_BF16 ? shrink_of<Bf16>(g, st) : shrink_of<F16>(g, st);
}

static int run_forward(const moe_adapter_linear_args *a, Arena &ws, hipStream_t st) {
  const int64_t T = a->tokens;
  const int I = a->in, O = a->out;
  int status = MOE_OK;
  if (T == 0) return MOE_OK;
  const moe_expert_rows dense = {};
  const Plan plan = row_plan(dense, true, T, O, I);
  float *s = a->s ? a->s : reinterpret_cast<float *>(ws.take((size_t)T * a->rank * sizeof(float)));
  const Operand x = operand(a->x, T, I, 1, ws, st, &status);
  const Operand w = operand(a->w, O, I, 1, ws, st, &status);
  if (status != MOE_OK) return status;
  if (!ws.dry) {
    ShrinkArgs k = {};
    k.x = (const uint16_t *)a->x.p, k.ldx = a->x.ld;
    k.a = (const uint16_t *)a->a.p, k.lda = a->a.ld, k.stride = a->a.stride;
    k.ids = a->ids, k.scale = a->scale, k.s = s;
    k.M = (int)T, k.K = I, k.rank = a->rank, k.n = a->adapters;
    MOE_TRY(shrink(a->dtype, k, st));
  }
  GemmArgs g = {};
  g.segs = 1;
  g.a = x.p, g.lda = x.ld, g.a_rows = T;
  g.b0 = w.p, g.ldb0 = w.ld;
  g.c0 = (uint16_t *)a->y.p, g.ldc0 = a->y.ld;
  g.bias = (const uint16_t *)a->bias.p;
  g.res = (const uint16_t *)a->residual.p, g.ldr = a->residual.ld;
  g.M = (int)T, g.N = O, g.K = I, g.act = MOE_ACT_NONE;
  g.low = {a->ids, s, (const uint16_t *)a->b.p, a->b.ld, a->b.stride, a->adapters, a->rank};
  return run_product(a->dtype, LINEAR, plan, g, O, 0, ws, st);
}

// Tokens of a block of the gradients: some 512 blocks over both sides, and no fewer
// than 256 tokens, below which the partial sums outweigh what they are made from.
static int grad_chunk(int64_t tokens, int tiles) {
  const int64_t chunks = (512 + tiles - 1) / tiles;
  const int64_t each = ((tokens + chunks - 1) / chunks + GRAD_K - 1) / GRAD_K * GRAD_K;
  return (int)(each < 256 ? 256 : each);
}

template <class D>
static int grads_of(const GradArgs &g, dim3 grid, hipStream_t st) {
  const int rb = (g.rank + 15) / 16;
  const auto kernel = rb == 1   ? grad_kernel<D, 1>
                      : rb == 2 ? grad_kernel<D, 2>
                      : rb <= 4 ? grad_kernel<D, 4>
                                : grad_kernel<D, 8>;
  kernel<<<grid, 64 * GRAD_WAVES, 0, st>>>(g);
  return hip_status();
}

static int run_backward(const moe_adapter_linear_args *a, Arena &ws, hipStream_t st) {
  const int64_t T = a->tokens;
  const int I = a->in, O = a->out, R = a->rank, n = a->adapters;
  const int R8 = round8(R), O8 = round8(O), I4 = (I + 3) & ~3, O4 = (O + 3) & ~3;
  const bool dx = a->dx.p && T > 0, grads = a->da.p || a->db.p, needs_u = T > 0 && (a->dx.p || a->da.p);
  const bool bf = a->dtype == MOE_BF16;
  int status = MOE_OK;
  if (!dx && !grads) return MOE_OK;
  int32_t *offsets = reinterpret_cast<int32_t *>(ws.take((size_t)(n + 1) * 4));
  int32_t *perm = reinterpret_cast<int32_t *>(ws.take((size_t)T * 4));
  uint16_t *at = dx ? ws.take((size_t)n * I * R8 * 2) : nullptr;
  uint16_t *bt = needs_u ? ws.take((size_t)n * R * O8 * 2) : nullptr;
  float *u = needs_u ? reinterpret_cast<float *>(ws.take((size_t)T * R * 4)) : nullptr;
  if (!ws.dry) {
    sort_ids_kernel<<<n, SORT_THREADS, 0, st>>>(a->ids, (int)T, n, offsets, perm);
    MOE_TRY(hip_status());
  }
  if (needs_u && !ws.dry) {
    const TransposeArgs ta = {(const uint16_t *)a->a.p, a->a.ld, a->a.stride, at, R, I, R8};
    const TransposeArgs tb = {(const uint16_t *)a->b.p, a->b.ld, a->b.stride, bt, R, O, O8};
    const int a_blocks = dx ? (I + 255) / 256 : 0;
    transpose_kernel<<<dim3(a_blocks + (O + 255) / 256, n), 256, 0, st>>>(ta, tb, offsets, n, a_blocks);
    MOE_TRY(hip_status());
    ShrinkArgs k = {};
    k.x = (const uint16_t *)a->dy.p, k.ldx = a->dy.ld;
    k.a = bt, k.lda = O8, k.stride = (int64_t)R * O8;
    k.ids = a->ids, k.scale = a->scale, k.s = u;
    k.M = (int)T, k.K = O, k.rank = R, k.n = n;
    MOE_TRY(shrink(a->dtype, k, st));
  }
  if (dx) {
    const moe_expert_rows dense = {};
    const Operand dy = operand(a->dy, T, O, 1, ws, st, &status);
    const Operand w = operand(a->w, O, I, 1, ws, st, &status);
    if (status != MOE_OK) return status;
    GemmArgs g = {};
    g.segs = 1;
    g.a = dy.p, g.lda = dy.ld, g.a_rows = T;
    g.b0 = w.p, g.ldb0 = w.ld;
    g.c0 = (uint16_t *)a->dx.p, g.ldc0 = a->dx.ld;
    g.M = (int)T, g.N = I, g.K = O;
    g.low = {a->ids, u, at, R8, (int64_t)I * R8, n, R};
    MOE_TRY(run_product(a->dtype, DGRAD, row_plan(dense, false, T, I, O), g, I, 0, ws, st));
  }
  if (!grads) return MOE_OK;
  const int a_tiles = a->da.p ? (I + GRAD_COLS - 1) / GRAD_COLS : 0;
  const int b_tiles = a->db.p ? (O + GRAD_COLS - 1) / GRAD_COLS : 0;
  const int chunk = grad_chunk(T, a_tiles + b_tiles);
  const int64_t chunks = (T + chunk - 1) / chunk, slots = chunks + n - 1;
  GradArgs g = {};
  g.side[0] = {(const uint16_t *)a->x.p, a->x.ld, u, nullptr, I, I4, a_tiles};
  g.side[1] = {(const uint16_t *)a->dy.p, a->dy.ld, a->s, nullptr, O, O4, b_tiles};
  if (a->da.p) g.side[0].part = reinterpret_cast<float *>(ws.take((size_t)slots * R * I4 * 4));
  if (a->db.p) g.side[1].part = reinterpret_cast<float *>(ws.take((size_t)slots * R * O4 * 4));
  if (ws.dry) return MOE_OK;
  g.offsets = offsets, g.perm = perm, g.rank = R, g.n = n, g.chunk = chunk;
  if (T > 0) {
    const dim3 grid(a_tiles + b_tiles, (uint32_t)chunks);
    MOE_TRY(bf ? grads_of<Bf16>(g, grid, st) : grads_of<F16>(g, grid, st));
  }
  const int64_t a_runs = a->da.p ? (int64_t)R * ((I + 7) / 8) : 0;
  const int64_t b_runs = a->db.p ? (int64_t)((R + 7) / 8) * O : 0;
  const JoinSide da = {g.side[0].part, (uint16_t *)a->da.p, a->da.ld, a->da.stride, I, I4, (int)((a_runs + 255) / 256)};
  const JoinSide db = {g.side[1].part, (uint16_t *)a->db.p, a->db.ld, a->db.stride, O, O4, (int)((b_runs + 255) / 256)};
  const auto kernel = bf ? grad_join_kernel<Bf16> : grad_join_kernel<F16>;
  kernel<<<dim3(da.blocks + db.blocks, n), 256, 0, st>>>(da, db, offsets, R, chunk);
  return hip_status();
}

}  // namespace moe_adapter

extern "C" {

int64_t moe_adapter_linear_workspace_bytes(const moe_adapter_linear_args *a, int32_t backward) {
  using namespace moe_adapter;
  return sized(a, check(a, backward != 0), backward ? run_backward : run_forward);
}
int moe_adapter_linear(const moe_adapter_linear_args *a, void *workspace, size_t workspace_bytes,
                       void *stream) {
  using namespace moe_adapter;
  return checked_run(a, check(a, false), run_forward, workspace, workspace_bytes, stream);
}
int moe_adapter_linear_backward(const moe_adapter_linear_args *a, void *workspace,
                                size_t workspace_bytes, void *stream) {
  using namespace moe_adapter;
  return checked_run(a, check(a, true), run_backward, workspace, workspace_bytes, stream);
}

}  // extern "C"
