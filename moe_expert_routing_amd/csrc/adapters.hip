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

// Whether rows can be staged: their 16-byte pieces are aligned.
static bool staged(const void *p, int64_t ld, int64_t stride, int cols) {
  return ((uintptr_t)p & 15) == 0 && ((ld | stride | cols) & 7) == 0;
}

template <class D, int MT, int RB, int WAVES, int NS, int NS2>
static int shrink_as(ShrinkArgs g, int turns, hipStream_t st) {
  g.turns = turns;
  const int64_t blocks = (int64_t)((g.M + 16 * MT - 1) / (16 * MT)) * turns;
  const bool whole = staged(g.x, g.ldx, 0, g.K) && staged(g.a, g.lda, g.stride, g.K);
  const auto kernel =
      whole ? shrink_kernel<D, MT, RB, WAVES, NS, NS2, true> : shrink_kernel<D, MT, RB, WAVES, NS, NS2, false>;
  return in_parts(blocks, 64 * WAVES, [&](int64_t first, uint32_t n) {
    g.block0 = first;
    kernel<<<n, 64 * WAVES, 0, st>>>(g);
    return hip_status();
  });
}
// Few rows: 16 a block, of which a decode batch has up to 16 adapters. More: 32, so that
// A is read half as often, once that many blocks fill the card. (With the product, us, by 32
// and by 16: 2048 rows of 7168, rank 32, 91 and 81; 2048 rows of 4096 from 300 requests 122
// and 105; 8192 rows of 7168, then with half the waves, 218 and 222.) Up to 4096 rows, too, the
// rounds over a row's adapters are shared, by as many blocks as there is room for.
template <class D>
static int shrink_of(const ShrinkArgs &g, hipStream_t st) {
  const int distinct = g.n < 16 ? g.n : 16;
  const int rb = (g.rank + 15) / 16;
  if (g.M <= 1024) {
    if (rb == 1) return shrink_as<D, 1, 1, 8, 4, 0>(g, distinct, st);
    if (rb == 2) return shrink_as<D, 1, 2, 8, 3, 0>(g, distinct, st);
    if (rb <= 4) return shrink_as<D, 1, 4, 4, 3, 0>(g, distinct, st);
    return shrink_as<D, 1, 8, 4, 2, 0>(g, distinct, st);
  }
  if (g.M <= 4096) {
    const int turns = distinct < 4096 / g.M ? distinct : 4096 / g.M;
    if (rb == 1) return shrink_as<D, 1, 1, 8, 4, 3>(g, turns, st);
    if (rb == 2) return shrink_as<D, 1, 2, 4, 4, 3>(g, turns, st);
    if (rb <= 4) return shrink_as<D, 1, 4, 4, 3, 2>(g, turns, st);
  } else {
    if (rb == 1) return shrink_as<D, 2, 1, 8, 3, 2>(g, 1, st);
    if (rb == 2) return shrink_as<D, 2, 2, 4, 4, 3>(g, 1, st);
    if (rb <= 4) return shrink_as<D, 2, 4, 4, 3, 2>(g, 1, st);
  }
  return shrink_as<D, 1, 8, 4, 2, 0>(g, distinct < 2 ? 1 : 2, st);
}
static int shrink(int dtype, const ShrinkArgs &g, hipStream_t st) {
  return dtype == MOE_BF16 ? shrink_of<Bf16>(g, st) : shrink_of<F16>(g, st);
}

template <class D, int MT, int RB, int NS>
static int few_as(FewArgs g, hipStream_t st) {
  g.w_tiles = (g.N + 16 * RB - 1) / (16 * RB);
  g.rank_tiles = (g.rank + (RB < 2 ? 15 : 31)) / (RB < 2 ? 16 : 32);
  const int group = g.M < FEW_GROUP ? g.M : FEW_GROUP, slots = g.n < group ? g.n : group;
  const dim3 grid(g.w_tiles + slots * g.rank_tiles, g.splits, (g.M + FEW_GROUP - 1) / FEW_GROUP);
  const bool whole = staged(g.x, g.ldx, 0, g.K) && staged(g.w, g.ldw, 0, g.K) &&
                     staged(g.a, g.lda, g.a_stride, g.K);
  const auto kernel =
      whole ? few_stream_kernel<D, MT, RB, NS, true> : few_stream_kernel<D, MT, RB, NS, false>;
  kernel<<<grid, 64 * FEW_WAVES, 0, st>>>(g);
  MOE_TRY(hip_status());
  few_finish_kernel<D><<<dim3((g.N + 255) / 256, g.M), 256, 0, st>>>(g);
  return hip_status();
}
template <class D>
static int few_of(const FewArgs &g, hipStream_t st) {
  if (g.M <= 16) return few_as<D, 1, 1, 4>(g, st);
  if (g.M <= 32) return few_as<D, 2, 2, 3>(g, st);
  return few_as<D, 4, 4, 2>(g, st);
}
// Whether y goes by these kernels: up to 32 tokens, up to 64 but where many columns come of
// a short way, and with a long way to few columns up to 128. (Each token with one of 64 adapters
// of rank 16, these kernels and the tiles, us: 32 tokens 7168 -> 2048 19 and 25, 2048 -> 7168
// 17 and 20; 64 tokens 23 and 26, 24 and 20, 4096 -> 4096 28 and 25, 7168 -> 7168 40 and 54, 7168
// -> 512 19 and 25; 100 tokens 32 and 29, 36 and 24, 41 and 26, 61 and 58, 24 and 25.)
static bool is_few(int64_t T, int64_t I, int64_t O) {
  return T <= 32 || (T <= 64 && (I > 4096 || O < 4096)) || (T <= 128 && I >= 8 * O);
}
static int run_few(const moe_adapter_linear_args *a, Arena &ws, hipStream_t st) {
  FewArgs g = {};
  g.M = (int)a->tokens, g.N = a->out, g.K = a->in, g.rank = a->rank, g.n = a->adapters;
  // some 2048 waves, of at least 128 k
  const int blocks = (g.K + 63) / 64, tile = g.M <= 16 ? 16 : g.M <= 32 ? 32 : 64;
  const int tiles = (g.N + tile - 1) / tile;
  int splits = 512 / tiles;
  splits = splits < 1 ? 1 : splits > 8 ? 8 : splits;
  g.per = (blocks + splits * FEW_WAVES - 1) / (splits * FEW_WAVES);
  if (g.per < 2) g.per = 2;  // blocks of 64
  g.splits = (blocks + g.per * FEW_WAVES - 1) / (g.per * FEW_WAVES);  // none of them empty
  g.per *= 64;
  g.part_y = reinterpret_cast<float *>(ws.take((size_t)g.splits * g.M * g.N * sizeof(float)));
  g.part_s = reinterpret_cast<float *>(ws.take((size_t)g.splits * g.M * g.rank * sizeof(float)));
  if (ws.dry) return MOE_OK;
  g.x = (const uint16_t *)a->x.p, g.ldx = a->x.ld;
  g.w = (const uint16_t *)a->w.p, g.ldw = a->w.ld;
  g.a = (const uint16_t *)a->a.p, g.lda = a->a.ld, g.a_stride = a->a.stride;
  g.b = (const uint16_t *)a->b.p, g.ldb = a->b.ld, g.b_stride = a->b.stride;
  g.bias = (const uint16_t *)a->bias.p;
  g.res = (const uint16_t *)a->residual.p, g.ldr = a->residual.ld;
  g.ids = a->ids, g.scale = a->scale, g.s = a->s;
  g.y = (uint16_t *)a->y.p, g.ldy = a->y.ld;
  return a->dtype == MOE_BF16 ? few_of<Bf16>(g, st) : few_of<F16>(g, st);
}

// Plan of the product with its low-rank term. Of few rows the epilogue is the longer
// part, one adapter after the other for every 16 of them, so that it takes the small tiles,
// and ranges of k where these are few (by the dense product's plan and this one, us: 100 tokens
// 2048 -> 7168 26 and 24, 160 tokens 7168 -> 2048 46 and 30, 512 tokens 7168 -> 512 44 and 39; past
// the limits, 255 tokens 2048 -> 7168 33 and 37, 192 tokens 7168 -> 7168 75 and 91).
static Plan low_plan(int64_t T, int64_t I, int64_t O) {
  const int64_t tiles = (T + 31) / 32 * ((O + 63) / 64);
  if (T <= 512 && tiles < 256 && I >= 4096) return {TILE_32, 4};
  if (T <= 192 && I < 4096) return {TILE_32, 1};
  return row_plan({}, true, T, O, I);
}

static int run_forward(const moe_adapter_linear_args *a, Arena &ws, hipStream_t st) {
  const int64_t T = a->tokens;
  const int I = a->in, O = a->out;
  int status = MOE_OK;
  if (T == 0) return MOE_OK;
  if (is_few(T, I, O)) return run_few(a, ws, st);
  const Plan plan = low_plan(T, I, O);
  float *s = a->s ? a->s : reinterpret_cast<float *>(ws.take((size_t)T * a->rank * sizeof(float)));
  const Operand x = operand(a->x, T, I, 1, ws, st, &status);
  const Operand w = operand(a->w, O, I, 1, ws, st, &status);
  if (status != MOE_OK) return status;
  if (!ws.dry) {
    ShrinkArgs k = {};
    k.x = (const uint16_t *)a->x.p, k.ldx = a->x.ld;
    k.a = (const uint16_t *)a->a.p, k.lda = a->a.ld, k.stride = a->a.stride;
    k.ids = a->ids, k.scale = a->scale, k.s = s;
    k.M = (int)T, k.K = I, k.rank = k.lds = a->rank, k.n = a->adapters;
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
  g.low = {a->ids, s, (const uint16_t *)a->b.p, a->b.ld, a->b.stride, a->adapters, a->rank, a->rank};
  return run_product(a->dtype, LINEAR, plan, g, O, 0, ws, st);
}

// Tokens of a block of the gradients: some 512 blocks over both sides, and no fewer
// than 4 for each of the rank, where the partial sums are as many bytes as what they are
// made from.
static int grad_chunk(int64_t tokens, int tiles, int rank) {
  const int64_t chunks = (512 + tiles - 1) / tiles;
  int64_t each = (tokens + chunks - 1) / chunks;
  each = each > 4 * rank ? each : 4 * rank;
  return (int)((each + GRAD_K - 1) / GRAD_K * GRAD_K);
}

template <class D, bool WHOLE>
static int grads_of(const GradArgs &g, dim3 grid, hipStream_t st) {
  const int rb = (g.rank + 15) / 16;
  const auto kernel = rb == 1   ? grad_kernel<D, 1, 4, WHOLE>
                      : rb == 2 ? grad_kernel<D, 2, 3, WHOLE>
                      : rb <= 4 ? grad_kernel<D, 4, 3, WHOLE>
                                : grad_kernel<D, 8, 4, WHOLE>;
  kernel<<<grid, 64 * GRAD_WAVES, 0, st>>>(g);
  return hip_status();
}

static int run_backward(const moe_adapter_linear_args *a, Arena &ws, hipStream_t st) {
  const int64_t T = a->tokens;
  const int I = a->in, O = a->out, R = a->rank, n = a->adapters;
  const int R4 = (R + 3) & ~3, R8 = round8(R), O8 = round8(O), I4 = (I + 3) & ~3, O4 = (O + 3) & ~3;
  const bool dx = a->dx.p && T > 0, da = a->da.p, db = a->db.p, needs_u = T > 0 && (a->dx.p || da);
  const bool bf = a->dtype == MOE_BF16;
  int status = MOE_OK;
  if (!dx && !da && !db) return MOE_OK;
  int32_t *offsets = reinterpret_cast<int32_t *>(ws.take((size_t)(n + 1) * 4));
  int32_t *perm = reinterpret_cast<int32_t *>(ws.take((size_t)T * 4));
  float *zeros = reinterpret_cast<float *>(ws.take(16));
  // copies of A and B: of every adapter, or of the tokens' where these are fewer
  const bool by_token = needs_u && n > T;
  const int places = by_token ? (int)T : n;
  uint16_t *at = dx ? ws.take((size_t)places * I * R8 * 2) : nullptr;
  uint16_t *bt = needs_u ? ws.take((size_t)places * R * O8 * 2) : nullptr;
  int32_t *own = by_token ? reinterpret_cast<int32_t *>(ws.take((size_t)T * 4)) : nullptr;
  float *own_scale = by_token && a->scale ? reinterpret_cast<float *>(ws.take((size_t)T * 4)) : nullptr;
  float *u = needs_u ? reinterpret_cast<float *>(ws.take((size_t)T * R4 * 4)) : nullptr;
  // s where its rows are whole 16 bytes, else a copy of it whose rows are
  const bool copy_s = db && T > 0 && (R != R4 || (uintptr_t)a->s % 16 != 0);
  float *s4 = copy_s ? reinterpret_cast<float *>(ws.take((size_t)T * R4 * 4)) : nullptr;
  // dy is an operand of dx and of dB, x of dA
  Operand dy = {}, x = {}, w = {};
  if (dx || db) dy = operand(a->dy, T, O, 1, ws, st, &status);
  if (da) x = operand(a->x, T, I, 1, ws, st, &status);
  if (dx) w = operand(a->w, O, I, 1, ws, st, &status);
  if (status != MOE_OK) return status;
  if (!ws.dry) {
    PrepArgs p = {};
    p.ids = a->ids, p.offsets = offsets, p.perm = perm, p.T = (int)T, p.n = n;
    p.a = (const uint16_t *)a->a.p, p.lda = a->a.ld, p.a_stride = a->a.stride;
    p.b = (const uint16_t *)a->b.p, p.ldb = a->b.ld, p.b_stride = a->b.stride;
    p.at = at, p.bt = bt, p.in = I, p.out = O, p.rank = R, p.rank4 = R4, p.rank8 = R8, p.out8 = O8;
    p.s = a->s, p.s4 = s4, p.zeros = zeros;
    p.scale = a->scale, p.own = own, p.own_scale = own_scale;
    const int64_t items = (int64_t)((dx ? I : 0) + (needs_u ? O : 0)) * (R8 / 8);
    p.copy_block = n + places * ((items + PREP_THREADS - 1) / PREP_THREADS);
    const int64_t copies = copy_s ? (T * R4 + PREP_THREADS - 1) / PREP_THREADS : 0;
    MOE_TRY(in_parts(p.copy_block + copies, PREP_THREADS, [&](int64_t first, uint32_t blocks) {
      p.block0 = first;
      if (own)
        prep_kernel<true><<<blocks, PREP_THREADS, 0, st>>>(p);
      else
        prep_kernel<false><<<blocks, PREP_THREADS, 0, st>>>(p);
      return hip_status();
    }));
  }
  if (needs_u && !ws.dry) {
    ShrinkArgs k = {};
    k.x = (const uint16_t *)a->dy.p, k.ldx = a->dy.ld;
    k.a = bt, k.lda = O8, k.stride = (int64_t)R * O8;
    k.ids = own ? own : a->ids, k.scale = own_scale ? own_scale : a->scale, k.s = u;
    k.M = (int)T, k.K = O, k.rank = R, k.lds = R4, k.n = places;
    MOE_TRY(shrink(a->dtype, k, st));
  }
  if (dx) {
    const moe_expert_rows dense = {};
    GemmArgs g = {};
    g.segs = 1;
    g.a = dy.p, g.lda = dy.ld, g.a_rows = T;
    g.b0 = w.p, g.ldb0 = w.ld;
    g.c0 = (uint16_t *)a->dx.p, g.ldc0 = a->dx.ld;
    g.M = (int)T, g.N = I, g.K = O;
    g.low = {own ? own : a->ids, u, at, R8, (int64_t)I * R8, places, R, R4};
    MOE_TRY(run_product(a->dtype, DGRAD, row_plan(dense, false, T, I, O), g, I, 0, ws, st));
  }
  if (!da && !db) return MOE_OK;
  const int a_tiles = da ? (I + GRAD_COLS - 1) / GRAD_COLS : 0;
  const int b_tiles = db ? (O + GRAD_COLS - 1) / GRAD_COLS : 0;
  const int chunk = grad_chunk(T, a_tiles + b_tiles, R);
  const int64_t chunks = (T + chunk - 1) / chunk;
  const bool whole = n - 1 > chunks;
  const int64_t slots = !whole ? chunks + n - 1 : chunks > 1 ? 2 * chunks : 0;
  GradArgs g = {};
  g.side[0] = {x.p, x.ld, u, nullptr, (uint16_t *)a->da.p, a->da.ld, a->da.stride, I, I4, a_tiles};
  g.side[1] = {dy.p, dy.ld, s4 ? s4 : a->s, nullptr, (uint16_t *)a->db.p, a->db.ld, a->db.stride, O, O4, b_tiles};
  if (da) g.side[0].part = reinterpret_cast<float *>(ws.take((size_t)slots * R * I4 * 4));
  if (db) g.side[1].part = reinterpret_cast<float *>(ws.take((size_t)slots * R * O4 * 4));
  if (ws.dry) return MOE_OK;
  g.offsets = offsets, g.perm = perm, g.zeros = zeros;
  g.rank = R, g.ldv = R4, g.n = n, g.chunk = chunk;
  if (T > 0) {
    const dim3 grid(a_tiles + b_tiles, (uint32_t)chunks);
    MOE_TRY(bf ? (whole ? grads_of<Bf16, true>(g, grid, st) : grads_of<Bf16, false>(g, grid, st))
               : (whole ? grads_of<F16, true>(g, grid, st) : grads_of<F16, false>(g, grid, st)));
  }
  const int64_t a_runs = da ? (int64_t)R * ((I + 7) / 8) : 0;
  const int64_t b_runs = db ? (int64_t)((R + 7) / 8) * O : 0;
  const JoinSide ja = {g.side[0].part, (uint16_t *)a->da.p, a->da.ld, a->da.stride, I, I4, (int)((a_runs + 255) / 256)};
  const JoinSide jb = {g.side[1].part, (uint16_t *)a->db.p, a->db.ld, a->db.stride, O, O4, (int)((b_runs + 255) / 256)};
  const auto kernel = bf ? (whole ? grad_join_kernel<Bf16, true> : grad_join_kernel<Bf16, false>)
                         : (whole ? grad_join_kernel<F16, true> : grad_join_kernel<F16, false>);
  kernel<<<dim3(ja.blocks + jb.blocks, n), 256, 0, st>>>(ja, jb, offsets, R, chunk);
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
