// ffn.hip - the C entry points of the feed-forward operators: checks, padded
// copies where an operand needs one, and the launches.
#include "ffn_host.hpp"
#include "ffn_rows.hpp"

namespace moe_ffn {

static int launch_gemm(int dtype, int mode, int kind, const GemmArgs &g, hipStream_t st) {
  if (g.low.ids)
    return dtype == MOE_BF16 ? launch_low_bf16(mode, kind, g, st) : launch_low_f16(mode, kind, g, st);
  return dtype == MOE_BF16 ? launch_gemm_bf16(mode, kind, g, st) : launch_gemm_f16(mode, kind, g, st);
}

static dim3 row_grid(int64_t rows, int cols8, int z) {
  const int64_t y = (rows + ROW_THREADS - 1) / ROW_THREADS;
  return dim3((uint32_t)((cols8 / 8 + COL_THREADS - 1) / COL_THREADS),
              (uint32_t)(y < 65535 ? y : 65535), (uint32_t)z);
}

static bool is_aligned(const moe_matrix &m, int cols, int mats) {
  return ((uintptr_t)m.p & 15) == 0 && ((m.ld | cols) & 7) == 0 &&
         (mats == 1 || (m.stride & 7) == 0);
}
Operand operand(const moe_matrix &m, int64_t rows, int cols, int mats, Arena &a, hipStream_t st,
                int *status, bool copy) {
  if ((is_aligned(m, cols, mats) && !copy) || rows == 0) return {(const uint16_t *)m.p, m.ld, m.stride};
  const int c8 = round8(cols);
  uint16_t *dst = a.take((size_t)mats * rows * c8 * 2);
  if (!a.dry && *status == MOE_OK) {
    pad_rows_kernel<<<row_grid(rows, c8, mats), dim3(COL_THREADS, ROW_THREADS), 0, st>>>(
        (const uint16_t *)m.p, m.ld, m.stride, rows, cols, dst, c8);
    *status = hip_status();
  }
  return {dst, c8, rows * c8};
}

// Plan of `mats` products of M x N over K: the one with the least estimated time,
// its rounds over the 256 compute units times (64-k stages times a stage's
// time, plus a fixed part). The stage times, in microseconds, are measured
// with one tile on a compute unit, and with two where two fit. What
// the choice does, in us, for 256 / 128 / 64 / 32-row tiles:
//   1024 x 1024 x 2816     60 / 22 / 14 / 14    8192 x 7168 x 2048  265 / 295 / - / -
//   2048 x 2048 x 2048     49 / 21 / 31 / -     64 x 7168 x 2048    - / - / 11 / 8.7
// Where few tiles have a long way through k (may_split), up to 16 ranges of at
// least 6 stages each are summed apart, which costs the partial sums' way through
// memory, a workspace and a launch that joins them: 14 us fixed, so that calls
// bound by the host's side stay as they are. Measured, one range / split: 64 x
// 7168 -> 2048 gated 30 / 19 us, 64 x 7168 -> 1024 18 / 15, dW of 16384 x 1024 ->
// 512 53 / 36; with 12 us instead of 14, 64 x 4096 -> 1024 gated went 12 / 16.
static Plan dense_plan(int64_t mats, int64_t M, int64_t N, int64_t K, bool may_split) {
  static const struct {
    int kind, bm, bn, blocks;
    float one, full, fixed;
  } tiles[] = {{TILE_256, 256, 256, 1, 1.5f, 1.5f, 10.f},
               {TILE_128, 128, 128, 1, 0.46f, 0.46f, 4.f},
               {TILE_64, 64, 64, 2, 0.30f, 0.48f, 2.5f},
               {TILE_32, 32, 64, 2, 0.26f, 0.36f, 2.5f}};
  const int64_t stages = (K + 63) / 64;
  Plan best = {TILE_256, 1};
  float least = 0.f;
  for (int splits = 1; splits == 1 || (may_split && splits <= 16 && stages / splits >= 6);
       splits *= 2) {
    const float join =
        splits == 1 ? 0.f : 14.f + (float)(splits * mats * M * N) * 8.f / 4e6f;  // at 4 TB/s
    for (const auto &t : tiles) {
      const int64_t n = splits * mats * ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
      const int64_t rounds = (n + 256 * t.blocks - 1) / (256 * t.blocks);
      const float stage = n <= 256 ? t.one : t.full;
      const float time =
          (float)rounds * ((float)((stages + splits - 1) / splits) * stage + t.fixed) + join;
      if (least == 0.f || time < least) least = time, best = {t.kind, splits};
    }
  }
  return best;
}
// Rows that an expert with any has on average, by the layout's size: without the
// padding, half a tile for each of them. No more experts have rows than there are
// tiles: 64 experts, 2048 -> 1024 gated, two of them with 2000 rows each padded to 256
// take 34 us forward and 191 back by this estimate, 448 and 1011 by one that takes the
// padding off for all 64. Ten of them with 3 rows each padded to 128, which it takes for
// 64 rows each: 27 and 160, and 27 and 144.
static int64_t expert_rows(const moe_expert_rows &r, int64_t rows) {
  const int64_t tiles = (rows + r.tile_m - 1) / r.tile_m;
  const int64_t with_rows = tiles < r.num_experts ? tiles : r.num_experts;
  return with_rows ? rows / with_rows - r.tile_m / 2 : 0;
}
// Plan of the products whose M is the call's rows. Over experts a tile holds
// rows of one, and its rows go by how many an expert has on average. Where the tile does not divide the layout's alignment a launch
// finds the tiles first (about 5 us), for 64 rows an expert and more. (112 experts
// with about 146 rows padded to 128, 2048 -> 1024 gated: 128 x 256 tiles 252 us, 128 x
// 128 301, 64 x 256 306, 64 x 128 337; with about 277 rows in buffers for 400, 512 ->
// 4096: 256 x 256 tiles 302 us, 128 x 256 343, 512 -> 2048 gated 261 and 289.) A dense
// forward product of up to 16 rows goes by the skinny kernel; dx of as few, whose
// weights are read transposed, by the plan (16-row tiles and the plan: 8 rows of 7168
// from 7168 48 and 26 us, 12 rows of 4096 from 14336 87 and 31).
Plan row_plan(const moe_expert_rows &r, bool forward, int64_t M, int64_t N, int64_t K) {
  if (r.num_experts > 0) {
    const int64_t mean = expert_rows(r, M);
    if (mean >= 320) return {TILE_256, 1};
    if (mean >= 80) return {TILE_128W, 1};
    if (mean >= 40 && (mean >= 64 || r.tile_m % 64 == 0)) return {TILE_64W, 1};
    return {mean >= 20 && r.tile_m % 32 == 0 ? TILE_32 : TILE_16, 1};
  }
  if (forward && M <= 16) return {TILE_16, 1};
  return dense_plan(1, M, N, K, true);
}
static int rows_of_tile(int kind) {
  switch (kind) {
    case TILE_16: return 16;
    case TILE_32: return 32;
    case TILE_64:
    case TILE_64W: return 64;
    case TILE_256: return 256;
  }
  return 128;
}
static Plan weight_plan(const moe_expert_rows &r, int64_t segs, int64_t M, int64_t N,
                        int64_t rows) {
  if (r.num_experts > 0)
    return dense_plan(segs * r.num_experts, M, N, expert_rows(r, rows), false);
  return dense_plan(segs, M, N, rows, true);
}

// Runs a product by its plan, with the partial sums of a split one in the
// workspace. `width`: the partial sums of a row of C. `tile_m`: the alignment of
// the layout, 0 for a dense product.
int run_product(int dtype, int mode, const Plan &plan, GemmArgs &g, int width, int tile_m,
                Arena &ws, hipStream_t st) {
  const int64_t stages = (g.K + 63) / 64;
  const int bm = rows_of_tile(plan.kind);
  if (mode != WGRAD && tile_m % bm != 0) {
    // tiles that follow the experts' rows instead of the layout's alignment
    g.m_tiles = (int)((g.M + bm - 1) / bm + g.r.num_experts);
    int4 *map = reinterpret_cast<int4 *>(ws.take((size_t)(g.m_tiles + 1) * sizeof(int4)));
    g.tile_map = map;
    if (!ws.dry) {
      tile_map_kernel<<<1, MAP_THREADS, 0, st>>>(g.r, bm, g.m_tiles, map);
      const int got = hip_status();
      if (got != MOE_OK) return got;
    }
  }
  if (plan.splits > 1) {
    g.k_split = (int)((stages + plan.splits - 1) / plan.splits) * 64;
    g.splits = (g.K + g.k_split - 1) / g.k_split;  // none of them empty
    const int segs = mode == WGRAD ? g.segs : 1;
    g.partial = reinterpret_cast<float *>(
        ws.take((size_t)g.splits * segs * g.M * width * sizeof(float)));
    if (ws.dry) return MOE_OK;
    const int got = launch_gemm(dtype, mode, plan.kind, g, st);
    if (got != MOE_OK) return got;
    const auto kernel = dtype == MOE_BF16 ? join_kernel<Bf16> : join_kernel<F16>;
    kernel<<<row_grid(g.M, round8(g.N), segs), dim3(COL_THREADS, ROW_THREADS), 0, st>>>(g, mode);
    return hip_status();
  }
  return ws.dry ? MOE_OK : launch_gemm(dtype, mode, plan.kind, g, st);
}

static int check_common(int dtype, int act, int64_t tokens, int w0, int w1,
                        const moe_expert_rows &r, bool backward) {
  if (dtype != MOE_BF16 && dtype != MOE_F16) return MOE_ERR_UNSUPPORTED;
  if (act < MOE_ACT_NONE || act > MOE_ACT_GELU) return MOE_ERR_UNSUPPORTED;
  if (tokens < 0 || w0 <= 0 || w1 <= 0) return MOE_ERR_SHAPE;
  if (w0 > MOE_FFN_MAX_WIDTH || w1 > MOE_FFN_MAX_WIDTH || tokens > MAX_ROWS)
    return MOE_ERR_UNSUPPORTED;
  if (r.num_experts < 0) return MOE_ERR_SHAPE;
  if (r.num_experts > 0) {
    if (r.rows < 0) return MOE_ERR_SHAPE;
    if (r.num_experts > MOE_FFN_MAX_EXPERTS || r.rows > MAX_ROWS) return MOE_ERR_UNSUPPORTED;
    if (r.tile_m <= 0 || r.tile_m > MOE_GROUPED_MAX_TILE) return MOE_ERR_SHAPE;
    if (r.tile_m % 16 != 0) return MOE_ERR_UNSUPPORTED;
    if (!r.padded_offsets || (r.rows > 0 && !r.m_indices)) return MOE_ERR_NULL;
    if (backward && !r.counts) return MOE_ERR_NULL;
    if (r.row_entry && r.top_k <= 0) return MOE_ERR_SHAPE;
  }
  return MOE_OK;
}

// A matrix of `rows` x `cols`, one or `mats` of them. Optional matrices may be
// NULL, and any may where it has no elements.
int check_matrix(const moe_matrix &m, int64_t rows, int cols, int mats, bool optional) {
  if (!m.p) return optional || rows == 0 ? MOE_OK : MOE_ERR_NULL;
  if ((uintptr_t)m.p % 2 != 0) return MOE_ERR_SHAPE;
  if (rows > 1 && m.ld < cols) return MOE_ERR_SHAPE;
  if (m.ld < 0 || m.stride < 0) return MOE_ERR_SHAPE;
  if (m.ld > MOE_FFN_MAX_LD) return MOE_ERR_UNSUPPORTED;
  if (mats > 1 && m.stride < (rows - 1) * m.ld + cols) return MOE_ERR_SHAPE;
  return MOE_OK;
}
static int64_t call_rows(const moe_expert_rows &r, int64_t tokens) {
  return r.num_experts > 0 ? r.rows : tokens;
}
static int align_of(const moe_expert_rows &r) { return r.num_experts > 0 ? r.tile_m : 0; }
static int mats_of(const moe_expert_rows &r) { return r.num_experts > 0 ? r.num_experts : 1; }

// ---------------------------------------------------------------- gated block

static int check_gated(const moe_gated_ffn_args *a, bool backward) {
  if (!a) return MOE_ERR_NULL;
  MOE_TRY(check_common(a->dtype, a->activation, a->tokens, a->hidden, a->inter, a->rows, backward));
  if (a->inter > MOE_FFN_MAX_WIDTH / 2) return MOE_ERR_UNSUPPORTED;
  const int64_t rows = call_rows(a->rows, a->tokens);
  const int mats = mats_of(a->rows), H = a->hidden, F = a->inter;
  const bool gather = a->rows.num_experts > 0 && a->rows.row_entry;
  if (!gather && a->tokens < rows) return MOE_ERR_SHAPE;
  MOE_TRY(check_matrix(a->x, a->tokens, H, 1, backward && !a->dw_gate.p));
  MOE_TRY(check_matrix(a->w_gate, F, H, mats, backward && !a->dx.p));
  MOE_TRY(check_matrix(a->w_up, F, H, mats, backward && !a->dx.p));
  MOE_TRY(check_matrix(a->pre, rows, 2 * F, 1, !backward));
  if (!backward) return check_matrix(a->h, rows, F, 1, false);
  MOE_TRY(check_matrix(a->dh, rows, F, 1, false));
  MOE_TRY(check_matrix(a->dx, rows, H, 1, true));
  MOE_TRY(check_matrix(a->dw_gate, F, H, mats, true));
  MOE_TRY(check_matrix(a->dw_up, F, H, mats, true));
  return !a->dw_gate.p != !a->dw_up.p ? MOE_ERR_NULL : MOE_OK;
}

static GemmArgs gemm_args(const moe_expert_rows &r, int64_t rows, bool gather) {
  GemmArgs g = {};
  g.r = {r.counts, r.padded_offsets, r.m_indices, gather ? r.row_entry : nullptr, rows,
         r.num_experts, r.top_k};
  g.segs = 1;
  // entry / top_k for entries below 2^31: magic = ceil(2^(31 + s) / top_k) with
  // s = ceil(log2 top_k) fits 32 bits, and the product's error stays below 1
  if (gather && r.top_k > 1) {
    int s = 1;
    while ((int64_t)1 << s < r.top_k) ++s;
    g.top_k_magic = (uint32_t)((((uint64_t)1 << (31 + s)) + r.top_k - 1) / r.top_k);
    g.top_k_shift = s - 1;
  }
  return g;
}
// Gathered rows are addressed by 32-bit offsets from what the product reads: x,
// or the padded copy that operand() makes of it, whose rows may be longer than
// x's own. Where that is larger than they reach, the rows are gathered into the
// workspace first.
static bool is_wide(const moe_matrix &x, int64_t tokens, int cols) {
  const int64_t copy_ld = is_aligned(x, cols, 1) ? 0 : round8(cols);
  return tokens * (x.ld > copy_ld ? x.ld : copy_ld) * 2 >= 0xfffff000ll;
}
static Operand gathered(const moe_matrix &x, int64_t tokens, int cols, const Rows &r,
                        int64_t rows, Arena &a, hipStream_t st, int *status) {
  const int c8 = round8(cols);
  uint16_t *dst = a.take((size_t)rows * c8 * 2);
  if (!a.dry && *status == MOE_OK) {
    gather_rows_kernel<<<row_grid(rows, c8, 1), dim3(COL_THREADS, ROW_THREADS), 0, st>>>(
        (const uint16_t *)x.p, x.ld, tokens, cols, rows, r, dst, c8);
    *status = hip_status();
  }
  return {dst, c8, 0};
}
static void set_b0(GemmArgs &g, const Operand &b) {
  g.b0 = b.p, g.ldb0 = b.ld, g.b_stride0 = b.stride;
}
static void set_b1(GemmArgs &g, const Operand &b) {
  g.b1 = b.p, g.ldb1 = b.ld, g.b_stride1 = b.stride;
}
static void set_c0(GemmArgs &g, const moe_matrix &c) {
  g.c0 = (uint16_t *)c.p, g.ldc0 = c.ld, g.c_stride0 = c.stride;
}
static void set_c1(GemmArgs &g, const moe_matrix &c) {
  g.c1 = (uint16_t *)c.p, g.ldc1 = c.ld, g.c_stride1 = c.stride;
}

// The few-row forward products load their operands into registers, at any
// alignment. Over experts that is used, where padded copies would be made of every
// expert's weights, those without rows too (64 experts, 32 entries: 2047 -> 1024
// copied 158 us, direct 100, 4301 -> 512 149 and 86; 512 entries: 195 and 199, 189
// and 167). A dense product's copies are of one matrix.
static bool reads_directly(const moe_expert_rows &r, const Plan &plan) {
  return r.num_experts > 0 && plan.kind == TILE_16;
}
static Operand as_is(const moe_matrix &m) { return {(const uint16_t *)m.p, m.ld, m.stride}; }

// Whether the weight gradients go by few_rows_dw_kernel. Both gradients of a gated
// block, few rows and matrix cores: 7168 -> 2048 of 1 row 14 and 21 us, 8 rows 17 and
// 21, 16 rows 23 and 22; 64 experts of 2048 -> 512 with 1 row each 49 and 63, 8 rows 74
// and 78, 16 rows 102 and 79.
constexpr int FEW_DW_ROWS = 8;
static bool few_rows(const moe_expert_rows &r, int64_t rows) {
  return (r.num_experts > 0 ? expert_rows(r, rows) : rows) <= FEW_DW_ROWS;
}
static int run_few_rows(int dtype, bool gated, const moe_matrix &d,
                        const moe_matrix &pre, const moe_matrix &x, int64_t x_rows,
                        const moe_matrix &dw0, const moe_matrix &dw1, int64_t rows, int F, int H,
                        int act, int mats, const Rows &r, hipStream_t st) {
  FewRowsArgs a = {};
  a.d = (const uint16_t *)d.p, a.ld_d = d.ld;
  if (gated || act != MOE_ACT_NONE) a.pre = (const uint16_t *)pre.p, a.ld_pre = pre.ld;
  a.x = (const uint16_t *)x.p, a.ld_x = x.ld, a.x_rows = x_rows;
  a.dw0 = (uint16_t *)dw0.p, a.ld0 = dw0.ld, a.stride0 = dw0.stride;
  a.dw1 = (uint16_t *)dw1.p, a.ld1 = dw1.ld, a.stride1 = dw1.stride;
  a.rows = rows, a.F = F, a.H = H, a.act = act, a.r = r;
  a.f_blocks = (F + FEW_F * FEW_WAVES - 1) / (FEW_F * FEW_WAVES);
  const dim3 grid((H + 511) / 512, a.f_blocks * (gated ? 2 : 1), mats);
  const bool bf = dtype == MOE_BF16;
  const auto kernel = gated ? (bf ? few_rows_dw_kernel<Bf16, true> : few_rows_dw_kernel<F16, true>)
                            : (bf ? few_rows_dw_kernel<Bf16, false> : few_rows_dw_kernel<F16, false>);
  kernel<<<grid, 64 * FEW_WAVES, 0, st>>>(a);
  return hip_status();
}

static int run_gated(const moe_gated_ffn_args *a, Arena &ws, hipStream_t st) {
  const int64_t rows = call_rows(a->rows, a->tokens);
  const int mats = mats_of(a->rows), align = align_of(a->rows), H = a->hidden, F = a->inter;
  int status = MOE_OK;
  if (rows == 0) return MOE_OK;
  const bool gather = a->rows.num_experts > 0 && a->rows.row_entry;
  GemmArgs g = gemm_args(a->rows, rows, gather);
  g.a_rows = a->tokens;
  const Plan plan = row_plan(a->rows, true, rows, 2 * F, H);
  const bool direct = reads_directly(a->rows, plan);
  Operand x;
  if (direct) {
    x = as_is(a->x);
  } else if (gather && is_wide(a->x, a->tokens, H)) {
    x = gathered(a->x, a->tokens, H, g.r, rows, ws, st, &status);
    g.r.row_entry = nullptr;
    g.a_rows = rows;
  } else {
    x = operand(a->x, a->tokens, H, 1, ws, st, &status);
  }
  const Operand wg = direct ? as_is(a->w_gate) : operand(a->w_gate, F, H, mats, ws, st, &status);
  const Operand wu = direct ? as_is(a->w_up) : operand(a->w_up, F, H, mats, ws, st, &status);
  if (status != MOE_OK) return status;
  g.a = x.p, g.lda = x.ld;
  set_b0(g, wg);
  set_b1(g, wu);
  set_c0(g, a->h);
  g.pre = (uint16_t *)a->pre.p, g.ldp = a->pre.ld;
  g.M = (int)rows, g.N = F, g.K = H, g.act = a->activation;
  return run_product(a->dtype, GATED, plan, g, 2 * F, align, ws, st);
}

static int run_gated_backward(const moe_gated_ffn_args *a, Arena &ws, hipStream_t st) {
  const int64_t rows = call_rows(a->rows, a->tokens);
  const int mats = mats_of(a->rows), align = align_of(a->rows);
  const int H = a->hidden, F = a->inter, Fa = round8(F);
  const bool gather = a->rows.num_experts > 0 && a->rows.row_entry;
  int status = MOE_OK;
  Operand x = {}, wg = {}, wu = {};
  GemmArgs g = gemm_args(a->rows, rows, gather);
  const bool few = a->dw_gate.p && few_rows(a->rows, rows);
  const bool products = a->dx.p || (a->dw_gate.p && !few);
  uint16_t *dz = products ? ws.take((size_t)rows * 2 * Fa * 2) : nullptr;
  const bool wide = gather && is_wide(a->x, a->tokens, H);
  if (a->dw_gate.p && !few && wide) x = gathered(a->x, a->tokens, H, g.r, rows, ws, st, &status);
  if (a->dw_gate.p && !few && !wide) x = operand(a->x, a->tokens, H, 1, ws, st, &status);
  if (a->dx.p && rows > 0) {
    // the product goes from one weight to the other with the same offsets
    const bool copy = !is_aligned(a->w_gate, H, mats) || !is_aligned(a->w_up, H, mats) ||
                      a->w_gate.ld != a->w_up.ld;
    wg = operand(a->w_gate, F, H, mats, ws, st, &status, copy);
    wu = operand(a->w_up, F, H, mats, ws, st, &status, copy);
  }
  if (status != MOE_OK) return status;
  if (rows > 0 && products && !ws.dry) {
    const dim3 grid = row_grid(rows, Fa, 1), block(COL_THREADS, ROW_THREADS);
    const auto kernel = a->dtype == MOE_BF16 ? gated_dz_kernel<Bf16> : gated_dz_kernel<F16>;
    kernel<<<grid, block, 0, st>>>((const uint16_t *)a->dh.p, a->dh.ld,
                                   (const uint16_t *)a->pre.p, a->pre.ld, rows, F, a->activation,
                                   g.r, dz);
    MOE_TRY(hip_status());
  }
  g.a = dz, g.lda = 2 * Fa, g.a_seg = Fa, g.segs = 2;
  if (a->dx.p && rows > 0) {
    GemmArgs d = g;
    d.r.row_entry = nullptr;
    d.a_rows = rows;
    set_b0(d, wg);
    set_b1(d, wu);
    set_c0(d, a->dx);
    d.M = (int)rows, d.N = H, d.K = F;
    MOE_TRY(run_product(a->dtype, DGRAD, row_plan(a->rows, false, rows, H, 2 * F), d, H, align, ws, st));
  }
  if (few)
    return ws.dry ? MOE_OK
                  : run_few_rows(a->dtype, true, a->dh, a->pre, a->x, a->tokens, a->dw_gate,
                                 a->dw_up, rows, F, H, a->activation, mats, g.r, st);
  if (a->dw_gate.p) {
    set_b0(g, x);
    g.a_rows = wide ? rows : a->tokens;
    if (wide) g.r.row_entry = nullptr;
    set_c0(g, a->dw_gate);
    set_c1(g, a->dw_up);
    g.M = F, g.N = H, g.K = (int)rows;
    MOE_TRY(run_product(a->dtype, WGRAD, weight_plan(a->rows, 2, F, H, rows), g, H, align, ws, st));
  }
  return MOE_OK;
}

// --------------------------------------------------------------------- linear

static int check_linear(const moe_linear_args *a, bool backward) {
  if (!a) return MOE_ERR_NULL;
  MOE_TRY(check_common(a->dtype, a->activation, a->tokens, a->in, a->out, a->rows, backward));
  const int64_t rows = call_rows(a->rows, a->tokens);
  const int mats = mats_of(a->rows), I = a->in, O = a->out;
  MOE_TRY(check_matrix(a->x, rows, I, 1, backward && !a->dw.p));
  MOE_TRY(check_matrix(a->w, O, I, mats, backward && !a->dx.p));
  MOE_TRY(check_matrix(a->pre, rows, O, 1, !backward || a->activation == MOE_ACT_NONE));
  if (!backward) {
    MOE_TRY(check_matrix(a->bias, 1, O, mats, true));
    MOE_TRY(check_matrix(a->residual, rows, O, 1, true));
    return check_matrix(a->y, rows, O, 1, false);
  }
  MOE_TRY(check_matrix(a->dy, rows, O, 1, false));
  MOE_TRY(check_matrix(a->dx, rows, I, 1, true));
  MOE_TRY(check_matrix(a->dw, O, I, mats, true));
  return check_matrix(a->dbias, 1, O, mats, true);
}

static int run_linear(const moe_linear_args *a, Arena &ws, hipStream_t st) {
  const int64_t rows = call_rows(a->rows, a->tokens);
  const int mats = mats_of(a->rows), align = align_of(a->rows), I = a->in, O = a->out;
  int status = MOE_OK;
  if (rows == 0) return MOE_OK;
  const Plan plan = row_plan(a->rows, true, rows, O, I);
  const bool direct = reads_directly(a->rows, plan);
  const Operand x = direct ? as_is(a->x) : operand(a->x, rows, I, 1, ws, st, &status);
  const Operand w = direct ? as_is(a->w) : operand(a->w, O, I, mats, ws, st, &status);
  if (status != MOE_OK) return status;
  GemmArgs g = gemm_args(a->rows, rows, false);
  g.a = x.p, g.lda = x.ld, g.a_rows = rows;
  set_b0(g, w);
  set_c0(g, a->y);
  g.pre = (uint16_t *)a->pre.p, g.ldp = a->pre.ld;
  g.bias = (const uint16_t *)a->bias.p, g.bias_stride = a->bias.stride;
  g.res = (const uint16_t *)a->residual.p, g.ldr = a->residual.ld;
  g.M = (int)rows, g.N = O, g.K = I, g.act = a->activation;
  return run_product(a->dtype, LINEAR, plan, g, O, align, ws, st);
}

// Row ranges of the bias gradient's partial sums: dense, one for every 256
// rows, at most 64; one for an expert.
static int bias_splits(const moe_expert_rows &r, int64_t rows) {
  if (r.num_experts > 0) return 1;
  const int64_t s = rows / 256;
  return s < 1 ? 1 : s > 64 ? 64 : (int)s;
}

static int run_linear_backward(const moe_linear_args *a, Arena &ws, hipStream_t st) {
  const int64_t rows = call_rows(a->rows, a->tokens);
  const int mats = mats_of(a->rows), align = align_of(a->rows);
  const int I = a->in, O = a->out, Oa = round8(O);
  const bool bf = a->dtype == MOE_BF16;
  int status = MOE_OK;
  GemmArgs g = gemm_args(a->rows, rows, false);
  const uint16_t *dy = (const uint16_t *)a->dy.p, *pre = (const uint16_t *)a->pre.p;
  // dz: dy itself without an activation, where its pieces are aligned
  const bool few = a->dw.p && few_rows(a->rows, rows);
  const bool products = a->dx.p || (a->dw.p && !few), none = a->activation == MOE_ACT_NONE;
  Operand dz = {};
  if (products && none) dz = operand(a->dy, rows, O, 1, ws, st, &status);
  if (products && !none) dz = {ws.take((size_t)rows * Oa * 2), Oa, 0};
  uint16_t *dz_out = products && !none ? const_cast<uint16_t *>(dz.p) : nullptr;
  if (a->dbias.p) {
    const int S = bias_splits(a->rows, rows);
    float *part = reinterpret_cast<float *>(ws.take((size_t)mats * S * O * 4));
    if (!ws.dry && status == MOE_OK) {
      const dim3 grid((O + 63) / 64, S, mats), block(8, BIAS_ROWS);
      const auto sums = bf ? bias_grad_kernel<Bf16> : bias_grad_kernel<F16>;
      sums<<<grid, block, 0, st>>>(dy, a->dy.ld, pre, a->pre.ld, rows, O, a->activation, g.r, S,
                                   part, dz_out, (uint16_t *)a->dbias.p, a->dbias.stride);
      MOE_TRY(hip_status());
      if (S > 1) {
        const auto join = bf ? bias_sum_kernel<Bf16> : bias_sum_kernel<F16>;
        join<<<dim3((O + 63) / 64), 256, 0, st>>>(part, S, O, (uint16_t *)a->dbias.p);
        MOE_TRY(hip_status());
      }
    }
  } else if (dz_out && !ws.dry && rows > 0) {
    const auto kernel = bf ? linear_dz_kernel<Bf16> : linear_dz_kernel<F16>;
    kernel<<<row_grid(rows, Oa, 1), dim3(COL_THREADS, ROW_THREADS), 0, st>>>(
        dy, a->dy.ld, pre, a->pre.ld, rows, O, a->activation, g.r, dz_out);
    MOE_TRY(hip_status());
  }
  Operand x = {}, w = {};
  if (a->dw.p && !few) x = operand(a->x, rows, I, 1, ws, st, &status);
  if (a->dx.p && rows > 0) w = operand(a->w, O, I, mats, ws, st, &status);
  if (status != MOE_OK) return status;
  g.a = dz.p, g.lda = dz.ld, g.a_rows = rows;
  if (a->dx.p && rows > 0) {
    GemmArgs d = g;
    set_b0(d, w);
    set_c0(d, a->dx);
    d.M = (int)rows, d.N = I, d.K = O;
    MOE_TRY(run_product(a->dtype, DGRAD, row_plan(a->rows, false, rows, I, O), d, I, align, ws, st));
  }
  if (few)
    return ws.dry ? MOE_OK
                  : run_few_rows(a->dtype, false, a->dy, a->pre, a->x, rows, a->dw, a->dw, rows, O, I,
                                 a->activation, mats, g.r, st);
  if (a->dw.p) {
    set_b0(g, x);
    set_c0(g, a->dw);
    g.M = O, g.N = I, g.K = (int)rows;
    MOE_TRY(run_product(a->dtype, WGRAD, weight_plan(a->rows, 1, O, I, rows), g, I, align, ws, st));
  }
  return MOE_OK;
}

// -------------------------------------------------------------------- combine

static int check_combine(const moe_combine_args *a, bool backward) {
  if (!a) return MOE_ERR_NULL;
  if (a->dtype != MOE_BF16 && a->dtype != MOE_F16) return MOE_ERR_UNSUPPORTED;
  if (a->tokens < 0 || a->rows < 0 || a->width <= 0 || a->top_k <= 0 || a->num_experts < 0 ||
      a->num_ids < a->num_experts)
    return MOE_ERR_SHAPE;
  if (a->width > MOE_FFN_MAX_WIDTH || a->top_k > COMBINE_MAX_TOPK || a->tokens > MAX_ROWS ||
      a->rows > MAX_ROWS || a->tokens * a->top_k > 0x7fffffff)
    return MOE_ERR_UNSUPPORTED;
  const bool entries = a->tokens > 0 && (!backward || a->dweights);
  if (entries && (!a->packed || !a->inv_perm || !a->offsets || !a->padded_offsets))
    return MOE_ERR_NULL;
  if (!backward) {
    MOE_TRY(check_matrix(a->y, a->rows, a->width, 1, false));
    MOE_TRY(check_matrix(a->residual, a->tokens, a->width, 1, true));
    return check_matrix(a->out, a->tokens, a->width, 1, false);
  }
  if (a->rows > 0 && (!a->m_indices || !a->row_entry)) return MOE_ERR_NULL;
  MOE_TRY(check_matrix(a->y, a->rows, a->width, 1, !a->dweights));
  MOE_TRY(check_matrix(a->dout, a->tokens, a->width, 1, false));
  return check_matrix(a->dy, a->rows, a->width, 1, false);
}

static CombineArgs combine_args(const moe_combine_args *a) {
  CombineArgs c = {};
  c.width = a->width, c.top_k = a->top_k, c.num_experts = a->num_experts, c.num_ids = a->num_ids;
  c.tokens = a->tokens, c.rows = a->rows;
  c.packed = a->packed, c.inv_perm = a->inv_perm, c.offsets = a->offsets;
  c.padded_offsets = a->padded_offsets, c.m_indices = a->m_indices, c.row_entry = a->row_entry;
  c.weights = a->weights;
  c.y = (const uint16_t *)a->y.p, c.residual = (const uint16_t *)a->residual.p;
  c.dout = (const uint16_t *)a->dout.p;
  c.out = (uint16_t *)a->out.p, c.dy = (uint16_t *)a->dy.p;
  c.ld_y = a->y.ld, c.ld_res = a->residual.ld, c.ld_out = a->out.ld, c.ld_dout = a->dout.ld;
  c.ld_dy = a->dy.ld;
  c.dweights = a->dweights;
  return c;
}

}  // namespace moe_ffn

extern "C" {

int64_t moe_gated_ffn_workspace_bytes(const moe_gated_ffn_args *a, int32_t backward) {
  using namespace moe_ffn;
  return sized(a, check_gated(a, backward != 0), backward ? run_gated_backward : run_gated);
}
int moe_gated_ffn(const moe_gated_ffn_args *a, void *workspace, size_t workspace_bytes,
                  void *stream) {
  using namespace moe_ffn;
  return checked_run(a, check_gated(a, false), run_gated, workspace, workspace_bytes, stream);
}
int moe_gated_ffn_backward(const moe_gated_ffn_args *a, void *workspace, size_t workspace_bytes,
                           void *stream) {
  using namespace moe_ffn;
  return checked_run(a, check_gated(a, true), run_gated_backward, workspace, workspace_bytes,
                     stream);
}

int64_t moe_linear_workspace_bytes(const moe_linear_args *a, int32_t backward) {
  using namespace moe_ffn;
  return sized(a, check_linear(a, backward != 0), backward ? run_linear_backward : run_linear);
}
int moe_linear(const moe_linear_args *a, void *workspace, size_t workspace_bytes, void *stream) {
  using namespace moe_ffn;
  return checked_run(a, check_linear(a, false), run_linear, workspace, workspace_bytes, stream);
}
int moe_linear_backward(const moe_linear_args *a, void *workspace, size_t workspace_bytes,
                        void *stream) {
  using namespace moe_ffn;
  return checked_run(a, check_linear(a, true), run_linear_backward, workspace, workspace_bytes,
                     stream);
}

int moe_combine(const moe_combine_args *a, void *stream) {
  using namespace moe_ffn;
  MOE_TRY(check_combine(a, false));
  CombineArgs c = combine_args(a);
  const int y = (round8(a->width) / 8 + COMBINE_THREADS - 1) / COMBINE_THREADS;
  const auto kernel = a->dtype == MOE_BF16 ? combine_kernel<Bf16> : combine_kernel<F16>;
  return in_parts(a->tokens, COMBINE_THREADS, [&](int64_t first, uint32_t n) {
    c.block0 = first;
    kernel<<<dim3(n, y), COMBINE_THREADS, 0, (hipStream_t)stream>>>(c);
    return hip_status();
  });
}
int moe_combine_backward(const moe_combine_args *a, void *stream) {
  using namespace moe_ffn;
  MOE_TRY(check_combine(a, true));
  CombineArgs c = combine_args(a);
  int64_t blocks = a->rows;
  if (a->dweights)
    blocks += (a->tokens * a->top_k + COMBINE_THREADS - 1) / COMBINE_THREADS;
  const auto kernel =
      a->dtype == MOE_BF16 ? combine_backward_kernel<Bf16> : combine_backward_kernel<F16>;
  return in_parts(blocks, COMBINE_THREADS, [&](int64_t first, uint32_t n) {
    c.block0 = first;
    kernel<<<n, COMBINE_THREADS, 0, (hipStream_t)stream>>>(c);
    return hip_status();
  });
}

}  // extern "C"
