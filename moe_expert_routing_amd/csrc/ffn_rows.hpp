// ffn_rows.hpp - the memory-bound kernels of the feed-forward operators: the
// gradient of the pre-activations, the bias gradient, padded copies of
// operands, and the combination of the experts' rows. All of them are bound by
// the bytes they move, 16 a lane (4.7-5.0 TB/s is a large copy's rate here).
// 32768 tokens of width 7168 combined from 65536 rows, 1.9 GB: 360-385 us, 4.9-5.2
// TB/s. Its backward pass for 8192 tokens, 36.6 thousand rows of which 16 thousand
// hold entries, 0.98 GB with the zeros of the others: 181-188 us. dz of these rows
// at 1024 wide, 170 MB: 48 us. dz and the bias sums of 4096 x 4096, 100 MB: 19 us.
#pragma once

#include "ffn_types.hpp"

namespace moe_ffn {

__device__ __forceinline__ bool row_is_real(const Rows &r, int64_t row) {
  if (r.num_experts == 0) return true;
  const int32_t e = r.m_indices[row];
  return e >= 0 && e < r.num_experts;
}

constexpr int COL_THREADS = 64, ROW_THREADS = 4;  // block of the row-wise kernels

// dst [mats][rows, cols8] = src [mats][rows, cols] with zeros in the padding.
__global__ __launch_bounds__(COL_THREADS *ROW_THREADS) void pad_rows_kernel(
    const uint16_t *__restrict__ src, int64_t ld, int64_t stride, int64_t rows, int cols,
    uint16_t *__restrict__ dst, int cols8) {
  const int c = (blockIdx.x * COL_THREADS + threadIdx.x) * 8;
  if (c >= cols8) return;
  src += blockIdx.z * stride;
  dst += (int64_t)blockIdx.z * rows * cols8;
  for (int64_t r = blockIdx.y * ROW_THREADS + threadIdx.y; r < rows;
       r += (int64_t)gridDim.y * ROW_THREADS) {
    const s16x8 w = load8_raw(src + r * ld, c, cols);
    *reinterpret_cast<s16x8 *>(dst + r * cols8 + c) = w;
  }
}

// dst [rows, cols8] = the token rows of x that the rows of a layout are made
// from, zeros on rows without one and in the padding.
__global__ __launch_bounds__(COL_THREADS *ROW_THREADS) void gather_rows_kernel(
    const uint16_t *__restrict__ x, int64_t ld, int64_t tokens, int cols, int64_t rows, Rows r,
    uint16_t *__restrict__ dst, int cols8) {
  const int c = (blockIdx.x * COL_THREADS + threadIdx.x) * 8;
  if (c >= cols8) return;
  for (int64_t m = blockIdx.y * ROW_THREADS + threadIdx.y; m < rows;
       m += (int64_t)gridDim.y * ROW_THREADS) {
    s16x8 w = {0, 0, 0, 0, 0, 0, 0, 0};
    const int32_t entry = row_is_real(r, m) ? r.row_entry[m] : -1;
    const int64_t t = entry / r.top_k;
    if (entry >= 0 && t < tokens) w = load8_raw(x + t * ld, c, cols);
    *reinterpret_cast<s16x8 *>(dst + m * cols8 + c) = w;
  }
}

// The m-tiles of bm rows over a layout, each within one expert's rows: rows
// [x, y) of tile i in map[i], the experts' first and in order, then the rows past
// them, then empty ones up to m_tiles; map[m_tiles].x: how many the experts have.
constexpr int MAP_THREADS = 1024;
__global__ __launch_bounds__(MAP_THREADS) void tile_map_kernel(Rows r, int bm, int m_tiles,
                                                               int4 *__restrict__ map) {
  __shared__ int sums[MAP_THREADS];
  constexpr int EACH = MOE_FFN_MAX_EXPERTS / MAP_THREADS;
  const int t = threadIdx.x, rows = (int)r.rows;
  auto first_row = [&](int e) { return min(max(r.padded_offsets[min(e, r.num_experts)], 0), rows); };
  int tiles[EACH], mine = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int e = t * EACH + i;
    tiles[i] = e < r.num_experts ? (max(first_row(e + 1) - first_row(e), 0) + bm - 1) / bm : 0;
    mine += tiles[i];
  }
  sums[t] = mine;
  __syncthreads();
  for (int d = 1; d < MAP_THREADS; d *= 2) {  // inclusive sums
    const int v = t >= d ? sums[t - d] : 0;
    __syncthreads();
    sums[t] += v;
    __syncthreads();
  }
  int at = sums[t] - mine;
  const int live = min(sums[MAP_THREADS - 1], m_tiles), end = first_row(r.num_experts);
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int e = t * EACH + i;
    const int lo = first_row(e), hi = first_row(e + 1);
    for (int k = 0; k < tiles[i]; ++k, ++at)
      if (at < m_tiles) map[at] = make_int4(lo + k * bm, min(lo + (k + 1) * bm, hi), 0, 0);
  }
  for (int i = live + t; i < m_tiles; i += MAP_THREADS) {
    const int64_t lo = end + (int64_t)(i - live) * bm;
    map[i] = make_int4((int)min(lo, (int64_t)rows), (int)min(lo + bm, (int64_t)rows), 0, 0);
  }
  if (t == 0) map[m_tiles] = make_int4(live, 0, 0, 0);
}

// Gradient of a gated block's pre-activations: dz [rows, 2 Fa] with dg = dh u
// act'(g) in the first Fa = round_up(F, 8) columns and du = dh act(g) in the
// others, zeros in the padding. Rows without an entry are left as they are: the
// products never read them.
//
// It is rounded to the matrices' type, because the matrix cores multiply 16-bit
// operands: dz in two halves, high and low, would keep fp32's bits at twice the
// operations of both products. The rounding adds as much error to dx and dW as
// their own final one, and independent of it: 0.0023 (bf16) and 0.00029 (fp16) in
// the 2-norm where that alone gives 0.0017 and 0.00021. With fp16 values above
// 65504 become infinite.
template <class D>
__global__ __launch_bounds__(COL_THREADS *ROW_THREADS) void gated_dz_kernel(
    const uint16_t *__restrict__ dh, int64_t ld_dh, const uint16_t *__restrict__ pre,
    int64_t ld_pre, int64_t rows, int F, int act, Rows r, uint16_t *__restrict__ dz) {
  const int Fa = (F + 7) & ~7;
  const int c = (blockIdx.x * COL_THREADS + threadIdx.x) * 8;
  if (c >= Fa) return;
  for (int64_t m = blockIdx.y * ROW_THREADS + threadIdx.y; m < rows;
       m += (int64_t)gridDim.y * ROW_THREADS) {
    if (!row_is_real(r, m)) continue;
    const f32x8 d = load8<D>(dh + m * ld_dh, c, F);
    const f32x8 gt = load8<D>(pre + m * ld_pre, c, F);
    const f32x8 up = load8<D>(pre + m * ld_pre + F, c, F);
    f32x8 dg, du, v, s;
    act_value_slope(gt, act, v, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dg[i] = d[i] * up[i] * s[i];
      du[i] = d[i] * v[i];
    }
    uint16_t *o = dz + m * (2 * (int64_t)Fa);
    *reinterpret_cast<s16x8 *>(o + c) = pack8<D>(dg);
    *reinterpret_cast<s16x8 *>(o + Fa + c) = pack8<D>(du);
  }
}

// dz [rows, Oa] = dy act'(pre), rounded as above.
template <class D>
__global__ __launch_bounds__(COL_THREADS *ROW_THREADS) void linear_dz_kernel(
    const uint16_t *__restrict__ dy, int64_t ld_dy, const uint16_t *__restrict__ pre,
    int64_t ld_pre, int64_t rows, int O, int act, Rows r, uint16_t *__restrict__ dz) {
  const int Oa = (O + 7) & ~7;
  const int c = (blockIdx.x * COL_THREADS + threadIdx.x) * 8;
  if (c >= Oa) return;
  for (int64_t m = blockIdx.y * ROW_THREADS + threadIdx.y; m < rows;
       m += (int64_t)gridDim.y * ROW_THREADS) {
    if (!row_is_real(r, m)) continue;
    f32x8 d = load8<D>(dy + m * ld_dy, c, O);
    f32x8 v, s;
    act_value_slope(load8<D>(pre + m * ld_pre, c, O), act, v, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] *= s[i];
    *reinterpret_cast<s16x8 *>(dz + m * (int64_t)Oa + c) = pack8<D>(d);
  }
}

// Column sums of dz = dy act'(pre) in fp32, from dy and pre themselves: the
// bias gradient does not see dz's rounding; dz itself is written on the way
// where it is wanted (not NULL), rounded as above. A block sums 64 columns of one of S row
// ranges: 8 lanes across, 32 rows at a time, then the 32 partial sums in a
// fixed order. part [mats][S][O]; one range is the whole sum and goes to db, a
// launch less (300 rows of 1024 -> 1024 with silu, whole backward: 25 and 23 us).
constexpr int BIAS_ROWS = 32;
template <class D>
__global__ __launch_bounds__(8 * BIAS_ROWS) void bias_grad_kernel(
    const uint16_t *__restrict__ dy, int64_t ld_dy, const uint16_t *__restrict__ pre,
    int64_t ld_pre, int64_t rows, int O, int act, Rows r, int S, float *__restrict__ part,
    uint16_t *__restrict__ dz, uint16_t *__restrict__ db, int64_t db_stride) {
  __shared__ float sum[BIAS_ROWS][65];
  const int c = blockIdx.x * 64 + threadIdx.x * 8;
  int64_t first = 0, n = rows;
  if (r.num_experts > 0) {
    first = min(max((int64_t)r.padded_offsets[blockIdx.z], (int64_t)0), r.rows);
    n = min(max((int64_t)r.counts[blockIdx.z], (int64_t)0), r.rows - first);
  }
  const int64_t per = (n + S - 1) / S, lo = min(n, blockIdx.y * per), hi = min(n, lo + per);
  f32x8 a = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < O) {
    for (int64_t m = first + lo + threadIdx.y; m < first + hi; m += BIAS_ROWS) {
      f32x8 d = load8<D>(dy + m * ld_dy, c, O);
      if (act != MOE_ACT_NONE) {
        f32x8 v, s;
        act_value_slope(load8<D>(pre + m * ld_pre, c, O), act, v, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= s[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] += d[i];
      if (dz) *reinterpret_cast<s16x8 *>(dz + m * ((O + 7) & ~7) + c) = pack8<D>(d);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[threadIdx.y][threadIdx.x * 8 + i] = a[i];
  __syncthreads();
  const int t = threadIdx.y * 8 + threadIdx.x;
  if (t < 64 && blockIdx.x * 64 + t < O) {
    float v = 0.f;
    for (int y = 0; y < BIAS_ROWS; ++y) v += sum[y][t];
    if (S == 1)
      db[blockIdx.z * db_stride + blockIdx.x * 64 + t] = from_f<D>(v);
    else
      part[((int64_t)blockIdx.z * S + blockIdx.y) * O + blockIdx.x * 64 + t] = v;
  }
}
// The S partial sums of 64 columns of a dense product: four ranges of them, then
// the four.
template <class D>
__global__ __launch_bounds__(256) void bias_sum_kernel(const float *__restrict__ part, int S, int O,
                                                       uint16_t *__restrict__ db) {
  __shared__ float sum[4][64];
  const int c = blockIdx.x * 64 + threadIdx.x % 64, q = threadIdx.x / 64;
  float v = 0.f;
  if (c < O) {
    const float *p = part + c;
#pragma unroll 8
    for (int s = S * q / 4; s < S * (q + 1) / 4; ++s) v += p[(int64_t)s * O];
  }
  sum[q][threadIdx.x % 64] = v;
  __syncthreads();
  if (q == 0 && c < O)
    db[c] = from_f<D>(((v + sum[1][threadIdx.x]) + sum[2][threadIdx.x]) + sum[3][threadIdx.x]);
}

// Weight gradients of few rows, dW[f, h] = sum over the rows of dz[row, f]
// x[row, h], in fp32 and with dz unrounded: over a handful of rows dz's rounding
// would not average out, and the matrix cores' 64-row stages are mostly
// empty. Bound by writing dW. A block takes 32 f and 512 h; the dz of its f are
// formed in LDS from dh or dy, 16 rows at a time, and a wave multiplies 8 f by 8
// consecutive h a lane, 64 sums.
constexpr int FEW_F = 8, FEW_WAVES = 4, FEW_ROWS = 16;
struct FewRowsArgs {
  const uint16_t *d, *pre, *x;  // d: dh or dy; pre: NULL without an activation
  int64_t ld_d, ld_pre, ld_x, x_rows, rows;
  uint16_t *dw0, *dw1;  // dw1: gated, of the second projection
  int64_t ld0, ld1, stride0, stride1;
  int F, H, f_blocks, act;
  Rows r;
};
template <class D, bool GATED_DZ>
__global__ __launch_bounds__(64 * FEW_WAVES) void few_rows_dw_kernel(const FewRowsArgs a) {
  __shared__ __attribute__((aligned(32))) float dz[FEW_ROWS][FEW_F * FEW_WAVES];
  __shared__ int64_t at[FEW_ROWS];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int seg = blockIdx.y / a.f_blocks, e = blockIdx.z;
  const int fb = blockIdx.y % a.f_blocks * FEW_F * FEW_WAVES, f0 = fb + wave * FEW_F;
  const int c = (blockIdx.x * 64 + lane) * 8;
  int64_t first = 0, n = a.rows;
  if (a.r.num_experts > 0) {
    first = min(max((int64_t)a.r.padded_offsets[e], (int64_t)0), a.rows);
    n = min(max((int64_t)a.r.counts[e], (int64_t)0), a.rows - first);
    if (a.r.row_entry && a.x_rows == 0) n = 0;  // not even a row 0 to gather
  }
  f32x8 acc[FEW_F];
#pragma unroll
  for (int i = 0; i < FEW_F; ++i) acc[i] = f32x8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t m0 = first; m0 < first + n; m0 += FEW_ROWS) {
    const int rows = (int)min(first + n - m0, (int64_t)FEW_ROWS);
    __syncthreads();
    if (lane < rows) {  // each wave its own 8 f, a row a lane
      const int64_t m = m0 + lane;
      f32x8 v = load8<D>(a.d + m * a.ld_d, f0, a.F);
      if (a.pre) {
        f32x8 value, slope;
        act_value_slope(load8<D>(a.pre + m * a.ld_pre, f0, a.F), a.act, value, slope);
        if (GATED_DZ && seg == 0) v *= load8<D>(a.pre + m * a.ld_pre + a.F, f0, a.F);
        v *= GATED_DZ && seg == 1 ? value : slope;
      }
      *reinterpret_cast<f32x8 *>(&dz[lane][wave * FEW_F]) = v;
      int64_t row = m;
      if (a.r.row_entry) {
        const uint32_t t = (uint32_t)a.r.row_entry[m] / (uint32_t)a.r.top_k;
        row = t < (uint64_t)a.x_rows ? t : 0;
      }
      if (wave == 0) at[lane] = row * a.ld_x;
    }
    __syncthreads();
#pragma unroll 4
    for (int i = 0; i < rows; ++i) {
      const f32x8 x = load8<D>(a.x + at[i], c, a.H);
      const f32x8 d = *reinterpret_cast<const f32x8 *>(&dz[i][wave * FEW_F]);
#pragma unroll
      for (int f = 0; f < FEW_F; ++f)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[f][j] = fmaf(d[f], x[j], acc[f][j]);
    }
  }
  uint16_t *dw = seg ? a.dw1 + e * a.stride1 : a.dw0 + e * a.stride0;
  const int64_t ld = seg ? a.ld1 : a.ld0;
#pragma unroll
  for (int i = 0; i < FEW_F; ++i)
    if (f0 + i < a.F) store8<D>(dw + (f0 + i) * ld, c, a.H, acc[i]);
}

// The partial sums of a product that was split over k, added in the order of
// the ranges, and its epilogue. blockIdx.z: WGRAD's segment.
template <class D>
__global__ __launch_bounds__(COL_THREADS *ROW_THREADS) void join_kernel(const GemmArgs g, int mode) {
  const int c = (blockIdx.x * COL_THREADS + threadIdx.x) * 8;
  if (c >= g.N) return;
  const int width = mode == GATED ? 2 * g.N : g.N, segs = mode == WGRAD ? g.segs : 1;
  const int64_t range = (int64_t)segs * g.M * width;
  uint16_t *out = mode == WGRAD && blockIdx.z ? g.c1 : g.c0;
  const int64_t ldc = mode == WGRAD && blockIdx.z ? g.ldc1 : g.ldc0;
  for (int64_t m = blockIdx.y * ROW_THREADS + threadIdx.y; m < g.M;
       m += (int64_t)gridDim.y * ROW_THREADS) {
    const float *p = g.partial + (blockIdx.z * (int64_t)g.M + m) * width;
    f32x8 z = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, u = z;
#pragma unroll 4
    for (int s = 0; s < g.splits; ++s) {
      const f32x8 a = load8_f32(p + s * range, c, g.N);
#pragma unroll
      for (int v = 0; v < 8; ++v) z[v] += a[v];
      if (mode == GATED) {
        const f32x8 b = load8_f32(p + s * range + g.N, c, g.N);
#pragma unroll
        for (int v = 0; v < 8; ++v) u[v] += b[v];
      }
    }
    if (mode == GATED) {
      if (g.pre) {
        store8<D>(g.pre + m * g.ldp, c, g.N, z);
        store8<D>(g.pre + m * g.ldp + g.N, c, g.N, u);
      }
      z = act_value(z, g.act);
#pragma unroll
      for (int v = 0; v < 8; ++v) z[v] *= u[v];
    } else if (mode == LINEAR) {
      if (g.bias) {
        const f32x8 b = load8<D>(g.bias, c, g.N);
#pragma unroll
        for (int v = 0; v < 8; ++v) z[v] += b[v];
      }
      if (g.pre) store8<D>(g.pre + m * g.ldp, c, g.N, z);
      z = act_value(z, g.act);
      if (g.res) {
        const f32x8 r = load8<D>(g.res + m * g.ldr, c, g.N);
#pragma unroll
        for (int v = 0; v < 8; ++v) z[v] += r[v];
      }
    }
    store8<D>(out + m * ldc, c, g.N, z);
  }
}

// ------------------------------------------------------------------ combine

struct CombineArgs {
  int width, top_k, num_experts, num_ids;
  int64_t tokens, rows;
  const int32_t *packed, *inv_perm, *offsets, *padded_offsets, *m_indices, *row_entry;
  const float *weights;
  const uint16_t *y, *residual, *dout;
  uint16_t *out, *dy;
  int64_t ld_y, ld_res, ld_out, ld_dout, ld_dy;
  float *dweights;
  int64_t block0;  // number of the launch's first block
};

// Row of an entry, or -1 where it is left out.
__device__ __forceinline__ int64_t entry_row(const CombineArgs &a, int64_t entry) {
  const int32_t e = a.packed[entry] >> 16;
  if (e < 0 || e >= a.num_experts || e >= a.num_ids) return -1;
  const int64_t row = (int64_t)a.inv_perm[entry] - a.offsets[e] + a.padded_offsets[e];
  return row >= 0 && row < a.rows ? row : -1;
}

constexpr int COMBINE_MAX_TOPK = 64;
constexpr int COMBINE_THREADS = 256;

// One block per token and run of columns. The token's rows are found once,
// by one lane each, and closed up in the order of k.
template <class D>
__global__ __launch_bounds__(COMBINE_THREADS) void combine_kernel(const CombineArgs a) {
  __shared__ int64_t rows[COMBINE_MAX_TOPK];
  __shared__ float ws[COMBINE_MAX_TOPK];
  __shared__ int n_rows;
  const int64_t t = a.block0 + blockIdx.x;
  if (threadIdx.x < 64) {
    const int k = threadIdx.x;
    int64_t row = -1;
    float w = 1.f;
    if (k < a.top_k) {
      row = entry_row(a, t * a.top_k + k);
      if (a.weights) w = a.weights[t * a.top_k + k];
    }
    const uint64_t there = __ballot(row >= 0);
    if (row >= 0) {
      const int at = __popcll(there & ((1ull << k) - 1));
      rows[at] = row;
      ws[at] = w;
    }
    if (k == 0) n_rows = __popcll(there);
  }
  __syncthreads();
  const int n = n_rows;
  for (int c = (blockIdx.y * COMBINE_THREADS + threadIdx.x) * 8; c < a.width;
       c += gridDim.y * COMBINE_THREADS * 8) {
    f32x8 s = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a.residual) s = load8<D>(a.residual + t * a.ld_res, c, a.width);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const f32x8 v = load8<D>(a.y + rows[k] * a.ld_y, c, a.width);
      const float w = ws[k];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = fmaf(w, v[i], s[i]);
    }
    store8<D>(a.out + t * a.ld_out, c, a.width, s);
  }
}

// One block per row: dy of the row, and its entry's dweights. The blocks
// after the rows' clear dweights of the entries that have no row.
template <class D>
__global__ __launch_bounds__(COMBINE_THREADS) void combine_backward_kernel(const CombineArgs a) {
  __shared__ float part[COMBINE_THREADS / 64];
  const int64_t row = a.block0 + blockIdx.x;
  if (row >= a.rows) {
    const int64_t i = (row - a.rows) * COMBINE_THREADS + threadIdx.x;
    if (i < a.tokens * a.top_k && entry_row(a, i) < 0) a.dweights[i] = 0.f;
    return;
  }
  const int32_t e = a.m_indices[row], entry = a.row_entry[row];
  const bool real = e >= 0 && e < a.num_experts && entry >= 0 &&
                    entry < a.tokens * a.top_k;
  const int64_t t = real ? entry / a.top_k : 0;
  const float w = real ? (a.weights ? a.weights[entry] : 1.f) : 0.f;
  float dot = 0.f;
  for (int c = threadIdx.x * 8; c < a.width; c += COMBINE_THREADS * 8) {
    f32x8 d = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (real) {
      d = load8<D>(a.dout + t * a.ld_dout, c, a.width);
      if (a.dweights) {
        const f32x8 v = load8<D>(a.y + row * a.ld_y, c, a.width);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(d[i], v[i], dot);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] *= w;
    }
    store8<D>(a.dy + row * a.ld_dy, c, a.width, d);
  }
  if (!real || !a.dweights) return;
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) dot += __shfl_xor(dot, s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.f;
    for (int i = 0; i < COMBINE_THREADS / 64; ++i) v += part[i];
    a.dweights[entry] = v;
  }
}

}  // namespace moe_ffn
