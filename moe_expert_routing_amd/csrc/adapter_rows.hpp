// adapter_rows.hpp - the kernels of the low-rank adapters beside the product: s = c_a
// x A_a^T (and u = c_a dy B_a, the same on a transposed copy of B), the tokens in
// the order of their adapters, transposed copies, and the adapters' gradients.
#pragma once

#include "../../include/moe_adapter.h"
#include "adapter_expand.hpp"
#include "ffn_gemm.hpp"

namespace moe_adapter {

using namespace moe_ffn;

// ------------------------------------------------------------ s = c_a x A_a^T

struct ShrinkArgs {
  const uint16_t *x, *a;  // a [rank, K] of each adapter
  int64_t ldx, lda, stride;
  const int32_t *ids;
  const float *scale;  // NULL: 1
  float *s;            // [M, rank]
  int32_t M, K, rank, n;
};

// A block takes 16 MT rows, its waves share K; x and A go from memory straight into
// MFMA operands, one batch of U k-steps loading while the other multiplies, and the
// waves' sums meet in LDS. For each adapter among the rows the block goes through
// K once: requests lie together, so a prompt's blocks have one or two. A decode
// batch's rows may all have adapters of their own, and gridDim.y blocks share them.
template <class D, int MT, int RB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void shrink_kernel(const ShrinkArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int ROWS = 16 * MT, U = MT + RB <= 3 ? 4 : 2;
  __shared__ __attribute__((aligned(16))) float part[WAVES][ROWS][16 * RB + 4];
  const int lane = threadIdx.x & 63, fr = lane & 15, fq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row0 = blockIdx.x * ROWS;
  int id = lane < ROWS && row0 + lane < g.M ? g.ids[row0 + lane] : -1;
  if ((uint32_t)id >= (uint32_t)g.n) id = -1;
  const uint64_t with = __ballot(id >= 0);
  // rows without an adapter
  if (blockIdx.y == 0)
    for (int o = threadIdx.x; o < ROWS * g.rank; o += 64 * WAVES) {
      const int r = o / g.rank;
      if (row0 + r < g.M && !(with >> r & 1)) g.s[(int64_t)row0 * g.rank + o] = 0.f;
    }
  const int steps = (g.K + 31) / 32, per = ((steps + WAVES - 1) / WAVES + 1) & ~1;
  const int s0 = min(steps, wave * per), s1 = min(steps, s0 + per);
  const int whole = max(0, (min(s1, g.K / 32) - s0) / U);
  const uint16_t *xr[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
    xr[i] = g.x + (int64_t)min(row0 + 16 * i + fr, g.M - 1) * g.ldx + s0 * 32 + fq * 8;
  uint64_t todo = with;
  for (uint32_t turn = 0; todo; ++turn) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t mine = __ballot(id == a);
    todo &= ~mine;
    if (turn % gridDim.y != blockIdx.y) continue;
    const uint16_t *ar[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r)
      ar[r] = g.a + a * g.stride + (int64_t)min(16 * r + fr, g.rank - 1) * g.lda + s0 * 32 + fq * 8;
    f32x4 acc[RB][MT];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    s16x8 fa[2][U][RB], fx[2][U][MT];
    auto load = [&](int set, int s) MOE_INLINE {
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int r = 0; r < RB; ++r)
          fa[set][u][r] = *reinterpret_cast<const s16x8_any *>(ar[r] + (s + u) * 32);
#pragma unroll
        for (int i = 0; i < MT; ++i)
          fx[set][u][i] = *reinterpret_cast<const s16x8_any *>(xr[i] + (s + u) * 32);
      }
    };
    auto multiply = [&](int set) MOE_INLINE {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
          for (int i = 0; i < MT; ++i)
            acc[r][i] = D::mfma(fa[set][u][r], fx[set][u][i], acc[r][i]);
    };
    int b = 0;
    if (whole > 0) load(0, 0);
    for (; b + 2 <= whole; b += 2) {
      load(1, (b + 1) * U);
      multiply(0);
      if (b + 2 < whole) load(0, (b + 2) * U);
      multiply(1);
    }
    if (b < whole) multiply(0);
    for (int s = whole * U; s < s1 - s0; ++s) {  // the rest, and K's own tail
      const int in = g.K - (s0 + s) * 32 - fq * 8;
      s16x8 ta[RB];
#pragma unroll
      for (int r = 0; r < RB; ++r) ta[r] = load8_raw(ar[r] + s * 32, 0, in);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const s16x8 tx = load8_raw(xr[i] + s * 32, 0, in);
#pragma unroll
        for (int r = 0; r < RB; ++r) acc[r][i] = D::mfma(ta[r], tx, acc[r][i]);
      }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        *reinterpret_cast<f32x4 *>(&part[wave][16 * i + fr][16 * r + 4 * fq]) = acc[r][i];
    __syncthreads();
    const float c = g.scale ? g.scale[a] : 1.f;
    for (int o = threadIdx.x; o < ROWS * 16 * RB; o += 64 * WAVES) {
      const int t = o / (16 * RB), r = o % (16 * RB);
      if (!(mine >> t & 1) || r >= g.rank) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v += part[w][t][r];
      g.s[(int64_t)(row0 + t) * g.rank + r] = v * c;
    }
    __syncthreads();  // before the next adapter's sums
  }
#endif
}

// ------------------------------------------- the tokens of each adapter, in order

constexpr int SORT_THREADS = 1024;

// perm: the tokens with an adapter, by adapter and then by number; offsets[a]: where
// those of adapter a begin. A block for each adapter counts the ids below its own and
// its own, and writes its tokens: two reads of the ids a block, and no atomics.
__global__ __launch_bounds__(SORT_THREADS) void sort_ids_kernel(const int32_t *__restrict__ ids,
                                                                int T, int n,
                                                                int32_t *__restrict__ offsets,
                                                                int32_t *__restrict__ perm) {
  __shared__ int sums[SORT_THREADS], below;
  const int a = blockIdx.x, t = threadIdx.x;
  if (t == 0) below = 0;
  __syncthreads();
  const int each = (T + SORT_THREADS - 1) / SORT_THREADS;
  const int lo = (int)min((int64_t)t * each, (int64_t)T), hi = (int)min((int64_t)lo + each, (int64_t)T);
  int less = 0, same = 0;
  for (int i = lo; i < hi; ++i) {
    const int id = ids[i];
    less += id >= 0 && id < a;
    same += id == a;
  }
  atomicAdd(&below, less);  // a sum of whole numbers: any order
  sums[t] = same;
  __syncthreads();
  for (int d = 1; d < SORT_THREADS; d *= 2) {  // inclusive sums
    const int v = t >= d ? sums[t - d] : 0;
    __syncthreads();
    sums[t] += v;
    __syncthreads();
  }
  const int first = below;
  if (t == 0) offsets[a] = first;
  if (a == n - 1 && t == SORT_THREADS - 1) offsets[n] = first + sums[t];
  int at = first + sums[t] - same;
  for (int i = lo; i < hi; ++i)
    if (ids[i] == a) perm[at++] = i;
}

// ---------------------------------------------------------- transposed copies

// dst [cols, rows8] = src [rows, cols] transposed, zeros from rows to rows8, of the
// adapters that have tokens: A for dx's product, whose operand needs the rank along
// its rows, and B (rows and columns exchanged) for u's.
struct TransposeArgs {
  const uint16_t *src;
  int64_t ld, stride;
  uint16_t *dst;
  int32_t rank, width, ld_dst;  // the long side's length
};
// A [rank, in] -> [in, rank8]
__device__ __forceinline__ void transpose_a(const TransposeArgs &g, int a, int c) {
  const uint16_t *src = g.src + a * g.stride + c;
  uint16_t *dst = g.dst + ((int64_t)a * g.width + c) * g.ld_dst;
  for (int r = 0; r < g.rank; r += 8) {
    s16x8 w = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < 8; ++v)
      if (r + v < g.rank) w[v] = (short)src[(r + v) * g.ld];
    *reinterpret_cast<s16x8 *>(dst + r) = w;
  }
}
// B [out, rank] -> [rank, out8]
__device__ __forceinline__ void transpose_b(const TransposeArgs &g, int a, int c) {
  const uint16_t *src = g.src + a * g.stride + c * g.ld;
  uint16_t *dst = g.dst + (int64_t)a * g.rank * g.ld_dst + c;
  for (int r = 0; r < g.rank; r += 8) {
    const s16x8 w = load8_raw(src, r, g.rank);
#pragma unroll
    for (int v = 0; v < 8; ++v)
      if (r + v < g.rank) dst[(int64_t)(r + v) * g.ld_dst] = (uint16_t)w[v];
  }
}
__global__ __launch_bounds__(256) void transpose_kernel(const TransposeArgs a, const TransposeArgs b,
                                                        const int32_t *__restrict__ offsets, int n,
                                                        int a_blocks) {
  const int e = blockIdx.y;
  if (offsets[e + 1] == offsets[e]) return;
  const bool second = (int)blockIdx.x >= a_blocks;
  const int c = (blockIdx.x - (second ? a_blocks : 0)) * 256 + threadIdx.x;
  if (!second && c < a.width) transpose_a(a, e, c);
  if (second && c < b.width) transpose_b(b, e, c);
}

// ------------------------------------------------------- the adapters' gradients

// sum over the tokens t of adapter a of v[t, r] m[t, c]: dA with v = u and m = x, dB
// (transposed) with v = s and m = dy.
struct GradSide {
  const uint16_t *m;
  int64_t ld;
  const float *v;  // [T, rank]
  float *part;     // [slots][rank][width4]
  int32_t width, width4, tiles;
};
struct GradArgs {
  GradSide side[2];
  const int32_t *offsets, *perm;
  int32_t rank, n, chunk;  // sorted tokens of a block
};

constexpr int GRAD_COLS = 256, GRAD_K = 64, GRAD_WAVES = 4;

// A block takes 256 columns of m and `chunk` tokens of the sorted order, and adds
// up each adapter among them apart: the part of adapter a in chunk k goes to slot
// a + k, of which there is one for each pair that meets. 64 tokens at a time go through
// LDS: m as it lies, read through the transposing LDS load, and v in two halves of the
// type, transposed as it is written. In fp16, whose range v may pass, the 64
// values of a column of v are taken at a power of two of their own.
template <class D, int RB>
__global__ __launch_bounds__(64 * GRAD_WAVES, RB <= 2 ? 2 : 1) void grad_kernel(const GradArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool SCALED = D::MAX_EXPONENT < 127;
  constexpr int ROW = GRAD_COLS * 2, M_BYTES = GRAD_K * ROW, V_BYTES = 16 * RB * GRAD_K * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t m_lds[2][M_BYTES];
  __shared__ __attribute__((aligned(1024))) uint8_t v_lds[2][2][V_BYTES];  // high, low
  __shared__ int power[2][16 * RB];
  const int lane = threadIdx.x & 63, fr = lane & 15, fq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool second = (int)blockIdx.x >= g.side[0].tiles;
  const GradSide &sd = g.side[second];
  const int c0 = (blockIdx.x - (second ? g.side[0].tiles : 0)) * GRAD_COLS;
  const int total = g.offsets[g.n];
  const int64_t first64 = (int64_t)blockIdx.y * g.chunk;
  if (first64 >= total) return;
  const int first = (int)first64, last = min(first + g.chunk, total);

  // the adapter of the chunk's first token: the last one that begins at or before it
  int lo = 0, hi = g.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.offsets[mid] <= first) lo = mid; else hi = mid - 1;
  }

  // this thread's pieces of a stage: 16 bytes of rows k0 + 8 q
  const int k0 = threadIdx.x >> 5, piece = threadIdx.x & 31;
  auto chunk_at = [&](int k, int c) MOE_INLINE { return k * ROW + ((c ^ swz<GRAD_COLS>(k)) * 16); };
  // transposed reads: a lane's k-row and chunk of the wave's first 16 columns
  const int tk = fq * 8 + (fr >> 2);
  const uint32_t tr = tk * ROW + (((wave * 8) + ((fr & 3) >> 1)) ^ swz<GRAD_COLS>(tk)) * 16 + (fr & 1) * 8;

  for (int a = lo; a < g.n && g.offsets[a] < last; ++a) {
    const int begin = max(g.offsets[a], first), end = min(g.offsets[a + 1], last);
    if (begin >= end) continue;
    const int stages = (end - begin + GRAD_K - 1) / GRAD_K;
    f32x4 acc[RB][4];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    int token[8], v_token;
    s16x8 m[8];
    f32x4 v[RB];
    auto load_tokens = [&](int s) MOE_INLINE {
#pragma unroll
      for (int q = 0; q < 8; ++q) token[q] = g.perm[min(begin + s * GRAD_K + k0 + 8 * q, end - 1)];
      v_token = g.perm[min(begin + s * GRAD_K + lane, end - 1)];
    };
    // rows past the end are zeros on both sides
    auto load_stage = [&](int s) MOE_INLINE {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        m[q] = s16x8{0, 0, 0, 0, 0, 0, 0, 0};
        if (begin + s * GRAD_K + k0 + 8 * q < end)
          m[q] = load8_raw(sd.m + (int64_t)token[q] * sd.ld, c0 + piece * 8, sd.width);
      }
#pragma unroll
      for (int r = 0; r < RB; ++r) {  // this wave's 4 RB of the rank
        const int at = (wave * RB + r) * 4;
        v[r] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (begin + s * GRAD_K + lane < end) {
          const float *p = sd.v + (int64_t)v_token * g.rank + at;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (at + e < g.rank) v[r][e] = p[e];
        }
      }
    };
    auto store_stage = [&](int buf) MOE_INLINE {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *reinterpret_cast<s16x8 *>(m_lds[buf] + chunk_at(k0 + 8 * q, piece)) = m[q];
#pragma unroll
      for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = (wave * RB + r) * 4 + e;
          float f = v[r][e];
          if constexpr (SCALED) {
            float most = fabsf(f);
#pragma unroll
            for (int d = 1; d < 64; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
            const int p = exponent_for(most);
            if (lane == 0) power[buf][at] = p;
            f = __builtin_amdgcn_ldexpf(f, p);
          }
          const uint16_t h = from_f<D>(f);
          const float fh = to_f<D>(h);
          const int o = at * (GRAD_K * 2) + (((lane >> 3) ^ (at & 7)) * 16) + (lane & 7) * 2;
          *reinterpret_cast<uint16_t *>(v_lds[buf][0] + o) = h;
          *reinterpret_cast<uint16_t *>(v_lds[buf][1] + o) = from_f<D>(__builtin_isfinite(fh) ? f - fh : 0.f);
        }
    };
    load_tokens(0);
    load_stage(0);
    if (stages > 1) load_tokens(1);
    for (int s = 0; s < stages; ++s) {
      const int buf = s & 1;
      store_stage(buf);
      if (s + 1 < stages) load_stage(s + 1);
      if (s + 2 < stages) load_tokens(s + 2);
      // the buffer's last readers, two stages ago, passed the barrier in between
      __syncthreads();
      f32x4 sum[SCALED ? RB : 1][4];
      if constexpr (SCALED) {
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        s16x8 fm[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint8_t *p = m_lds[buf] + (tr ^ (j * 32)) + ks * 32 * ROW;
          const s16x4 x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr_t)p);
          const s16x4 x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr_t)(p + 4 * ROW));
          fm[j] = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const int row = 16 * r + fr;
          const int o = row * (GRAD_K * 2) + (((ks * 4 + fq) ^ (row & 7)) * 16);
          const s16x8 hi = *reinterpret_cast<const s16x8 *>(v_lds[buf][0] + o);
          const s16x8 low = *reinterpret_cast<const s16x8 *>(v_lds[buf][1] + o);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f32x4 &to = SCALED ? sum[SCALED ? r : 0][j] : acc[r][j];
            to = D::mfma(fm[j], low, to);
            to = D::mfma(fm[j], hi, to);
          }
        }
      }
      if constexpr (SCALED) {
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const int p = -power[buf][16 * r + fr];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[r][j][e] += __builtin_amdgcn_ldexpf(sum[r][j][e], p);
        }
      }
    }
    float *part = sd.part + (int64_t)(a + blockIdx.y) * g.rank * sd.width4;
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + wave * 64 + 16 * j + 4 * fq, row = 16 * r + fr;
        if (row < g.rank && c < sd.width4)
          *reinterpret_cast<f32x4 *>(part + (int64_t)row * sd.width4 + c) = acc[r][j];
      }
    __syncthreads();  // before the next adapter's stages
  }
#endif
}

// The chunks' sums added in their order: da [rank, in], rows of 8 columns a thread; db
// [out, rank], 8 of the rank a thread and the columns along the lanes.
struct JoinSide {
  const float *part;
  uint16_t *out;
  int64_t ld, stride;
  int32_t width, width4, blocks;
};
template <class D>
__global__ __launch_bounds__(256) void grad_join_kernel(const JoinSide da, const JoinSide db,
                                                        const int32_t *__restrict__ offsets,
                                                        int rank, int chunk) {
  const int a = blockIdx.y, begin = offsets[a], end = offsets[a + 1];
  const int k0 = begin / chunk, k1 = end > begin ? (end - 1) / chunk : k0 - 1;
  f32x8 v = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if ((int)blockIdx.x < da.blocks) {
    const int runs = (da.width + 7) / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int r = (int)(i / runs), c = (int)(i % runs) * 8;
    if (r >= rank) return;
    for (int k = k0; k <= k1; ++k) {
      const f32x8 p = load8_f32(da.part + ((int64_t)(a + k) * rank + r) * da.width4, c, da.width);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += p[e];
    }
    store8<D>(da.out + a * da.stride + r * da.ld, c, da.width, v);
  } else {
    const int64_t i = (int64_t)(blockIdx.x - da.blocks) * 256 + threadIdx.x;
    const int r = (int)(i / db.width) * 8, c = (int)(i % db.width);
    if (r >= rank) return;
    for (int k = k0; k <= k1; ++k) {
      const float *p = db.part + ((int64_t)(a + k) * rank + r) * db.width4 + c;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (r + e < rank) v[e] += p[(int64_t)e * db.width4];
    }
    store8<D>(db.out + a * db.stride + c * db.ld, r, rank, v);
  }
}

}  // namespace moe_adapter
