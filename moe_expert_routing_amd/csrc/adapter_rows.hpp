// adapter_rows.hpp - the kernels of the low-rank adapters beside the product: s = c_a
// x A_a^T (and u = c_a dy B_a, the same on a transposed copy of B), y of a few rows,
// the tokens in the order of their adapters, and the adapters' gradients.
#pragma once

#include "../../include/moe_adapter.h"
#include "adapter_expand.hpp"
#include "ffn_gemm.hpp"

namespace moe_adapter {

using namespace moe_ffn;

// acc[r][i] += rows of the operands a[0 .. NA - 1] times rows of x over k elements, for
// products whose operands have few rows: 16 RB rows of each a, 16 MT of x, each wave on
// its own range of k.
//
// What a compute unit can take in depends on how its lanes ask. Measured with
// one block alone, 672 KB of 14 KB rows from L2: 5.7 us contiguous, 11 with loads of 8
// rows x 128 bytes in the order of the lanes, 19.5 with 16 rows x 64 bytes, as MFMA
// fragments lie, or 8 x 128 in another order. So each wave stages blocks of 64 k in
// LDS of its own with loads of the second kind, NS blocks deep, and reads fragments
// there; there are no barriers. Lane l of a load takes row l >> 3 of eight and chunk (l &
// 7) ^ (l >> 3) of its line, which it writes at 16 l: reading 16 rows of one chunk
// then goes over all banks. Loads past k's end, or past the range, bring zeros.
// Rows that are not 16-byte aligned, or whose k is no multiple of 8, are read as fragments.
template <int MT, int RB, int NS>
struct Stream {
  static constexpr int PIECES = 2 * (MT + RB);      // loads of a block of 64 k
  static constexpr int BYTES = NS * PIECES * 1024;  // a wave's LDS
  static_assert(PIECES * (NS - 1) <= 63, "vmcnt range");
};
struct StreamRows {
  const uint16_t *p;  // first row, at the wave's first k
  int64_t ld;
  int rows;       // at least 1; rows past them repeat the last one
  uint64_t some;  // not 0: the rows are those whose bits are set, no more than 16

  __device__ __forceinline__ int64_t at(int row) const {  // elements from p
    row = min(row, rows - 1);
    if (some) {
      int b = 0;
      uint64_t left = some;
      for (int i = 0; i < 16 && left; ++i, left &= left - 1) b = i <= row ? __builtin_ctzll(left) : b;
      row = b;
    }
    return row * ld;
  }
};

template <class D, int NA, int RB, int MT, int NS, bool STAGED>
__device__ __forceinline__ void stream_products(f32x4 (&acc)[NA * RB][MT], const StreamRows (&a)[NA],
                                                const StreamRows &x, int k, uint8_t *lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int lane = threadIdx.x & 63, fr = lane & 15, fq = lane >> 4;
  if constexpr (STAGED) {
    constexpr int F = NA * RB;  // fragments of the a
    typedef Stream<MT, F, NS> S;
    const int chunk = (lane & 7) ^ (lane >> 3);
    uint32_t off[S::PIECES];  // bytes, below 2^31 (128 rows of MOE_FFN_MAX_LD)
    auto operand_of = [&](int q) MOE_INLINE -> const StreamRows & {
      return q < 2 * F ? a[q / (2 * RB) % NA] : x;
    };
#pragma unroll
    for (int q = 0; q < S::PIECES; ++q) {
      const StreamRows &s = operand_of(q);
      const int row = (q < 2 * F ? q % (2 * RB) : q - 2 * F) * 8 + (lane >> 3);
      off[q] = (uint32_t)(s.at(row) + chunk * 8) * 2;
    }
    const int blocks = (k + 63) / 64;
    auto issue = [&](int s) MOE_INLINE {
      const bool past = s * 64 + chunk * 8 >= k;
#pragma unroll
      for (int q = 0; q < S::PIECES; ++q)
        lds_piece<true>(reinterpret_cast<const uint8_t *>(operand_of(q).p + s * 64),
                        past ? PAST : off[q], lds + (s % NS * S::PIECES + q) * 1024);
    };
#pragma unroll
    for (int s = 0; s < NS; ++s) issue(s);
#pragma unroll 1
    for (int s = 0; s < blocks; ++s) {
      wait_vmcnt_imm<S::PIECES *(NS - 1)>();
      const uint8_t *from = lds + s % NS * S::PIECES * 1024;
      s16x8 f[2][F + MT];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int q = 0; q < F + MT; ++q)
          f[ks][q] = *reinterpret_cast<const s16x8 *>(from + q * 2048 + fr * 128 +
                                                      (((ks * 4 + fq) ^ (fr & 7)) * 16));
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before it is filled again
      issue(s + NS);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int r = 0; r < F; ++r)
#pragma unroll
          for (int i = 0; i < MT; ++i) acc[r][i] = D::mfma(f[ks][r], f[ks][F + i], acc[r][i]);
    }
    wait_vmcnt_imm<0>();  // the zeros still on their way
  } else {
    const uint16_t *ar[NA * RB], *xr[MT];
#pragma unroll
    for (int r = 0; r < NA * RB; ++r)
      ar[r] = a[r / RB].p + a[r / RB].at(16 * (r % RB) + fr) + fq * 8;
#pragma unroll
    for (int i = 0; i < MT; ++i) xr[i] = x.p + x.at(16 * i + fr) + fq * 8;
    int s = 0;
#pragma unroll 4
    for (; s + 32 <= k; s += 32) {
      s16x8 fa[NA * RB];
#pragma unroll
      for (int r = 0; r < NA * RB; ++r) fa[r] = *reinterpret_cast<const s16x8_any *>(ar[r] + s);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const s16x8 fx = *reinterpret_cast<const s16x8_any *>(xr[i] + s);
#pragma unroll
        for (int r = 0; r < NA * RB; ++r) acc[r][i] = D::mfma(fa[r], fx, acc[r][i]);
      }
    }
    if (s < k) {
      const int left = k - s - fq * 8;
      s16x8 fa[NA * RB];
#pragma unroll
      for (int r = 0; r < NA * RB; ++r) fa[r] = load8_raw(ar[r] + s, 0, left);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const s16x8 fx = load8_raw(xr[i] + s, 0, left);
#pragma unroll
        for (int r = 0; r < NA * RB; ++r) acc[r][i] = D::mfma(fa[r], fx, acc[r][i]);
      }
    }
  }
#endif
}

// The waves' sums of a block, [WAVES][16 MT rows][16 RB + 4] in `part`.
template <int WAVES, int RB, int MT>
struct Part {
  static constexpr int LD = 16 * RB + 4, BYTES = WAVES * 16 * MT * LD * 4;
  template <int F>
  static __device__ __forceinline__ void put(float *part, int wave, const f32x4 (&acc)[F][MT], int first) {
    const int lane = threadIdx.x & 63, fr = lane & 15, fq = lane >> 4;
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        *reinterpret_cast<f32x4 *>(part + (wave * 16 * MT + 16 * i + fr) * LD + 16 * r + 4 * fq) = acc[first + r][i];
  }
  // of row t and column r, in the order of the waves
  static __device__ __forceinline__ float sum(const float *part, int t, int r) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += part[(w * 16 * MT + t) * LD + r];
    return v;
  }
};
template <int RB, int MT>
__device__ __forceinline__ void clear(f32x4 (&acc)[RB][MT]) {
#pragma unroll
  for (int r = 0; r < RB; ++r)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
}
constexpr int most(int a, int b) { return a > b ? a : b; }

// ------------------------------------------------------------ s = c_a x A_a^T

struct ShrinkArgs {
  const uint16_t *x, *a;  // a [rank, K] of each adapter
  int64_t ldx, lda, stride;
  const int32_t *ids;
  const float *scale;  // NULL: 1
  float *s;            // [M, rank], rows lds elements apart
  int32_t M, K, rank, n, lds;
  int32_t turns;       // blocks for the same rows
  int64_t block0;      // number of the launch's first block
};

// A block takes 16 MT rows, its waves share K and their sums meet in LDS. For each
// adapter among the rows the block goes through K once, or with NS2 for two of them
// at a time (that many stages then): requests lie together, so a prompt's rows have one
// or two, and with one block to a compute unit those that went through K twice took as
// long again as all others (8192 rows of 7168, 16 requests, rank 16: 33 us, now 28-31). A
// decode batch's rows may have 16, which the blocks of `turns` rounds over the rows share.
// (The rounds follow each other: with the blocks of the same rows side by side every second
// one ends at once, and as they go to the XCDs in turn, half of these stood idle: 66 us.)
//
// Bound by reading x: 8192 rows of 7168 with one adapter of rank 16 20 us (6 TB/s, part of x in
// the last cache), of rank 64 26. Rows with three and more adapters take a second way through
// K and are what the 16 requests pay for; each XCD with rows side by side, so that its L2
// holds few adapters, gained nothing (217 and 218 us with the product; 32768 rows 963 and
// 950), nor did one more block of x on its way in the pairs.
template <class D, int MT, int RB, int WAVES, int NS, int NS2, bool STAGED>
__global__ __launch_bounds__(64 * WAVES) void shrink_kernel(const ShrinkArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int ROWS = 16 * MT, NA = NS2 ? 2 : 1;
  constexpr int RING = STAGED ? most(Stream<MT, RB, NS>::BYTES, NS2 ? Stream<MT, 2 * RB, NS2 ? NS2 : 1>::BYTES : 0) : 0;
  typedef Part<WAVES, RB, MT> P;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[most(WAVES * RING, NA * P::BYTES)];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t block = (uint32_t)(blockIdx.x + g.block0);
  const uint32_t row_blocks = (g.M + ROWS - 1) / ROWS;
  const int row0 = block % row_blocks * ROWS, my_turn = block / row_blocks;
  int id = lane < ROWS && row0 + lane < g.M ? g.ids[row0 + lane] : -1;
  if ((uint32_t)id >= (uint32_t)g.n) id = -1;
  const uint64_t with = __ballot(id >= 0);
  // rows without an adapter
  if (my_turn == 0 && __popcll(with) < ROWS)
    for (int o = threadIdx.x; o < ROWS * g.rank; o += 64 * WAVES) {
      const int r = o / g.rank;
      if (row0 + r < g.M && !(with >> r & 1)) g.s[(int64_t)(row0 + r) * g.lds + o % g.rank] = 0.f;
    }
  const int per = ((g.K + 63) / 64 + WAVES - 1) / WAVES * 64;
  const int k0 = min(g.K, wave * per), k = min(g.K - k0, per);
  const StreamRows x = {g.x + row0 * g.ldx + k0, g.ldx, g.M - row0, 0};
  uint64_t todo = with;
  auto next = [&](uint64_t &mine) MOE_INLINE {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    mine = __ballot(id == a);
    todo &= ~mine;
    return a;
  };
  auto rows_of = [&](int a) MOE_INLINE {
    return StreamRows{g.a + a * g.stride + k0, g.lda, g.rank, 0};
  };
  auto write = [&](int a, uint64_t mine, const float *part) MOE_INLINE {
    const float c = g.scale ? g.scale[a] : 1.f;
    for (int o = threadIdx.x; o < ROWS * 16 * RB; o += 64 * WAVES) {
      const int t = o / (16 * RB), r = o % (16 * RB);
      if ((mine >> t & 1) && r < g.rank)
        g.s[(int64_t)(row0 + t) * g.lds + r] = P::sum(part, t, r) * c;
    }
  };
  float *part = reinterpret_cast<float *>(lds), *part1 = part + P::BYTES / 4;
  for (int turn = 0; todo; ++turn) {
    uint64_t mine, mine1 = 0;
    const int a = next(mine), a1 = NS2 && todo ? next(mine1) : -1;
    if (turn % g.turns != my_turn) continue;
    if (a1 >= 0) {
      f32x4 acc[NA * RB][MT];
      clear(acc);
      const StreamRows rows[2] = {rows_of(a), rows_of(a1)};
      if constexpr (NS2 > 0)
        stream_products<D, 2, RB, MT, NS2, STAGED>(acc, rows, x, k, lds + wave * RING);
      __syncthreads();  // the waves' staging memory holds the sums now
      P::put(part, wave, acc, 0);
      if constexpr (NS2 > 0) P::put(part1, wave, acc, RB);
      __syncthreads();
      write(a, mine, part);
      write(a1, mine1, part1);
    } else {
      f32x4 acc[RB][MT];
      clear(acc);
      const StreamRows rows[1] = {rows_of(a)};
      stream_products<D, 1, RB, MT, NS, STAGED>(acc, rows, x, k, lds + wave * RING);
      __syncthreads();
      P::put(part, wave, acc, 0);
      __syncthreads();
      write(a, mine, part);
    }
    __syncthreads();  // before the next adapter's rows
  }
#endif
}

// ----------------------------------------------------- y of few rows, two launches

// For a decode batch, bound by reading W and the adapters among its tokens once.
// First launch: x times the rows of W and of each such A_a together, so that reading
// the adapters costs no time of its own; k is split over the waves of `splits` blocks,
// each of which leaves fp32 sums. Second launch: the sums added in their order, s B_a^T in
// fp32, bias and residual, one rounding.
// Tokens go in groups of 64, each with blocks of its own.
// 16 tokens, 7168 -> 2048, an adapter of rank 16 each: 10.5 us (33 MB, 3.2 TB/s with some 4 us of
// launch and first loads in it) and 4.
constexpr int FEW_GROUP = 64;
struct FewArgs {
  const uint16_t *x, *w, *a, *b, *bias, *res;
  int64_t ldx, ldw, lda, a_stride, ldb, b_stride, ldr, ldy;
  const int32_t *ids;
  const float *scale;
  float *part_y, *part_s;  // [splits][M][N], [splits][M][rank]
  float *s;                // [M, rank] or NULL
  uint16_t *y;
  int32_t M, N, K, rank, n, splits, per;  // per: k of a wave, a multiple of 64
  int32_t w_tiles, rank_tiles;
};
constexpr int FEW_WAVES = 4;

template <class D, int MT, int RB, int NS, bool STAGED>
__global__ __launch_bounds__(64 * FEW_WAVES) void few_stream_kernel(const FewArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int TILE = 16 * RB, ARB = RB < 2 ? 1 : 2, ATILE = 16 * ARB;  // rows of W, and of an A
  constexpr int RING = STAGED ? most(Stream<MT, RB, NS>::BYTES, Stream<1, ARB, NS>::BYTES) : 0;
  typedef Part<FEW_WAVES, RB, MT> P;
  typedef Part<FEW_WAVES, ARB, 1> PA;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[most(FEW_WAVES * RING, most(P::BYTES, PA::BYTES))];
  float *part = reinterpret_cast<float *>(lds);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k0 = min(g.K, ((int)blockIdx.y * FEW_WAVES + wave) * g.per), k = min(g.K - k0, g.per);
  const int t0 = blockIdx.z * FEW_GROUP, M = min(g.M - t0, FEW_GROUP);
  const uint16_t *x = g.x + t0 * g.ldx + k0;
  int tile = blockIdx.x;
  if (tile < g.w_tiles) {
    const int r0 = tile * TILE;
    f32x4 acc[RB][MT];
    clear(acc);
    const StreamRows w[1] = {{g.w + r0 * g.ldw + k0, g.ldw, g.N - r0, 0}};
    stream_products<D, 1, RB, MT, NS, STAGED>(acc, w, {x, g.ldx, M, 0}, k, lds + wave * RING);
    __syncthreads();
    P::put(part, wave, acc, 0);
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * MT * TILE; o += 64 * FEW_WAVES) {
      const int t = o / TILE, r = o % TILE;
      if (t < M && r0 + r < g.N)
        g.part_y[((int64_t)blockIdx.y * g.M + t0 + t) * g.N + r0 + r] = P::sum(part, t, r);
    }
    return;
  }
  // of the slot-th adapter among the tokens: its own tokens, 16 at a time
  const int slot = (tile - g.w_tiles) / g.rank_tiles, r0 = (tile - g.w_tiles) % g.rank_tiles * ATILE;
  int id = lane < M ? g.ids[t0 + lane] : -1;
  if ((uint32_t)id >= (uint32_t)g.n) id = -1;
  uint64_t todo = __ballot(id >= 0), mine = 0;
  int a = 0;
  for (int i = 0; todo && i <= slot; ++i) {
    a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    mine = __ballot(id == a);
    if (i < slot) todo &= ~mine;
  }
  if (!todo) return;
  const StreamRows rows[1] = {{g.a + a * g.a_stride + r0 * g.lda + k0, g.lda, g.rank - r0, 0}};
  while (mine) {
    uint64_t some = 0;
    for (int i = 0; i < 16 && mine; ++i, mine &= mine - 1) some |= mine & -mine;
    f32x4 acc[ARB][1];
    clear(acc);
    stream_products<D, 1, ARB, 1, NS, STAGED>(acc, rows, {x, g.ldx, (int)__popcll(some), some}, k,
                                              lds + wave * RING);
    __syncthreads();
    PA::put(part, wave, acc, 0);
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * ATILE; o += 64 * FEW_WAVES) {
      const int i = o / ATILE, r = o % ATILE;
      if (i >= (int)__popcll(some) || r0 + r >= g.rank) continue;
      uint64_t left = some;
      for (int q = 0; q < i; ++q) left &= left - 1;
      g.part_s[((int64_t)blockIdx.y * g.M + t0 + __builtin_ctzll(left)) * g.rank + r0 + r] = PA::sum(part, i, r);
    }
    __syncthreads();
  }
#endif
}

// A column of one token's y a thread.
template <class D>
__global__ __launch_bounds__(256) void few_finish_kernel(const FewArgs g) {
  __shared__ __attribute__((aligned(16))) float s[MOE_ADAPTER_MAX_RANK];
  const int t = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x, at = min(n, g.N - 1);
  const int id = g.ids[t];
  const bool with = (uint32_t)id < (uint32_t)g.n;
  float y = 0.f;
  for (int k = 0; k < g.splits; ++k) y += g.part_y[((int64_t)k * g.M + t) * g.N + at];
  if ((int)threadIdx.x < MOE_ADAPTER_MAX_RANK) {
    float v = 0.f;
    if (with && (int)threadIdx.x < g.rank) {
      for (int k = 0; k < g.splits; ++k) v += g.part_s[((int64_t)k * g.M + t) * g.rank + threadIdx.x];
      v *= g.scale ? g.scale[id] : 1.f;
    }
    s[threadIdx.x] = v;
    if (g.s && blockIdx.x == 0 && (int)threadIdx.x < g.rank) g.s[(int64_t)t * g.rank + threadIdx.x] = v;
  }
  __syncthreads();
  if (with) {
    const uint16_t *b = g.b + id * g.b_stride + at * g.ldb;
    float d = 0.f;
#pragma unroll 4
    for (int k = 0; k < g.rank; k += 8) {
      const f32x8 w = unpack8<D>(load8_raw(b, k, g.rank));
      const f32x8 v = *reinterpret_cast<const f32x8_any *>(s + k);
#pragma unroll
      for (int e = 0; e < 8; ++e) d = fmaf(v[e], w[e], d);
    }
    y += d;
  }
  if (n >= g.N) return;
  if (g.bias) y += to_f<D>(g.bias[n]);
  if (g.res) y += to_f<D>(g.res[t * g.ldr + n]);
  g.y[t * g.ldy + n] = from_f<D>(y);
}

// ------------------- the tokens of each adapter, in order, and transposed copies

constexpr int PREP_THREADS = 1024, PREP_WAVES = PREP_THREADS / 64;

// at [in, rank8] = A transposed of each adapter, for dx's product, whose operand needs
// the rank along its rows; bt [rank, out8] = B transposed, for u's. NULL: not needed.
// perm: the tokens with an adapter, by adapter and then by number; offsets[a]: where
// those of adapter a begin. s4: s with rows of whole 16 bytes (NULL: not needed). zeros:
// 16 bytes that the gradients' loads take for what is not there.
// Where there are more adapters than tokens, the copies are made for the tokens' adapters
// alone, that of the first token t with each of them at place t: own[t] is the place of token
// t's adapter (-1: none), own_scale[place] its scale. Else the places are the adapters.
struct PrepArgs {
  const int32_t *ids;
  int32_t *offsets, *perm;
  const uint16_t *a, *b;
  int64_t lda, a_stride, ldb, b_stride;
  uint16_t *at, *bt;
  const float *s, *scale;
  float *s4, *zeros, *own_scale;
  int32_t *own;
  int32_t T, n, in, out, rank, rank4, rank8, out8;
  int64_t block0, copy_block;  // numbers of the launch's first block, and of the first that copies s
};

// A block for each adapter counts the ids below its own and its own, a wave 64 tokens
// at a time by ballots, and then writes its tokens: two reads of the ids a block, no
// order that changes. The blocks after those make the copies, 8 of the rank a thread.
// Bound by the two reads' latency: 8192 tokens, 8 adapters, 2048 -> 4096 with rank 64 6-8 us in
// one launch, 512 tokens and 4 adapters 5.
template <bool OWN>
__global__ __launch_bounds__(PREP_THREADS) void prep_kernel(const PrepArgs g) {
  __shared__ int sames[PREP_WAVES], lesses[PREP_WAVES];
  const int64_t block = blockIdx.x + g.block0;
  if (block < g.n) {
    const int a = (int)block, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t each = ((int64_t)(g.T + PREP_THREADS - 1) / PREP_THREADS) * 64;
    const int lo = (int)min(wave * each, (int64_t)g.T), hi = (int)min(lo + each, (int64_t)g.T);
    int less = 0, same = 0;
    constexpr int AT_ONCE = 8;  // groups of 64 whose ids are loaded together
    int ids[AT_ONCE];
    auto load_ids = [&](int i) MOE_INLINE {
#pragma unroll
      for (int q = 0; q < AT_ONCE; ++q) {
        const int t = i + q * 64 + lane;
        ids[q] = g.ids[min(t, hi - 1)];
        if (t >= hi) ids[q] = -1;
      }
    };
    for (int i = lo; i < hi; i += 64 * AT_ONCE) {
      load_ids(i);
#pragma unroll
      for (int q = 0; q < AT_ONCE; ++q) {
        less += __popcll(__ballot(ids[q] >= 0 && ids[q] < a));
        same += __popcll(__ballot(ids[q] == a));
      }
    }
    if (lane == 0) sames[wave] = same, lesses[wave] = less;
    __syncthreads();
    int first = 0, before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < PREP_WAVES; ++w) {
      first += lesses[w];
      before += w < wave ? sames[w] : 0;
      total += sames[w];
    }
    if (a == 0 && threadIdx.x < 4 && g.zeros) g.zeros[threadIdx.x] = 0.f;
    if (threadIdx.x == 0) {
      g.offsets[a] = first;
      if (a == g.n - 1) g.offsets[g.n] = first + total;
    }
    int at = first + before;
    for (int i = lo; i < hi; i += 64 * AT_ONCE) {
      if (hi - lo > 64 * AT_ONCE) load_ids(i);
#pragma unroll
      for (int q = 0; q < AT_ONCE; ++q) {
        const uint64_t all = __ballot(ids[q] == a);
        if (ids[q] == a) g.perm[at + __popcll(all & ((1ull << lane) - 1))] = i + q * 64 + lane;
        at += __popcll(all);
      }
    }
    return;
  }
  if (block >= g.copy_block) {
    const int64_t i = (block - g.copy_block) * PREP_THREADS + threadIdx.x;
    const int64_t t = i / g.rank4;
    const int r = (int)(i % g.rank4);
    if (t < g.T) g.s4[i] = r < g.rank ? g.s[t * g.rank + r] : 0.f;
    return;
  }
  const int runs = g.rank8 / 8, a_items = g.at ? g.in * runs : 0, items = a_items + g.out * runs;
  const int blocks = (items + PREP_THREADS - 1) / PREP_THREADS;
  const int place = (int)((block - g.n) / blocks);
  int i = (int)((block - g.n) % blocks) * PREP_THREADS + threadIdx.x;
  int a = place;
  if constexpr (OWN) {
    a = g.ids[place];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int first = place;
    for (int t = wave * 64; t < first; t += PREP_THREADS) {
      const uint64_t all = __ballot(t + lane < place && g.ids[t + lane] == a);
      if (all) first = t + __builtin_ctzll(all);
    }
    if (lane == 0) sames[wave] = first;
    __syncthreads();
    for (int w = 0; w < PREP_WAVES; ++w) first = min(first, sames[w]);
    if ((uint32_t)a >= (uint32_t)g.n) first = -1;
    if (i == 0) g.own[place] = first;
    if (i == 0 && first == place && g.scale) g.own_scale[place] = g.scale[a];
    if (first != place) return;
  }
  if (i < a_items) {
    const int c = i / runs, r = i % runs * 8;  // a row's 16-byte runs side by side
    const uint16_t *src = g.a + a * g.a_stride + c;
    s16x8 w = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < 8; ++v)
      if (r + v < g.rank) w[v] = (short)src[(r + v) * g.lda];
    *reinterpret_cast<s16x8 *>(g.at + ((int64_t)place * g.in + c) * g.rank8 + r) = w;
  } else if (i < items) {
    i -= a_items;
    const int c = i / runs, r = i % runs * 8;
    const s16x8 w = load8_raw(g.b + a * g.b_stride + c * g.ldb, r, g.rank);
    uint16_t *dst = g.bt + (int64_t)place * g.rank * g.out8 + c;
#pragma unroll
    for (int v = 0; v < 8; ++v)
      if (r + v < g.rank) dst[(int64_t)(r + v) * g.out8] = (uint16_t)w[v];
  }
}

// ------------------------------------------------------- the adapters' gradients

// sum over the tokens t of adapter a of v[t, r] m[t, c]: dA with v = u and m = x, dB
// (transposed) with v = s and m = dy.
struct GradSide {
  const uint16_t *m;  // rows 16-byte aligned
  int64_t ld;
  const float *v;     // [T, rank], rows ldv elements (whole 16 bytes) apart
  float *part;        // [slots][rank][width4]
  uint16_t *out;      // dA [rank, width] or dB [width, rank] of each adapter
  int64_t ld_out, stride;
  int32_t width, width4, tiles;
};
struct GradArgs {
  GradSide side[2];
  const int32_t *offsets, *perm;
  const float *zeros;  // 16 bytes
  int32_t rank, ldv, n, chunk;  // chunk: sorted tokens of a block
};

// 16 bytes a lane, each from its own address, to dst + 16 lane in LDS. As in lds_piece the
// compiler is not told of the write: the kernel's own waits order it.
__device__ __forceinline__ void lds_gather(const void *from, uint8_t *dst) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t to = (uint32_t)(uintptr_t)(lds_ptr_t)dst;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from)
               : "m0");
#endif
}

typedef s16x4 s16x4_any __attribute__((aligned(2)));
constexpr int GRAD_COLS = 256, GRAD_K = 32, GRAD_WAVES = 4, GRAD_WINDOW = 1024;

// A block takes 256 columns of m and `chunk` tokens of the sorted order, and adds
// up each adapter among them apart: the part of adapter a in chunk k goes to slot
// a + k, of which there is one for each pair that meets.
// WHOLE, for more adapters than chunks: one whose tokens all lie in the chunk is written as it
// is, and of the others a chunk has two at most, the one that goes on from the chunk before
// (slot 2 k of chunk k) and the one that begins in it and goes on behind it (slot 2 k + 1).
// So the parts' memory does not grow with the adapters (4096 of rank 64, 7168 + 7168 columns: 15
// GB otherwise). A whole backward pass of 4096 tokens of 256 adapters, rank 16, 4096 + 4096
// columns takes 397 us, by pairs 437; 8192 tokens of 1024, rank 32, 2048 + 2048 columns 831 and
// 1017. With few adapters the pairs' kernel, which keeps less through the products, is the
// faster (8192 tokens of 8, as below: gradients and join 50 us, WHOLE 52).
// 32 tokens at a time go through LDS, NS stages deep: m as it lies, read through the transposing
// LDS load, and v in fp32, which each wave takes into three parts of the type in the
// registers of its fragments, so that none of its 24 bits is lost where tokens cancel. In
// fp16, whose range v may pass, the 32 values of a column of v are taken at a power
// of two of their own. What is not there (tokens past the end, columns past the width or the
// rank) is loaded from a few zeros, so that nothing a buffer happens to hold counts.
// 8192 tokens, 2048 + 4096 columns, rank 64, 8 adapters: 39 us for 101 MB in and 35 MB of
// sums out (3.5 TB/s; with two parts of v 35; with plain loads 62 where this took 36, with a
// branch for each missing row 54); rank 16 and 7168 + 2048 columns 33 us. 256 columns, so that rows come in whole 512 bytes; 2 blocks of a compute
// unit cover each other's waits (6 stages in one: slower).
template <class D, int RB, int NS, bool WHOLE>
__global__ __launch_bounds__(64 * GRAD_WAVES, RB <= 4 ? 2 : 1) void grad_kernel(const GradArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool SCALED = D::MAX_EXPONENT < 127;
  constexpr int ROW = GRAD_COLS * 2, M_BYTES = GRAD_K * ROW;
  constexpr int V_CHUNKS = 4 * RB, V_ROW = V_CHUNKS * 16, V_BYTES = GRAD_K * V_ROW;
  constexpr int STAGE = M_BYTES + V_BYTES;
  constexpr int M_LOADS = M_BYTES / 1024 / GRAD_WAVES;                          // of a wave
  constexpr int V_PIECES = V_BYTES / 1024, V_LOADS = (V_PIECES + GRAD_WAVES - 1) / GRAD_WAVES;
  constexpr int LOADS_MIN = M_LOADS + V_PIECES / GRAD_WAVES;
  // waves side by side over the rank, each with RW 16s of it and J 16s of the columns: a
  // wave converts what it multiplies
  constexpr int WR = RB < 4 ? 1 : RB / 2, WC = GRAD_WAVES / WR, RW = RB / WR, J = 16 / WC;
  static_assert((RB <= 4 ? 2 : 1) * (NS * STAGE + GRAD_WINDOW * 4) <= 160 * 1024, "blocks of a compute unit");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NS * STAGE];
  __shared__ int token_of[GRAD_WINDOW];
  const int lane = threadIdx.x & 63, fr = lane & 15, fq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool second = (int)blockIdx.x >= g.side[0].tiles;
  const GradSide sd = g.side[second];
  const uint64_t zeros = (uint64_t)g.zeros;
  const int c0 = (blockIdx.x - (second ? g.side[0].tiles : 0)) * GRAD_COLS;
  const int total = g.offsets[g.n];
  const int64_t first64 = (int64_t)blockIdx.y * g.chunk;
  if (first64 >= total) return;
  const int first = (int)first64, last = (int)min(first64 + g.chunk, (int64_t)total);

  // the adapter of the chunk's first token: the last one that begins at or before it
  int lo = 0, hi = g.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.offsets[mid] <= first) lo = mid; else hi = mid - 1;
  }

  // where this lane's pieces lie: m's are 2 rows of 32 chunks, v's 64 chunks of its rows;
  // past the width or the rank the zeros, whatever the token
  int row[M_LOADS + V_LOADS];
  uint64_t at[M_LOADS + V_LOADS];
  uint32_t ld[M_LOADS + V_LOADS];  // bytes
#pragma unroll
  for (int q = 0; q < M_LOADS; ++q) {
    const int k = (q * GRAD_WAVES + wave) * 2 + (lane >> 5);
    const int c = c0 + ((lane & 31) ^ swz<GRAD_COLS>(k)) * 8;
    row[q] = k;
    at[q] = c < sd.width ? (uint64_t)(sd.m + c) : zeros;
    ld[q] = c < sd.width ? (uint32_t)(sd.ld * 2) : 0;
  }
#pragma unroll
  for (int q = 0; q < V_LOADS; ++q) {
    const int i = (q * GRAD_WAVES + wave) * 64 + lane, c = i % V_CHUNKS * 4;
    row[M_LOADS + q] = i / V_CHUNKS;
    at[M_LOADS + q] = c < g.rank ? (uint64_t)(sd.v + c) : zeros;
    ld[M_LOADS + q] = c < g.rank ? (uint32_t)(g.ldv * 4) : 0;
  }
  const int my_col = wave % WC * J * 16, my_rank = wave / WC * RW * 16;
  // transposed reads: a lane's k-row and, in chunk c of it, the place of column 16 j
  const int tk = fq * 8 + (fr >> 2);
  auto tr = [&](int j) MOE_INLINE {
    const int c = my_col / 8 + 2 * j + ((fr & 3) >> 1);
    return (uint32_t)(tk * ROW + (c ^ swz<GRAD_COLS>(tk)) * 16 + (fr & 1) * 8);
  };

  for (int a = lo; a < g.n && g.offsets[a] < last; ++a) {
    const int begin = max(g.offsets[a], first), end = min(g.offsets[a + 1], last);
    if (begin >= end) continue;
    f32x4 acc[RW][J];
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int j = 0; j < J; ++j) acc[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int from = begin; from < end; from += GRAD_WINDOW) {
      const int count = min(end - from, GRAD_WINDOW), stages = (count + GRAD_K - 1) / GRAD_K;
      __syncthreads();  // everybody is done with the window before
      for (int i = threadIdx.x; i < count; i += 64 * GRAD_WAVES) token_of[i] = g.perm[from + i];
      __syncthreads();
      auto issue = [&](int s) MOE_INLINE {
        uint8_t *to = lds + s % NS * STAGE;
        int token[M_LOADS + V_LOADS];
#pragma unroll
        for (int q = 0; q < M_LOADS + V_LOADS; ++q)
          token[q] = token_of[min(s * GRAD_K + row[q], count - 1)];
#pragma unroll
        for (int q = 0; q < M_LOADS + V_LOADS; ++q) {
          const int piece = (q < M_LOADS ? q : q - M_LOADS) * GRAD_WAVES + wave;
          if (V_PIECES % GRAD_WAVES != 0 && q >= M_LOADS && piece >= V_PIECES) continue;
          const uint64_t p = at[q] + (uint64_t)(uint32_t)token[q] * ld[q];
          lds_gather(reinterpret_cast<const void *>(s * GRAD_K + row[q] < count ? p : zeros),
                     to + (q < M_LOADS ? 0 : M_BYTES) + piece * 1024);
        }
      };
#pragma unroll
      for (int s = 0; s < NS - 1; ++s)
        if (s < stages) issue(s);
#pragma unroll 1
      for (int s = 0; s < stages; ++s) {
        if (s + NS - 1 <= stages)
          wait_vmcnt_imm<LOADS_MIN *(NS - 2)>();
        else
          wait_vmcnt_imm<0>();
        // every wave's loads of this stage are here, and its reads of the last one done
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (s + NS - 1 < stages) issue(s + NS - 1);
        const uint8_t *m_lds = lds + s % NS * STAGE, *v_lds = m_lds + M_BYTES;
        s16x8 fm[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const uint8_t *p = m_lds + tr(j);
          const s16x4 x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr_t)p);
          const s16x4 x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr_t)(p + 4 * ROW));
          fm[j] = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
        }
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          f32x8 v;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = *reinterpret_cast<const float *>(v_lds + (fq * 8 + e) * V_ROW + (my_rank + 16 * r + fr) * 4);
          int power = 0;
          if constexpr (SCALED) {
            float most = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(v[e]));
            most = fmaxf(most, __shfl_xor(most, 16));
            most = fmaxf(most, __shfl_xor(most, 32));
            power = exponent_for(most);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __builtin_amdgcn_ldexpf(v[e], power);
          }
          s16x8 piece[3];
          three_parts<D>(v, piece);
#pragma unroll
          for (int j = 0; j < J; ++j) {
            f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 2; q >= 0; --q) {
              if constexpr (SCALED)
                t = D::mfma(fm[j], piece[q], t);
              else
                acc[r][j] = D::mfma(fm[j], piece[q], acc[r][j]);
            }
            if constexpr (SCALED)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[r][j][e] += __builtin_amdgcn_ldexpf(t[e], -power);
          }
        }
      }
    }
    const int c = c0 + my_col + 4 * fq, row = my_rank + fr;
    const bool before = g.offsets[a] < first, behind = g.offsets[a + 1] > last;
    if (!WHOLE || before || behind) {
      const uint32_t slot = WHOLE ? 2 * blockIdx.y + (before ? 0 : 1) : a + blockIdx.y;
      float *part = sd.part + ((int64_t)slot * g.rank + row) * sd.width4 + c;
#pragma unroll
      for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (row + 16 * r < g.rank && c + 16 * j < sd.width4)
            *reinterpret_cast<f32x4 *>(part + (int64_t)16 * r * sd.width4 + 16 * j) = acc[r][j];
    } else {
      // elements from one rank, and from one column, to the next; the compiler is not
      // to keep the addresses and conditions of all of them through the products (which spilled)
      int64_t by_rank = second ? 1 : sd.ld_out, by_col = second ? sd.ld_out : 1;
      int ranks = g.rank, cols = sd.width;
      asm volatile("" : "+s"(by_rank), "+s"(by_col), "+s"(ranks), "+s"(cols));
      uint16_t *out = sd.out + a * sd.stride + row * by_rank + c * by_col;
#pragma unroll
      for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int left = row + 16 * r < ranks ? cols - (c + 16 * j) : 0;
          uint16_t *to = out + 16 * (r * by_rank + j * by_col);
          const s16x4 v = __builtin_bit_cast(s16x4, __builtin_convertvector(acc[r][j], typename D::v4));
          if (!second && left >= 4) {
            *reinterpret_cast<s16x4_any *>(to) = v;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (e < left) to[e * by_col] = (uint16_t)v[e];
          }
        }
    }
  }
#endif
}

// The chunks' sums added in their order, and zeros for the adapters without tokens; WHOLE:
// but for those that grad_kernel has written: da [rank, in], rows of 8 columns a thread; db [out, rank], 8 of
// the rank a thread and the columns along the lanes. Bound by reading the
// sums, which are still in the caches: 35 MB in 9 us (one chunk's load after the other: 20).
struct JoinSide {
  const float *part;
  uint16_t *out;
  int64_t ld, stride;
  int32_t width, width4, blocks;
};
template <class D, bool WHOLE>
__global__ __launch_bounds__(256) void grad_join_kernel(const JoinSide da, const JoinSide db,
                                                        const int32_t *__restrict__ offsets,
                                                        int rank, int chunk) {
  const int a = blockIdx.y, begin = offsets[a], end = offsets[a + 1];
  const int k0 = begin / chunk, k1 = end > begin ? (end - 1) / chunk : k0 - 1;
  if (WHOLE && k0 == k1) return;
  auto slot = [&](int k) MOE_INLINE { return (int64_t)(WHOLE ? 2 * k + (k == k0) : a + k); };
  // four chunks' parts at a time, those past the last one without their value
  constexpr int AT_ONCE = 4;
  f32x8 v = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if ((int)blockIdx.x < da.blocks) {
    const int runs = (da.width + 7) / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int r = (int)(i / runs), c = (int)(i % runs) * 8;
    if (r >= rank) return;
    for (int k = k0; k <= k1; k += AT_ONCE) {
      f32x8 p[AT_ONCE];
#pragma unroll
      for (int q = 0; q < AT_ONCE; ++q)
        p[q] = load8_f32(da.part + (slot(min(k + q, k1)) * rank + r) * da.width4, c, da.width);
#pragma unroll
      for (int q = 0; q < AT_ONCE; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k + q <= k1 ? v[e] + p[q][e] : v[e];
    }
    store8<D>(da.out + a * da.stride + r * da.ld, c, da.width, v);
  } else {
    const int64_t i = (int64_t)(blockIdx.x - da.blocks) * 256 + threadIdx.x;
    const int r = (int)(i / db.width) * 8, c = (int)(i % db.width);
    if (r >= rank) return;
    for (int k = k0; k <= k1; k += AT_ONCE) {
      float p[AT_ONCE][8];
#pragma unroll
      for (int q = 0; q < AT_ONCE; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          p[q][e] = db.part[(slot(min(k + q, k1)) * rank + min(r + e, rank - 1)) * db.width4 + c];
#pragma unroll
      for (int q = 0; q < AT_ONCE; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k + q <= k1 ? v[e] + p[q][e] : v[e];
    }
    store8<D>(db.out + a * db.stride + c * db.ld, r, rank, v);
  }
}

}  // namespace moe_adapter
