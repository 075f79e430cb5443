// ffn_gemm.hpp - the tiled products of the feed-forward operators on the
// gfx950 matrix cores.
//
// One kernel template computes C[m, n] = sum over k of A(m, k) B(n, k) for
// four uses, which differ in how the operands lie in memory and in what the
// epilogue does:
//   GATED   A = x rows (gathered by token), B = Wg and Wu rows; epilogue
//           h = act(g) u, optionally g and u themselves
//   LINEAR  A = x rows, B = W rows; epilogue bias, activation, residual
//   DGRAD   A = dz rows, B(n, k) = W[k, n]; one or two segments of k
//           (gate, up) summed
//   WGRAD   A(m, k) = dz[k, m], B(n, k) = x[k, n] (gathered by token), k = the
//           rows of one expert
// An operand whose k is contiguous is staged as rows of 64 k (128 bytes, 8
// chunks of 16 bytes; chunk c of row r at position c ^ (r & 7), so that the 8
// rows that one pass of a fragment read touches hit 8 different bank quads).
// One whose m or n is contiguous is staged as 64 k-rows as they lie in memory
// and read through the transposing LDS load (4 k-rows x 16 columns per 16
// lanes); chunk c of k-row k sits at c ^ swz(k), which puts the 4 rows and the
// two 16-lane groups of a pass on different banks.
//
// Both operands go from global memory straight into LDS
// (global_load_lds_dwordx4). NS stage buffers: NS - 1 stages are in flight
// while one is consumed. The fragments of one MFMA k-step are read from LDS
// while the previous step's MFMAs run.
//
// The weights are the MFMA's first operand: a lane then holds 4 consecutive n
// of one row m, so the epilogue stores 8 bytes and the two projections of a
// gated block meet in the same lane (their rows are interleaved by 16).
#pragma once

#include <type_traits>

#include "ffn_types.hpp"

namespace moe_ffn {

typedef __attribute__((address_space(3))) void *lds_ptr_t;
typedef __attribute__((address_space(3))) s16x4 *lds_s16x4_ptr_t;
typedef __attribute__((address_space(1))) void *gbl_ptr_t;

constexpr int TK = 64;  // k per stage

// 16 bytes of zeros that out-of-range pieces are loaded from
__device__ const uint4 zero_piece = {0, 0, 0, 0};

template <int BM_, int BN_, int WM_, int WN_, int NS_, int BLOCKS_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int BLOCKS = BLOCKS_;  // blocks per compute unit
  static constexpr int WAVES_N = BN / WN, NW = (BM / WM) * WAVES_N;
  static constexpr int NTHREADS = 64 * NW;
  static constexpr int FM = WM / 16, FN = WN / 16;
  static constexpr int A_INSTR = BM / 8, B_INSTR = BN / 8;  // 1 KB loads per stage
  static constexpr int INSTR = A_INSTR + B_INSTR;
  static constexpr int LOADS = (INSTR + NW - 1) / NW;        // most of one wave
  static constexpr int LOADS_MIN = INSTR / NW;               // of every wave
  static constexpr int A_BYTES = BM * TK * 2, STAGE_BYTES = (BM + BN) * TK * 2;
  static_assert((NS - 2) * LOADS_MIN <= 63, "vmcnt range");
};

template <int N>
__device__ __forceinline__ void wait_vmcnt_imm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// s_waitcnt vmcnt(k * STEP) for a run-time k in [0, MAXK]
template <int STEP, int MAXK>
__device__ __forceinline__ void wait_vmcnt_steps(int k) {
  if constexpr (MAXK > 0) {
    if (k >= MAXK) {
      wait_vmcnt_imm<MAXK * STEP>();
      return;
    }
    wait_vmcnt_steps<STEP, MAXK - 1>(k);
  } else {
    wait_vmcnt_imm<0>();
  }
}

// Position of 16-byte chunk c in k-row k of an operand staged as it lies in
// memory, R columns wide.
template <int R>
__device__ __forceinline__ int swz(int k) {
  return R >= 128 ? ((k & 3) << 1) | (((k >> 3) & 1) << 3) : (k & 3) << 1;
}

// Tile of this block. The hardware sends block b to XCD b % 8: each XCD takes
// a contiguous run of tiles, and the run goes through the tiles in columns
// of 8 m-tiles, so that the tiles in flight on one XCD share operand rows in
// its L2.
__device__ __forceinline__ void tile_of_block(int b, int total, int m_tiles, int n_tiles, int &mt,
                                              int &nt) {
  constexpr int GROUP = 8;
  const int per = total / 8, rest = total % 8, x = b % 8;
  int t = x * per + min(x, rest) + b / 8;
  const int full = GROUP * n_tiles;
  const int g = t / full, first = g * GROUP, size = min(GROUP, m_tiles - first);
  t -= g * full;
  mt = first + t % size;
  nt = t / size;
}

template <class D>
__device__ __forceinline__ void store4(uint16_t *p, f32x4 v, int left, bool vec) {
  const s16x4 w = pack4<D>(v);
  if (vec && left >= 4) {
    *reinterpret_cast<s16x4 *>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = (uint16_t)w[i];
  }
}
template <class D>
__device__ __forceinline__ f32x4 load4(const uint16_t *p, int left, bool vec) {
  s16x4 w = {0, 0, 0, 0};
  if (vec && left >= 4) {
    w = *reinterpret_cast<const s16x4 *>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) w[i] = (short)p[i];
  }
  return unpack4<D>(w);
}
// whether 4 consecutive elements at a multiple-of-4 column are one aligned load
__device__ __forceinline__ bool vec4(const void *p, int64_t ld, int64_t stride = 0) {
  return (((uintptr_t)p & 7) | (uintptr_t)((ld | stride) & 3)) == 0;
}

template <class D, int MODE, class C>
__global__ __launch_bounds__(C::NTHREADS, (C::BLOCKS * C::NW + 3) / 4) void gemm_kernel(
    const GemmArgs g) {
  constexpr int BM = C::BM, BN = C::BN, NS = C::NS;
  constexpr bool A_TR = MODE == WGRAD, B_TR = MODE == DGRAD || MODE == WGRAD;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * C::STAGE_BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool grouped = g.r.num_experts > 0;

  int mt, nt, e = 0, seg0 = 0;
  int64_t k_row0 = 0;  // WGRAD: first row of the expert
  int K = g.K;
  if constexpr (MODE == WGRAD) {
    // one expert and projection after the other, all its tiles together
    const int per = g.m_tiles * g.n_tiles;
    const int chunk = blockIdx.x / per;
    e = chunk / g.segs;
    seg0 = chunk % g.segs;
    tile_of_block(blockIdx.x % per, per, g.m_tiles, g.n_tiles, mt, nt);
    if (grouped) {
      const int64_t p0 = g.r.padded_offsets[e], cnt = g.r.counts[e];
      k_row0 = min(max(p0, (int64_t)0), g.r.rows);
      K = (int)min(max(cnt, (int64_t)0), g.r.rows - k_row0);
    }
  } else {
    tile_of_block(blockIdx.x, gridDim.x, g.m_tiles, g.n_tiles, mt, nt);
  }
  const int m0 = mt * BM;
  const int n0 = nt * (MODE == GATED ? BN / 2 : BN);  // column of C

  if constexpr (MODE != WGRAD) {
    if (grouped) {
      e = g.r.m_indices[m0];
      if (e < 0 || e >= g.r.num_experts || g.a_rows == 0) {  // no entry here: zeros
        constexpr int W = MODE == GATED ? BN / 2 : BN;
        const int width = min(W, g.N - n0), height = min(BM, g.M - m0);
        for (int i = threadIdx.x; i < height * W; i += C::NTHREADS) {
          const int r = i / W, c = i % W;
          if (c < width) {
            g.c0[(int64_t)(m0 + r) * g.ldc0 + n0 + c] = 0;
            if (MODE <= LINEAR && g.pre) {
              g.pre[(int64_t)(m0 + r) * g.ldp + n0 + c] = 0;
              if (MODE == GATED) g.pre[(int64_t)(m0 + r) * g.ldp + g.N + n0 + c] = 0;
            }
          }
        }
        return;
      }
    }
  }
  const uint16_t *b0 = g.b0, *b1 = g.b1;
  if (MODE != WGRAD) {
    b0 += e * g.b_stride0;
    b1 += e * g.b_stride1;
  }
  const int seg_stages = (K + TK - 1) / TK;
  const int nk = seg_stages * (MODE == DGRAD ? g.segs : 1);
  // last 8-element piece of an operand whose m or n is contiguous
  const int m_last = ((g.M + 7) & ~7) - 8, n_last = ((g.N + 7) & ~7) - 8;
  const bool gather = (MODE == GATED || MODE == WGRAD) && g.r.row_entry != nullptr;

  // Load q of this wave is piece id = q * NW + wave of the stage: 1 KB, the A
  // pieces first. Per lane: where it reads next, how far one stage is, and
  // the k of its 8 elements within a stage.
  const uint16_t *src[C::LOADS];
  int kpos[C::LOADS];
  auto start = [&](int seg) {
#pragma unroll
    for (int q = 0; q < C::LOADS; ++q) {
      const int id = q * C::NW + wave;
      if (id < C::A_INSTR) {
        if constexpr (A_TR) {
          constexpr int PER = BM / 8, KR = 64 / PER;  // chunks in a k-row, k-rows of a piece
          const int k = id * KR + lane / PER, c = (lane % PER) ^ swz<BM>(k);
          kpos[q] = k;
          src[q] = g.a + (k_row0 + k) * g.lda + seg0 * g.a_seg + min(m0 + c * 8, m_last);
        } else {
          const int r = id * 8 + (lane >> 3), c = (lane & 7) ^ (lane >> 3);
          int64_t row = min(m0 + r, g.M - 1);
          if (gather) {
            const uint32_t tok = (uint32_t)g.r.row_entry[row] / (uint32_t)g.r.top_k;
            row = tok < (uint64_t)g.a_rows ? tok : 0;
          }
          kpos[q] = c * 8;
          src[q] = g.a + row * g.lda + seg * g.a_seg + c * 8;
        }
      } else {
        const int ib = id - C::A_INSTR;
        if constexpr (B_TR) {
          constexpr int PER = BN / 8, KR = 64 / PER;
          const int k = ib * KR + lane / PER, c = (lane % PER) ^ swz<BN>(k);
          kpos[q] = k;
          const bool second = MODE == DGRAD && seg;
          src[q] = (second ? b1 : b0) + (k_row0 + k) * (second ? g.ldb1 : g.ldb0) +
                   min(n0 + c * 8, n_last);
        } else {
          const int j = ib * 8 + (lane >> 3), c = (lane & 7) ^ (lane >> 3);
          kpos[q] = c * 8;
          if constexpr (MODE == GATED) {  // 16 gate rows, their 16 up rows, ...
            const int f = min(n0 + (j >> 5) * 16 + (j & 15), g.N - 1);
            const bool up = (j >> 4) & 1;
            src[q] = (up ? b1 : b0) + f * (up ? g.ldb1 : g.ldb0) + c * 8;
          } else {
            src[q] = b0 + min(n0 + j, g.N - 1) * g.ldb0 + c * 8;
          }
        }
      }
    }
  };
  // WGRAD with gathered x: the tokens of the next stage's rows
  int32_t entry[C::LOADS];
  auto fetch_entries = [&](int s) {
    if constexpr (MODE == WGRAD) {
      if (gather) {
#pragma unroll
        for (int q = 0; q < C::LOADS; ++q)
          if (q * C::NW + wave >= C::A_INSTR)
            entry[q] = g.r.row_entry[k_row0 + min(s * TK + kpos[q], K - 1)];
      }
    }
  };
  const uint16_t *zeros = reinterpret_cast<const uint16_t *>(&zero_piece);
  // Stages are issued in order, each once.
  auto issue = [&](int s) {
    uint8_t *base = smem + (s % NS) * C::STAGE_BYTES;
    int ls = s;
    int64_t ldb = g.ldb0;
    if (MODE == DGRAD && g.segs > 1 && s >= seg_stages) {
      ls = s - seg_stages;
      ldb = g.ldb1;
      if (ls == 0) start(1);
    }
    const bool tail = (ls + 1) * TK > K;
#pragma unroll
    for (int q = 0; q < C::LOADS; ++q) {
      const int id = q * C::NW + wave;
      if (C::INSTR % C::NW != 0 && id >= C::INSTR) break;
      const uint16_t *p = src[q];
      const bool is_a = id < C::A_INSTR;
      if constexpr (MODE == WGRAD) {
        if (gather && !is_a) {
          const uint32_t tok = (uint32_t)entry[q] / (uint32_t)g.r.top_k;
          // src holds the column in row 0 .. of x: rebuilt from the token
          p = tok < (uint64_t)g.a_rows
                  ? g.b0 + (int64_t)tok * ldb +
                        min(n0 + ((lane % (BN / 8)) ^ swz<BN>(kpos[q])) * 8, n_last)
                  : zeros;
        }
      }
      if (tail && ls * TK + kpos[q] >= K) p = zeros;
      __builtin_amdgcn_global_load_lds((gbl_ptr_t)p, (lds_ptr_t)(base + id * 1024), 16, 0, 0);
      src[q] += is_a ? (A_TR ? TK * g.lda : TK) : (B_TR ? TK * ldb : TK);
    }
    fetch_entries(s + 1);
  };

  f32x4 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int wm = (wave / C::WAVES_N) * C::WM, wn = (wave % C::WAVES_N) * C::WN;
  const int fr = lane & 15, fq = lane >> 4;

  s16x8 fa[2][C::FM], fb[2][C::FN];
  // one operand's fragment of 16 rows (columns) x 32 k at k-step ks
  auto frag_k = [&](const uint8_t *t, int row, int ks) {
    return *reinterpret_cast<const s16x8 *>(t + (row + fr) * 128 +
                                            (((ks * 4 + fq) ^ (fr & 7)) * 16));
  };
  auto frag_tr = [&](const uint8_t *t, int col, int ks, auto width) {
    constexpr int R = decltype(width)::value;
    s16x8 f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = ks * 32 + fq * 8 + h * 4 + (fr >> 2);
      const int c = (col >> 3) + ((fr & 3) >> 1);
      const uint8_t *p = t + k * (R * 2) + ((c ^ swz<R>(k)) * 16) + (fr & 1) * 8;
      const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr_t)p);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[h * 4 + i] = v[i];
    }
    return f;
  };
  auto read_frags = [&](int s, int ks, int set) {
    const uint8_t *As = smem + (s % NS) * C::STAGE_BYTES, *Bs = As + C::A_BYTES;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
      if constexpr (A_TR)
        fa[set][i] = frag_tr(As, wm + 16 * i, ks, std::integral_constant<int, BM>());
      else
        fa[set][i] = frag_k(As, wm + 16 * i, ks);
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
      if constexpr (B_TR)
        fb[set][j] = frag_tr(Bs, wn + 16 * j, ks, std::integral_constant<int, BN>());
      else
        fb[set][j] = frag_k(Bs, wn + 16 * j, ks);
  };
  // The wait in stage_ready has drained this set's LDS reads, which the
  // compiler cannot see: naming the registers here keeps it from waiting
  // for the next set's reads as well.
  auto settle = [&](int set) {
#pragma unroll
    for (int i = 0; i < C::FM; ++i) asm volatile("" : "+v"(fa[set][i]));
#pragma unroll
    for (int j = 0; j < C::FN; ++j) asm volatile("" : "+v"(fb[set][j]));
  };
  auto mfmas = [&](int set) {
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) acc[i][j] = D::mfma(fb[set][j], fa[set][i], acc[i][j]);
  };
  // Stage s has landed for every wave, and every wave has read the buffer
  // that the next issue fills.
  auto stage_ready = [&](int s) {
    wait_vmcnt_steps<C::LOADS_MIN, NS - 2>(min(NS - 2, nk - 1 - s));
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (s + NS - 1 < nk) issue(s + NS - 1);
  };

  if (nk > 0) {
    start(0);
    fetch_entries(0);
#pragma unroll
    for (int s = 0; s < NS - 1; ++s)
      if (s < nk) issue(s);
    stage_ready(0);
    read_frags(0, 0, 0);
    for (int s = 0; s < nk; ++s) {
      read_frags(s, 1, 1);
      mfmas(0);
      if (s + 1 < nk) {
        stage_ready(s + 1);
        settle(1);
        read_frags(s + 1, 0, 0);
      }
      mfmas(1);
    }
  }

  // Lane: row m = fr, columns n = 4 fq .. 4 fq + 3 of every 16 x 16 tile.
  if constexpr (MODE == WGRAD) {
    uint16_t *c = seg0 ? g.c1 + e * g.c_stride1 : g.c0 + e * g.c_stride0;
    const int64_t ldc = seg0 ? g.ldc1 : g.ldc0;
    const bool vec = vec4(c, ldc);
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      const int m = m0 + wm + 16 * i + fr;
      if (m >= g.M) continue;
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        const int n = n0 + wn + 16 * j + 4 * fq;
        if (n < g.N) store4<D>(c + m * ldc + n, acc[i][j], g.N - n, vec);
      }
    }
  } else {
    const bool vec_c = vec4(g.c0, g.ldc0), vec_p = vec4(g.pre, g.ldp, g.N);
    const bool vec_r = vec4(g.res, g.ldr);
    const uint16_t *bias = g.bias ? g.bias + e * g.bias_stride : nullptr;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      const int64_t m = m0 + wm + 16 * i + fr;
      if (m >= g.M) continue;
      const bool real = !grouped || g.r.m_indices[m] == e;
      if constexpr (MODE == GATED) {
#pragma unroll
        for (int j = 0; j < C::FN / 2; ++j) {
          const int n = n0 + (wn >> 1) + 16 * j + 4 * fq, left = g.N - n;
          if (left <= 0) continue;
          f32x4 gt = acc[i][2 * j], up = acc[i][2 * j + 1], h;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            if (!real) gt[v] = up[v] = 0.f;
            h[v] = real ? act_value(gt[v], g.act) * up[v] : 0.f;
          }
          store4<D>(g.c0 + m * g.ldc0 + n, h, left, vec_c);
          if (g.pre) {
            store4<D>(g.pre + m * g.ldp + n, gt, left, vec_p);
            store4<D>(g.pre + m * g.ldp + g.N + n, up, left, vec_p);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
          const int n = n0 + wn + 16 * j + 4 * fq, left = g.N - n;
          if (left <= 0) continue;
          f32x4 z = acc[i][j];
          if constexpr (MODE == LINEAR) {
            if (bias) {
#pragma unroll
              for (int v = 0; v < 4; ++v)
                if (v < left) z[v] += to_f<D>(bias[n + v]);
            }
            if (!real) z = f32x4{0.f, 0.f, 0.f, 0.f};
            if (g.pre) store4<D>(g.pre + m * g.ldp + n, z, left, vec_p);
            if (g.act != MOE_ACT_NONE) {
#pragma unroll
              for (int v = 0; v < 4; ++v) z[v] = act_value(z[v], g.act);
            }
            if (g.res && real) {
              const f32x4 r = load4<D>(g.res + m * g.ldr + n, left, vec_r);
#pragma unroll
              for (int v = 0; v < 4; ++v) z[v] += r[v];
            }
          } else if (!real) {
            z = f32x4{0.f, 0.f, 0.f, 0.f};
          }
          store4<D>(g.c0 + m * g.ldc0 + n, z, left, vec_c);
        }
      }
    }
  }
}

}  // namespace moe_ffn
