// ffn_skinny.hpp - the forward products for few rows (decode): h or y of 16
// rows of one weight matrix, bound by reading that matrix once.
//
// The weights go from global memory straight into MFMA operands, with no
// LDS and no barrier in the loop: a wave takes 16 weight rows (GATED: 8 of
// the gate, their 8 of the other projection) and a range of k, loads U k-steps of
// them (1 KB each) and of the few x rows, and multiplies one batch while the
// next is on its way. KW waves of a block share their weight rows, each with
// its own k range; their partial sums are added through LDS in the order of
// k. GW such groups stand in a block.
//
// One row, 7168 -> 2048 gated (59 MB): 11.5-12.5 us, 4.7-5.1 TB/s, what a large
// copy reaches here. 28 live experts of 112, 7168 -> 1024 gated (822 MB): 130-150
// us, 5.5-6.3 TB/s. 1024 -> 7168 (411 MB): 90-105 us; a wave has only 32 k-steps
// there. Batches of 8 k-steps instead of 4 took 10 to 25 % longer (more registers,
// fewer waves); the tiled kernel, with the weights staged in LDS, took 37 us and
// 309 us for the first two.
#pragma once

#include "ffn_gemm.hpp"

namespace moe_ffn {

constexpr int SKINNY_WAVES = 8;

template <class D, int MODE, int KW, int U, bool GATHER>
__global__ __launch_bounds__(64 * SKINNY_WAVES) void skinny_kernel(const GemmArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int GW = SKINNY_WAVES / KW, NC = MODE == GATED ? 8 : 16, BM = 16;
  __shared__ __attribute__((aligned(16))) float part[SKINNY_WAVES][BM][20];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = wave % KW, gw = wave / KW;
  const bool grouped = g.r.num_experts > 0;
  const uint32_t block = blockIdx.x + g.block0;
  const int nt = block % g.n_tiles, mt = block / g.n_tiles;
  const int m0 = mt * BM, n0 = nt * GW * NC;
  int e = 0;
  bool live = true;
  if (grouped) {
    e = g.r.m_indices[m0];
    live = e >= 0 && e < g.r.num_experts && g.a_rows > 0;
  }
  const int K = g.K, fr = lane & 15, fq = lane >> 4;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};

  if (live) {
    // whole k-steps, handed out in pairs so that waves part at 128-byte lines
    const int steps = (K + 31) / 32, per = ((steps + KW - 1) / KW + 1) & ~1;
    const int s0 = min(steps, kw * per), s1 = min(steps, s0 + per);
    const bool second = MODE == GATED && fr >= 8;
    const int nb = n0 + gw * NC + (MODE == GATED ? fr & 7 : fr);
    const uint16_t *w = second ? g.b1 + e * g.b_stride1 + (int64_t)min(nb, g.N - 1) * g.ldb1
                               : g.b0 + e * g.b_stride0 + (int64_t)min(nb, g.N - 1) * g.ldb0;
    w += s0 * 32 + fq * 8;
    const uint32_t magic = g.top_k_magic, shift = g.top_k_shift;
    int64_t row = min(m0 + fr, g.M - 1);
    if (GATHER) {
      const uint32_t en = (uint32_t)g.r.row_entry[row];
      const uint32_t t = magic ? __umulhi(en, magic) >> shift : en;
      row = t < (uint64_t)g.a_rows ? t : 0;
    }
    const uint16_t *xr = g.a + row * g.lda + s0 * 32 + fq * 8;
    s16x8 fw[2][U], fx[2][U];
    auto load = [&](int set, int s) MOE_INLINE {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        fw[set][u] = *reinterpret_cast<const s16x8_any *>(w + (s + u) * 32);
        fx[set][u] = *reinterpret_cast<const s16x8_any *>(xr + (s + u) * 32);
      }
    };
    auto multiply = [&](int set) MOE_INLINE {
#pragma unroll
      for (int u = 0; u < U; ++u) acc = D::mfma(fw[set][u], fx[set][u], acc);
    };
    // batches whose last step lies inside K
    const int whole = max(0, (min(s1, K / 32) - s0) / U);
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
      const int in = K - (s0 + s) * 32 - fq * 8;  // elements left in this lane's piece
      const s16x8 a = load8_raw(w + s * 32, 0, in);
      const s16x8 c = load8_raw(xr + s * 32, 0, in);
      acc = D::mfma(a, c, acc);
    }
    *reinterpret_cast<f32x4 *>(&part[wave][fr][4 * fq]) = acc;
  }
  __syncthreads();
  // eight columns of a row a thread
  constexpr int RUNS = NC / 8;
  for (int o = threadIdx.x; o < GW * BM * RUNS; o += 64 * SKINNY_WAVES) {
    const int c = o % RUNS * 8, gr = o / RUNS % GW, r = o / (RUNS * GW);
    const int n = n0 + gr * NC + c;
    const int64_t m = m0 + r;
    if (n >= g.N || m >= g.M) continue;
    const bool real = live && (!grouped || g.r.m_indices[m] == e);
    f32x8 z = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, u = z;
    if (real) {
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const float *p = &part[gr * KW + k][r][c];
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          z[v] += p[v];
          if (MODE == GATED) u[v] += p[8 + v];
        }
      }
    }
    if constexpr (MODE == GATED) {
      if (g.pre) {
        store8<D>(g.pre + m * g.ldp, n, g.N, z);
        store8<D>(g.pre + m * g.ldp + g.N, n, g.N, u);
      }
      z = act_value(z, g.act);
#pragma unroll
      for (int v = 0; v < 8; ++v) z[v] = real ? z[v] * u[v] : 0.f;
    } else {
      if (real && g.bias) {
        const f32x8 b = load8<D>(g.bias + e * g.bias_stride, n, g.N);
#pragma unroll
        for (int v = 0; v < 8; ++v) z[v] += b[v];
      }
      if (g.pre) store8<D>(g.pre + m * g.ldp, n, g.N, z);
      z = act_value(z, g.act);  // 0 stays 0
      if (real && g.res) {
        const f32x8 b = load8<D>(g.res + m * g.ldr, n, g.N);
#pragma unroll
        for (int v = 0; v < 8; ++v) z[v] += b[v];
      }
    }
    store8<D>(g.c0 + m * g.ldc0, n, g.N, z);
  }
#endif
}

}  // namespace moe_ffn
