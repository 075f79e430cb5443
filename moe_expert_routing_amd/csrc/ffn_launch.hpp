// ffn_launch.hpp - tile shapes and launches of the products, for one type.
#pragma once

#include "ffn.hpp"
#include "ffn_gemm.hpp"
#include "ffn_skinny.hpp"

namespace moe_ffn {

//           BM   BN   WM  WN TK NS blocks/CU
typedef Tile<256, 256, 128, 64, 64, 2, 1> Tile256;
typedef Tile<128, 128, 64, 64, 64, 2, 2> Tile128;
typedef Tile<64, 128, 64, 32, 64, 3, 2> Tile64;
typedef Tile<32, 128, 32, 32, 64, 3, 2> Tile32;
typedef Tile<16, 128, 16, 32, 64, 4, 2> Tile16;

template <class D, int MODE, class C>
static int launch(GemmArgs g, hipStream_t st) {
  const int bn = MODE == GATED ? C::BN / 2 : C::BN;
  g.m_tiles = (g.M + C::BM - 1) / C::BM;
  g.n_tiles = (g.N + bn - 1) / bn;
  int64_t blocks = (int64_t)g.m_tiles * g.n_tiles;
  if (MODE == WGRAD) blocks *= (int64_t)(g.r.num_experts > 0 ? g.r.num_experts : 1) * g.segs;
  if (blocks == 0) return MOE_OK;
  if (blocks > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  const dim3 grid((uint32_t)blocks), block(C::NTHREADS);
  if constexpr (MODE == GATED || MODE == WGRAD) {
    if (g.r.row_entry) {
      gemm_kernel<D, MODE, C, true><<<grid, block, 0, st>>>(g);
      return hip_status();
    }
  }
  gemm_kernel<D, MODE, C, false><<<grid, block, 0, st>>>(g);
  return hip_status();
}

// Waves that share weight rows: a wave's k range is at least 512.
template <class D, int MODE, int RX, int KW, int U>
static int launch_skinny_kw(GemmArgs g, hipStream_t st) {
  constexpr int COLS = SKINNY_WAVES / KW * (MODE == GATED ? 8 : 16);
  g.m_tiles = (g.M + 16 * RX - 1) / (16 * RX);
  g.n_tiles = (g.N + COLS - 1) / COLS;
  const int64_t blocks = (int64_t)g.m_tiles * g.n_tiles;
  if (blocks == 0) return MOE_OK;
  if (blocks > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  const dim3 grid((uint32_t)blocks), block(64 * SKINNY_WAVES);
  if (MODE == GATED && g.r.row_entry)
    skinny_kernel<D, MODE, RX, KW, U, MODE == GATED><<<grid, block, 0, st>>>(g);
  else
    skinny_kernel<D, MODE, RX, KW, U, false><<<grid, block, 0, st>>>(g);
  return hip_status();
}
template <class D, int MODE, int RX, int U>
static int launch_skinny(const GemmArgs &g, hipStream_t st) {
  if (g.K >= 4096) return launch_skinny_kw<D, MODE, RX, 8, U>(g, st);
  if (g.K >= 2048) return launch_skinny_kw<D, MODE, RX, 4, U>(g, st);
  if (g.K >= 1024) return launch_skinny_kw<D, MODE, RX, 2, U>(g, st);
  return launch_skinny_kw<D, MODE, RX, 1, U>(g, st);
}

template <class D, int MODE>
static int launch_bm(int bm, const GemmArgs &g, hipStream_t st) {
  if constexpr (MODE == GATED || MODE == LINEAR) {
    if (bm == 16) return launch_skinny<D, MODE, 1, 8>(g, st);
    if (bm == 32) return launch_skinny<D, MODE, 2, 4>(g, st);
    if (bm == 64) return launch_skinny<D, MODE, 4, 4>(g, st);
  }
  if (bm == 256) return launch<D, MODE, Tile256>(g, st);
  if (bm == 128) return launch<D, MODE, Tile128>(g, st);
  if constexpr (MODE == DGRAD) {
    if (bm == 64) return launch<D, MODE, Tile64>(g, st);
    if (bm == 32) return launch<D, MODE, Tile32>(g, st);
    if (bm == 16) return launch<D, MODE, Tile16>(g, st);
  }
  return MOE_ERR_UNSUPPORTED;
}

template <class D>
static int launch_mode(int mode, int bm, const GemmArgs &g, hipStream_t st) {
  switch (mode) {
    case GATED: return launch_bm<D, GATED>(bm, g, st);
    case LINEAR: return launch_bm<D, LINEAR>(bm, g, st);
    case DGRAD: return launch_bm<D, DGRAD>(bm, g, st);
    case WGRAD: return launch_bm<D, WGRAD>(bm, g, st);
  }
  return MOE_ERR_UNSUPPORTED;
}

}  // namespace moe_ffn
