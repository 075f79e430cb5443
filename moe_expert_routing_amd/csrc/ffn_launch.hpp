// ffn_launch.hpp - tile shapes and launches of the products, for one type.
#pragma once

#include "ffn.hpp"
#include "ffn_gemm.hpp"

namespace moe_ffn {

//            BM   BN   WM  WN NS blocks/CU
typedef Tile<256, 256, 128, 64, 2, 1> Tile256;
typedef Tile<128, 128, 64, 64, 2, 2> Tile128;
typedef Tile<64, 128, 64, 32, 3, 2> Tile64;
typedef Tile<32, 128, 32, 32, 3, 2> Tile32;
typedef Tile<16, 128, 16, 32, 4, 2> Tile16;

template <class D, int MODE, class C>
static int launch(GemmArgs g, hipStream_t st) {
  const int bn = MODE == GATED ? C::BN / 2 : C::BN;
  g.m_tiles = (g.M + C::BM - 1) / C::BM;
  g.n_tiles = (g.N + bn - 1) / bn;
  int64_t blocks = (int64_t)g.m_tiles * g.n_tiles;
  if (MODE == WGRAD) blocks *= (int64_t)(g.r.num_experts > 0 ? g.r.num_experts : 1) * g.segs;
  if (blocks == 0) return MOE_OK;
  if (blocks > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  gemm_kernel<D, MODE, C><<<dim3((uint32_t)blocks), dim3(C::NTHREADS), 0, st>>>(g);
  return hip_status();
}

template <class D, int MODE>
static int launch_bm(int bm, const GemmArgs &g, hipStream_t st) {
  if (bm == 256) return launch<D, MODE, Tile256>(g, st);
  if (bm == 128) return launch<D, MODE, Tile128>(g, st);
  if constexpr (MODE != WGRAD) {
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
