// ffn_launch.hpp - tile shapes and launches of the products, for one type.
#pragma once

#include "ffn.hpp"
#include "ffn_gemm.hpp"
#include "ffn_skinny.hpp"

namespace moe_ffn {

//           BM   BN   WM  WN NS blocks/CU
typedef Tile<256, 256, 128, 64, 2, 1> Tile256;
typedef Tile<128, 256, 64, 64, 3, 1> Tile128w;
typedef Tile<128, 128, 64, 32, 4, 1> Tile128;
typedef Tile<64, 256, 32, 64, 2, 2> Tile64w;
typedef Tile<64, 64, 32, 32, 4, 2> Tile64;
typedef Tile<32, 64, 16, 32, 4, 2> Tile32;
typedef Tile<16, 128, 16, 32, 4, 2> Tile16;

template <class D, int MODE, class C, bool LOW = false>
static int launch(GemmArgs g, hipStream_t st) {
  const int bn = MODE == GATED ? C::BN / 2 : C::BN;
  if (!g.tile_map) g.m_tiles = (g.M + C::BM - 1) / C::BM;
  g.n_tiles = (g.N + bn - 1) / bn;
  int64_t blocks = (int64_t)g.m_tiles * g.n_tiles;
  if (MODE == WGRAD) blocks *= (int64_t)(g.r.num_experts > 0 ? g.r.num_experts : 1) * g.segs;
  if (g.partial) blocks *= g.splits;
  if (blocks > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  // the forward tiles of dense_plan alone never gather
  constexpr bool DENSE = std::is_same_v<C, Tile128> || std::is_same_v<C, Tile64>;
  constexpr bool GATHERS = !LOW && (MODE == WGRAD || (MODE == GATED && !DENSE));
  if (!GATHERS && g.r.row_entry) return MOE_ERR_UNSUPPORTED;
  const auto kernel =
      g.r.row_entry ? gemm_kernel<D, MODE, C, GATHERS, LOW> : gemm_kernel<D, MODE, C, false, LOW>;
  return in_parts(blocks, C::NTHREADS, [&](int64_t first, uint32_t n) {
    g.block0 = (uint32_t)first;
    kernel<<<n, C::NTHREADS, 0, st>>>(g);
    return hip_status();
  });
}

template <class D, int MODE, int KW>
static int launch_skinny_kw(GemmArgs g, hipStream_t st) {
  constexpr int COLS = SKINNY_WAVES / KW * (MODE == GATED ? 8 : 16);
  g.m_tiles = (g.M + 15) / 16;
  g.n_tiles = (g.N + COLS - 1) / COLS;
  const int64_t blocks = (int64_t)g.m_tiles * g.n_tiles;
  if (blocks > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  constexpr bool GATHERS = MODE == GATED && KW < 8;  // 8 waves: dense calls alone
  if (!GATHERS && g.r.row_entry) return MOE_ERR_UNSUPPORTED;
  const auto kernel =
      g.r.row_entry ? skinny_kernel<D, MODE, KW, 4, GATHERS> : skinny_kernel<D, MODE, KW, 4, false>;
  return in_parts(blocks, 64 * SKINNY_WAVES, [&](int64_t first, uint32_t n) {
    g.block0 = (uint32_t)first;
    kernel<<<n, 64 * SKINNY_WAVES, 0, st>>>(g);
    return hip_status();
  });
}
// Waves that share weight rows. Dense calls have few blocks: all 8, or 4 where
// that already gives more than one block and a half for each compute unit
// (1 row, 2048 -> 7168: 7.9 us with 4, 8.5 with 8; 7168 -> 2048 gated: 12.6 with
// 8, 19.1 with 4). Over experts there are enough blocks, and longer ranges of k
// read faster (28 live experts: 7168 -> 1024 gated 147 us with 4, 151 with 8, 159
// with 1; 1024 -> 7168 111 us with 1, 121 with 2, 148 with 8).
template <class D, int MODE>
static int launch_skinny(const GemmArgs &g, hipStream_t st) {
  if (g.r.num_experts == 0) {
    const int blocks = g.N / (MODE == GATED ? 8 : 16);
    return blocks >= 384 ? launch_skinny_kw<D, MODE, 4>(g, st)
                         : launch_skinny_kw<D, MODE, 8>(g, st);
  }
  if (g.K >= 4096) return launch_skinny_kw<D, MODE, 4>(g, st);
  if (g.K >= 2048) return launch_skinny_kw<D, MODE, 2>(g, st);
  return launch_skinny_kw<D, MODE, 1>(g, st);
}

template <class D, int MODE>
static int launch_kind(int kind, const GemmArgs &g, hipStream_t st) {
  switch (kind) {
    case TILE_256: return launch<D, MODE, Tile256>(g, st);
    case TILE_128: return launch<D, MODE, Tile128>(g, st);
    case TILE_64: return launch<D, MODE, Tile64>(g, st);
    case TILE_32: return launch<D, MODE, Tile32>(g, st);
  }
  if constexpr (MODE != WGRAD) {
    if (kind == TILE_128W) return launch<D, MODE, Tile128w>(g, st);
    if (kind == TILE_64W) return launch<D, MODE, Tile64w>(g, st);
  }
  if constexpr (MODE == DGRAD) {
    if (kind == TILE_16) return launch<D, MODE, Tile16>(g, st);
  } else if constexpr (MODE != WGRAD) {
    if (kind == TILE_16) return launch_skinny<D, MODE>(g, st);
  }
  return MOE_ERR_UNSUPPORTED;
}

// Dense products with a low-rank term: y's and dx's.
template <class D, int MODE>
static int launch_low_kind(int kind, const GemmArgs &g, hipStream_t st) {
  switch (kind) {
    case TILE_256: return launch<D, MODE, Tile256, true>(g, st);
    case TILE_128: return launch<D, MODE, Tile128, true>(g, st);
    case TILE_64: return launch<D, MODE, Tile64, true>(g, st);
    case TILE_32: return launch<D, MODE, Tile32, true>(g, st);
  }
  return MOE_ERR_UNSUPPORTED;
}
template <class D>
static int launch_low(int mode, int kind, const GemmArgs &g, hipStream_t st) {
  if (mode == LINEAR) return launch_low_kind<D, LINEAR>(kind, g, st);
  if (mode == DGRAD) return launch_low_kind<D, DGRAD>(kind, g, st);
  return MOE_ERR_UNSUPPORTED;
}

template <class D>
static int launch_mode(int mode, int kind, const GemmArgs &g, hipStream_t st) {
  switch (mode) {
    case GATED: return launch_kind<D, GATED>(kind, g, st);
    case LINEAR: return launch_kind<D, LINEAR>(kind, g, st);
    case DGRAD: return launch_kind<D, DGRAD>(kind, g, st);
    case WGRAD: return launch_kind<D, WGRAD>(kind, g, st);
  }
  return MOE_ERR_UNSUPPORTED;
}

}  // namespace moe_ffn
