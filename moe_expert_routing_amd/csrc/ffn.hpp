// ffn.hpp - host side shared by the feed-forward translation units.
#pragma once

#include "ffn_types.hpp"

namespace moe_ffn {

// Tile shapes of the products, named by their rows of M.
enum TileKind { TILE_16, TILE_32, TILE_64, TILE_64W, TILE_128, TILE_128W, TILE_256 };

// Launches a product of the given mode (Mode); compiled for each element type.
int launch_gemm_bf16(int mode, int kind, const GemmArgs &g, hipStream_t st);
int launch_gemm_f16(int mode, int kind, const GemmArgs &g, hipStream_t st);

// A launch takes fewer than 2^32 work items in a dimension of its grid: more blocks
// go in several, each of which is told the number of its first. Its status.
template <class Launch>
static int in_parts(int64_t blocks, int threads, Launch &&launch) {
  const int64_t most = ((((int64_t)1 << 32) - 1) / threads) & ~(int64_t)7;  // whole rounds of XCDs
  for (int64_t first = 0; first < blocks; first += most) {
    const int status = launch(first, (uint32_t)(blocks - first < most ? blocks - first : most));
    if (status != MOE_OK) return status;
  }
  return MOE_OK;
}

inline int hip_status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace moe_ffn
