// ffn.hpp - host side shared by the feed-forward translation units.
#pragma once

#include "ffn_types.hpp"

namespace moe_ffn {

// Tile shapes of the products, named by their rows of M.
enum TileKind { TILE_16, TILE_32, TILE_64, TILE_64W, TILE_128, TILE_128W, TILE_256 };

// Launches a product of the given mode (Mode); compiled for each element type.
int launch_gemm_bf16(int mode, int kind, const GemmArgs &g, hipStream_t st);
int launch_gemm_f16(int mode, int kind, const GemmArgs &g, hipStream_t st);

inline int hip_status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace moe_ffn
