// ffn.hpp - host side shared by the feed-forward translation units.
#pragma once

#include "ffn_types.hpp"

namespace moe_ffn {

// Launches a product of the given mode (Mode) on tiles of bm rows (of
// M for WGRAD); compiled once for each element type.
int launch_gemm_bf16(int mode, int bm, const GemmArgs &g, hipStream_t st);
int launch_gemm_f16(int mode, int bm, const GemmArgs &g, hipStream_t st);

inline int hip_status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace moe_ffn
