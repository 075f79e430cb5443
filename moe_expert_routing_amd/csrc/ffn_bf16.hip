// ffn_bf16.hip - the products of the feed-forward operators on bf16 matrices.
#include "ffn_launch.hpp"

namespace moe_ffn {
int launch_gemm_bf16(int mode, int kind, const GemmArgs &g, hipStream_t st) {
  return launch_mode<Bf16>(mode, kind, g, st);
}
}  // namespace moe_ffn
