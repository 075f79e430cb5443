// ffn_f16.hip - the products of the feed-forward operators on fp16 matrices.
#include "ffn_launch.hpp"

namespace moe_ffn {
int launch_gemm_f16(int mode, int kind, const GemmArgs &g, hipStream_t st) {
  return launch_mode<F16>(mode, kind, g, st);
}
}  // namespace moe_ffn
