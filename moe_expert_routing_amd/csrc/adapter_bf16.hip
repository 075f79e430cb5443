// adapter_bf16.hip - the products with a low-rank term on bf16 matrices.
#include "ffn_launch.hpp"

namespace moe_ffn {
int launch_low_bf16(int mode, int kind, const GemmArgs &g, hipStream_t st) {
  return launch_low<Bf16>(mode, kind, g, st);
}
}  // namespace moe_ffn
