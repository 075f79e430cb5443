// adapter_f16.hip - the products with a low-rank term on fp16 matrices.
#include "ffn_launch.hpp"

namespace moe_ffn {
int launch_low_f16(int mode, int kind, const GemmArgs &g, hipStream_t st) {
  return launch_low<F16>(mode, kind, g, st);
}
}  // namespace moe_ffn
