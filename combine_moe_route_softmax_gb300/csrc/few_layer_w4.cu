// The few-token layer with 4-bit weights (few_layer.cuh), one instance per group size.
#include "few_layer.cuh"

namespace moe {
namespace few {
cudaError_t launch_layer_w4(const LayerArgs& a, int group, cudaStream_t stream) {
  if (group == 32) return launch_layer<F_W4, 32>(a, stream);
  if (group == 64) return launch_layer<F_W4, 64>(a, stream);
  return launch_layer<F_W4, 128>(a, stream);
}
}  // namespace few
}  // namespace moe
