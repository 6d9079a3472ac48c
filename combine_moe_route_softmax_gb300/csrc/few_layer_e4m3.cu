// The few-token layer with E4M3 weights (few_layer.cuh).
#include "few_layer.cuh"

namespace moe {
namespace few {
cudaError_t launch_layer_e4m3(const LayerArgs& a, cudaStream_t stream) { return launch_layer<F_E4M3, 0>(a, stream); }
}  // namespace few
}  // namespace moe
