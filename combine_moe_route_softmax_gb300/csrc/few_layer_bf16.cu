// The few-token layer with BF16 weights (few_layer.cuh).
#include "few_layer.cuh"

namespace moe {
namespace few {
cudaError_t launch_layer_bf16(const LayerArgs& a, cudaStream_t stream) { return launch_layer<F_BF16, 0>(a, stream); }
}  // namespace few
}  // namespace moe
