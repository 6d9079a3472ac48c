// moe_route_hidden: router logits from hidden states, top-k and weights in one launch.
// The warps share out the tasks of route_few.cuh; the CTA that finishes last selects.  Bound:
// reading the router matrix (2 * E * H bytes) once; at these sizes it is in L2 and the
// time is the latency of a few CTAs (at most 16 have work with 64 experts, 64 with 256): 4.5 to 5.5 us for one
// token at H = 2048, E = 64, top-8; 6.8 to 7.8 at H = 7168, E = 256; 10 to 13 for 32 tokens there, 2 to 3 of them the
// selection.
#include <algorithm>

#include "route_few.cuh"

namespace moe {
namespace few {

constexpr int ROUTE_WARPS = 16;

// A CTA per task beyond ROUTE_TOKENS tokens; the last CTA of each 16 tokens selects for them, one warp
// a token.
__global__ void __launch_bounds__(ROUTE_WARPS * 32) route_hidden_kernel(
    const uint16_t* x, const uint16_t* wr, const float* bias, int T, int H, int E, int K, const int32_t* num_tokens,
    float* logits, int32_t* topk_idx, float* topk_w, uint32_t* count) {
  __shared__ bool last;
  __shared__ float2 scratch[ROUTE_SCRATCH];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  router_logits<ROUTE_WARPS>(x, wr, bias, T, H, E, logits, scratch, blockIdx.x, gridDim.x, warp, lane);
  const int groups = mma_groups(T), group = blockIdx.x % groups;     // of tokens (the grid is whole rounds of them)
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(&count[group], 1u) == gridDim.x / groups - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (threadIdx.x == 0) count[group] = 0;
  const int n = num_tokens ? *num_tokens : T;
  const int t = group * MMA_TOKENS + warp;
  if (t >= T) return;
  int id = -1;
  float w = 0.0f;
  if (t < n) select_topk(logits + (size_t)t * E, E, K, lane, id, w);
  if (lane < K) {
    topk_idx[t * K + lane] = id;
    topk_w[t * K + lane] = w;
  }
}
static_assert(ROUTE_WARPS == MMA_TOKENS, "a warp per token");

}  // namespace few
}  // namespace moe

extern "C" size_t moe_route_hidden_workspace_bytes(void) { return 256; }

extern "C" moe_status_t moe_route_hidden(const uint16_t* x, int T, int H, const uint16_t* w_router, const float* bias,
                                         int E, int K, const int32_t* num_tokens, float* logits, int32_t* topk_idx,
                                         float* topk_w, void* ws, size_t ws_bytes, void* stream) {
  using namespace moe;
  using namespace moe::few;
  if (T < 0 || T > MOE_FEW_MAX_TOKENS || H <= 0 || H % 128 || E < 1 || E > kMaxExperts || K < 1 || K > E ||
      K > kMaxTopK)
    return MOE_ERR_ARG;
  if (!ws || ws_bytes < moe_route_hidden_workspace_bytes()) return MOE_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) & 255) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !w_router || !logits || !topk_idx || !topk_w) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w_router)) & 15) return MOE_ERR_ARG;
  const int ctas = T > ROUTE_TOKENS ? mma_tasks(T, E) : std::min(E, num_sms() * 2);
  route_hidden_kernel<<<ctas, ROUTE_WARPS * 32, 0, as_stream(stream)>>>(
      x, w_router, bias, T, H, E, K, num_tokens, logits, topk_idx, topk_w, static_cast<uint32_t*>(ws));
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
