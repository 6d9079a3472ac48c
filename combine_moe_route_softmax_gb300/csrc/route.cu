// Router: softmax -> top-k -> renormalise, one warp per token.
//
// The DeepEP page passes per-token topk_weights / topk_ids into dispatch and the MoonEP
// page works with [T, K] expert ids; neither defines the router function, so this takes
// the plain softmax -> top-k -> renormalise reading.  Selection happens on the float32 logits
// (softmax is monotone): descending, ties to the lower expert id, so the ids are exact.
// The renormalised weights need only the chosen logits: the full softmax denominator
// cancels, w_k = e^{l_k - l_max} / sum_j e^{l_j - l_max}.
//
// Bound: HBM, T*E*4 bytes read + T*K*8 written; one warp reads its token's E logits
// with coalesced loads (lane l holds experts l, l+32, ...).  Each of the K selection rounds
// is one 64-bit max per lane and a 5-step warp butterfly on packed (logit, id) keys.
#include "route_topk.cuh"

namespace moe {

template <int EPL>  // experts per lane = ceil(E / 32)
__global__ void __launch_bounds__(256) route_topk_kernel(const float* __restrict__ logits, int T, int E,
                                                         int K, const int32_t* __restrict__ num_tokens,
                                                         int32_t* __restrict__ topk_idx,
                                                         float* __restrict__ topk_w) {
  const int lane = threadIdx.x & 31;
  const int t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (t >= T) return;
  const int n = num_tokens ? *num_tokens : T;
  if (t >= n) {
    if (lane < K) {
      topk_idx[(size_t)t * K + lane] = -1;
      topk_w[(size_t)t * K + lane] = 0.0f;
    }
    return;
  }
  const float* row = logits + (size_t)t * E;
  int my_id;
  float my_w;
  route_topk_warp<EPL>([&](int e) { return row[e]; }, E, K, lane, my_id, my_w);
  if (lane < K) {
    topk_idx[(size_t)t * K + lane] = my_id;
    topk_w[(size_t)t * K + lane] = my_w;
  }
}

}  // namespace moe

extern "C" moe_status_t moe_route_topk(const float* logits, int T, int E, int K, const int32_t* num_tokens,
                                       int32_t* topk_idx, float* topk_w, void* stream) {
  using namespace moe;
  if (T < 0 || E < 1 || E > kMaxExperts || K < 1 || K > E || K > kMaxTopK) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MOE_ERR_ARG;
  const int threads = 256;
  const int blocks = (T + 7) / 8;
  cudaStream_t s = as_stream(stream);
  const int epl = (E + 31) / 32;
  if (epl <= 1)
    route_topk_kernel<1><<<blocks, threads, 0, s>>>(logits, T, E, K, num_tokens, topk_idx, topk_w);
  else if (epl <= 2)
    route_topk_kernel<2><<<blocks, threads, 0, s>>>(logits, T, E, K, num_tokens, topk_idx, topk_w);
  else if (epl <= 4)
    route_topk_kernel<4><<<blocks, threads, 0, s>>>(logits, T, E, K, num_tokens, topk_idx, topk_w);
  else if (epl <= 8)
    route_topk_kernel<8><<<blocks, threads, 0, s>>>(logits, T, E, K, num_tokens, topk_idx, topk_w);
  else if (epl <= 16)
    route_topk_kernel<16><<<blocks, threads, 0, s>>>(logits, T, E, K, num_tokens, topk_idx, topk_w);
  else
    route_topk_kernel<32><<<blocks, threads, 0, s>>>(logits, T, E, K, num_tokens, topk_idx, topk_w);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
