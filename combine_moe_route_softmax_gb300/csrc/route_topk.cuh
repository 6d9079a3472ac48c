// Top-k selection of one token's router logits by one warp, shared by moe_route_topk
// (route.cu) and the few-token kernels (few_layer.cuh, few_route.cu).  Internal header.
//
// Selection happens on the float32 logits (softmax is monotone): descending, ties to the
// lower expert id, so the ids are exact.  The renormalised weights need only the chosen
// logits: the full softmax denominator cancels, w_k = e^{l_k - l_max} / sum_j e^{l_j - l_max}.
#pragma once

#include "common.cuh"

namespace moe {

// Order-preserving key of (logit, expert id): the float's bits mapped so that unsigned order
// is float order in the high word, the complemented id in the low word -- so the largest
// key is the largest logit, ties going to the lower id.  0 marks an empty entry (every
// finite logit maps above it).  -0 is keyed as +0: equal floats tie on the id.
__device__ __forceinline__ unsigned long long route_key(float v, int e) {
  const uint32_t b = v == 0.0f ? 0u : __float_as_uint(v);
  const uint32_t ord = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((unsigned long long)ord << 32) | (uint32_t)(~e);
}
__device__ __forceinline__ float key_logit(unsigned long long k) {
  const uint32_t ord = (uint32_t)(k >> 32);
  return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7fffffffu) : ~ord);
}

// The whole warp selects from row [E] (EPL = ceil(E / 32) logits per lane); lane k < K gets
// the k-th expert id and its weight.
template <int EPL, class Load>
__device__ __forceinline__ void route_topk_warp(Load load, int E, int K, int lane, int& my_id, float& my_w) {
  unsigned long long key[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 32 * j;
    key[j] = e < E ? route_key(load(e), e) : 0ull;
  }
  my_id = -1;          // lane k keeps the k-th chosen id and logit
  float my_logit = 0.0f;
  float top_logit = 0.0f;
  for (int k = 0; k < K; ++k) {
    unsigned long long m = key[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) m = key[j] > m ? key[j] : m;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const unsigned long long o = __shfl_xor_sync(0xffffffffu, m, off);
      m = o > m ? o : m;
    }
    // m is warp-uniform: its owner clears it
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (key[j] == m) key[j] = 0ull;
    const float lv = key_logit(m);
    if (lane == k) {
      my_id = (int)(~(uint32_t)m);
      my_logit = lv;
    }
    if (k == 0) top_logit = lv;
  }
  const float ex = (lane < K) ? expf(my_logit - top_logit) : 0.0f;
  // sum in ascending slot order (a fixed order, independent of the warp reduction tree)
  float sum = 0.0f;
  for (int k = 0; k < K; ++k) sum += __shfl_sync(0xffffffffu, ex, k);
  my_w = __fdiv_rn(ex, sum);
}

}  // namespace moe
