// Router logits of a few tokens from their hidden states, shared by moe_route_hidden
// (few_route.cu) and the few-token layer.  Internal header.
//
// logits[t, e] = x[t] . wr[e] + bias[e].  A near tie between two experts is decided by the last
// bits of the logits, so the sum is carried in two float32 words: products of BF16 are
// exact in float32, 8 of them are summed by fused multiply-adds, and each such partial sum
// enters the running pair by an error-free addition.  What is left of rounding is that of the
// 8-term sums, about 1e-9 of the logits' size each, below the final float32 rounding
// (the plain error-free sum of every product costs four times the instructions).
#pragma once

#include "route_topk.cuh"

namespace moe {
namespace few {

// (s, c) += v, with s + c the sum to about 48 bits (Knuth's two-sum).
__device__ __forceinline__ void add_pair(float& s, float& c, float v) {
  const float n = __fadd_rn(s, v);
  const float b = __fsub_rn(n, s);
  c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(n, b)), __fsub_rn(v, b)));
  s = n;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// One expert's logits for TT tokens from t0 on.
template <int TT>
__device__ __forceinline__ void router_row(const uint16_t* __restrict__ x, const uint16_t* __restrict__ wr,
                                           const float* __restrict__ bias, int T, int H, int E, int e, int t0,
                                           float* logits, int lane) {
  float s[TT], c[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) s[j] = c[j] = 0.0f;
  const uint4* w4 = reinterpret_cast<const uint4*>(wr + (size_t)e * H);
#pragma unroll 4
  for (int i = lane; i < H / 8; i += 32) {
    float w[8], v[8];
    unpack8(__ldg(w4 + i), w);
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      if (t0 + j < T) {
        unpack8(__ldg(reinterpret_cast<const uint4*>(x + (size_t)(t0 + j) * H) + i), v);
        float p = v[0] * w[0];
#pragma unroll
        for (int q = 1; q < 8; ++q) p = fmaf(v[q], w[q], p);
        add_pair(s[j], c[j], p);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < TT; ++j) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float so = __shfl_xor_sync(0xffffffffu, s[j], o), co = __shfl_xor_sync(0xffffffffu, c[j], o);
      // the two partners add in the same order, so every lane ends with the same bits
      float hi = (lane & o) ? so : s[j], lo = (lane & o) ? s[j] : so;
      float cc = (lane & o) ? co : c[j], cl = (lane & o) ? c[j] : co;
      cc = __fadd_rn(cc, cl);
      add_pair(hi, cc, lo);
      s[j] = hi;
      c[j] = cc;
    }
    if (bias) add_pair(s[j], c[j], __ldg(bias + e));
    if (lane == 0 && t0 + j < T) logits[(size_t)(t0 + j) * E + e] = __fadd_rn(s[j], c[j]);
  }
}

// All logits, (expert, up to 4 tokens) per warp: worker w of W warps.
__device__ __forceinline__ void router_logits(const uint16_t* x, const uint16_t* wr, const float* bias, int T, int H,
                                              int E, float* logits, int w, int W, int lane) {
  if (T == 1) {
    for (int e = w; e < E; e += W) router_row<1>(x, wr, bias, T, H, E, e, 0, logits, lane);
    return;
  }
  const int groups = (T + 3) / 4;
  for (int i = w; i < E * groups; i += W) router_row<4>(x, wr, bias, T, H, E, i / groups, (i % groups) * 4, logits, lane);
}

// One warp: the top K of a row of logits that other CTAs may have written in this launch.
__device__ __forceinline__ void select_topk(const float* row, int E, int K, int lane, int& id, float& w) {
  auto load = [&](int e) { return __ldcg(row + e); };
  if (E <= 64)
    route_topk_warp<2>(load, E, K, lane, id, w);
  else if (E <= 256)
    route_topk_warp<8>(load, E, K, lane, id, w);
  else
    route_topk_warp<32>(load, E, K, lane, id, w);
}

}  // namespace few
}  // namespace moe
