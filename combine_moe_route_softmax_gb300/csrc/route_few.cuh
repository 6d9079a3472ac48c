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
// (s, c) += (s2, c2); the same bits whichever of the two is added to the other.
__device__ __forceinline__ void join_pair(float& s, float& c, float s2, float c2) {
  c = __fadd_rn(c, c2);
  add_pair(s, c, s2);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

constexpr int ROUTE_TOKENS = 4;   // tokens of one task

// A task is one expert and up to ROUTE_TOKENS tokens; S warps share its columns when there are few
// tasks, so that every SM has some.  By sizes alone: the logits are the same bits in any grid.
__device__ __forceinline__ int router_split(int tasks, int H) {
  if (tasks > 1024) return 1;
  return H >= 1024 ? 4 : H >= 512 ? 2 : 1;
}

// This warp's share of one task: columns of chunks (8 each) first, first + step, ...  Lane 8 * j
// ends with token t0 + j's pair.
template <int TT>
__device__ __forceinline__ void router_dot(const uint16_t* __restrict__ x, const uint16_t* __restrict__ wr, int T,
                                           int H, int t0, int first, int step, int lane, float& rs, float& rc) {
  float s[TT], c[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) s[j] = c[j] = 0.0f;
  const uint4* w4 = reinterpret_cast<const uint4*>(wr);
  // tokens past T read the last one; their sums are dropped
  const uint4* x4[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) x4[j] = reinterpret_cast<const uint4*>(x + (size_t)min(t0 + j, T - 1) * H);
#pragma unroll 4
  for (int i = first; i < H / 8; i += step) {
    float w[8], v[8];
    unpack8(__ldg(w4 + i), w);
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      unpack8(__ldg(x4[j] + i), v);
      float p = v[0] * w[0];
#pragma unroll
      for (int q = 1; q < 8; ++q) p = fmaf(v[q], w[q], p);
      add_pair(s[j], c[j], p);
    }
  }
  // each halving of the lanes also halves the tokens a lane keeps
  int keep = TT;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (keep > 1) {
      keep >>= 1;
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int j = 0; j < TT / 2; ++j)
        if (j < keep) {
          const float gs = up ? s[j] : s[j + keep], gc = up ? c[j] : c[j + keep];
          float ks = up ? s[j + keep] : s[j], kc = up ? c[j + keep] : c[j];
          join_pair(ks, kc, __shfl_xor_sync(0xffffffffu, gs, o), __shfl_xor_sync(0xffffffffu, gc, o));
          s[j] = ks;
          c[j] = kc;
        }
    } else {
      join_pair(s[0], c[0], __shfl_xor_sync(0xffffffffu, s[0], o), __shfl_xor_sync(0xffffffffu, c[0], o));
    }
  }
  rs = s[0];
  rc = c[0];
}

// All logits, by every CTA of a grid (NW warps each, all threads call; NW need not be a multiple of
// the split).
template <int NW>
__device__ __forceinline__ void router_logits(const uint16_t* x, const uint16_t* wr, const float* bias, int T, int H,
                                              int E, float* logits, float2 (*scratch)[ROUTE_TOKENS], int cta, int ctas,
                                              int warp, int lane) {
  const int groups = (T + ROUTE_TOKENS - 1) / ROUTE_TOKENS, tasks = E * groups;
  const int S = router_split(tasks, H), per = NW / S;
  const int slice = warp % S, mine = warp / S;
  for (int r = cta * per; r < tasks; r += ctas * per) {
    const int task = r + mine;
    const int e = task / groups, t0 = (task - e * groups) * ROUTE_TOKENS;
    float s = 0.0f, c = 0.0f;
    if (mine < per && task < tasks) {
      const uint16_t* row = wr + (size_t)e * H;
      if (T == 1) router_dot<1>(x, row, T, H, 0, slice * 32 + lane, 32 * S, lane, s, c);
      else router_dot<ROUTE_TOKENS>(x, row, T, H, t0, slice * 32 + lane, 32 * S, lane, s, c);
    }
    const int j = lane >> 3;       // this lane's token
    if (S > 1) {
      __syncthreads();
      if (mine < per && (lane & 7) == 0) scratch[warp][j] = make_float2(s, c);
      __syncthreads();
      if (slice != 0) continue;
      for (int q = 1; q < S; ++q) {
        const float2 v = scratch[warp + q][j];
        join_pair(s, c, v.x, v.y);
      }
    }
    if (mine < per && task < tasks && (lane & 7) == 0 && j < (T == 1 ? 1 : ROUTE_TOKENS) && t0 + j < T) {
      if (bias) add_pair(s, c, __ldg(bias + e));
      logits[(size_t)(t0 + j) * E + e] = __fadd_rn(s, c);
    }
  }
}

// One warp: the selection of route_topk_warp (its order, ties and weights, bit for bit) by warp-wide
// integer reductions; `load` reads a logit.
template <int EPL, class Load>
__device__ __forceinline__ void select_topk_warp(Load load, int E, int K, int lane, int& my_id, float& my_w) {
  uint32_t key[EPL];             // the logit's place in float order, 0 when taken
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 32 * j;
    key[j] = e < E ? (uint32_t)(route_key(load(e), e) >> 32) : 0u;
  }
  my_id = -1;
  float my_logit = 0.0f, top = 0.0f;
#pragma unroll 1
  for (int k = 0; k < K; ++k) {
    uint32_t m = key[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) m = max(m, key[j]);
    m = __reduce_max_sync(0xffffffffu, m);
    uint32_t id = 0xffffffffu;
#pragma unroll
    for (int j = EPL - 1; j >= 0; --j)
      if (key[j] == m) id = lane + 32 * j;
    id = __reduce_min_sync(0xffffffffu, id);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (lane + 32 * j == (int)id) key[j] = 0u;
    const float v = key_logit((unsigned long long)m << 32);
    if (lane == k) {
      my_id = m ? (int)id : -1;   // nothing left to choose (a NaN keyed as an empty place)
      my_logit = v;
    }
    if (k == 0) top = v;
  }
  const float ex = lane < K ? expf(my_logit - top) : 0.0f;
  float sum = 0.0f;
#pragma unroll 1
  for (int k = 0; k < K; ++k) sum += __shfl_sync(0xffffffffu, ex, k);
  my_w = __fdiv_rn(ex, sum);
}

// The top K of a row of logits that other CTAs may have written in this launch.
__device__ __forceinline__ void select_topk(const float* row, int E, int K, int lane, int& id, float& w) {
  auto load = [&](int e) { return __ldcg(row + e); };
  if (E <= 256)
    select_topk_warp<8>(load, E, K, lane, id, w);
  else
    select_topk_warp<32>(load, E, K, lane, id, w);
}

}  // namespace few
}  // namespace moe
