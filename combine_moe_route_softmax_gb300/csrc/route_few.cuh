// Router logits of a few tokens from their hidden states, shared by moe_route_hidden
// (few_route.cu) and the few-token layer.  Internal header.
//
// logits[t, e] = x[t] . wr[e] + bias[e].  A near tie between two experts is decided by the last
// bits of the logits, so the sum is carried in two float32 words: products of BF16 are
// exact in float32, 8 of them are summed by fused multiply-adds (up to 4 tokens), or 16 by a tensor
// instruction (more), and each such partial sum enters the running pair by an error-free addition.  What
// is left of rounding is that of the partial sums, 7 half steps of 8 products (2^-21 of their magnitudes at
// worst) or 15 steps of 16 (2^-19), and the final one to float32.  Measured at H = 7168: an error of 9e-8 of the
// logits' size, of which a correctly rounded sum has 5e-8.  So the bits of a token's logits depend on its row,
// the sizes and on which side of 4 tokens the call is, not on the grid, the warps or the other tokens
// (the error-free sum of every product would cost four times the instructions).
#pragma once

#include "few.cuh"
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
// The pair's value.  An infinite or NaN sum (an expert masked by a bias of -infinity) is s alone: it is the plain
// sum then, and what the error-free addition left in c is NaN.
__device__ __forceinline__ float pair_value(float s, float c) {
  return (__float_as_uint(s) & 0x7fffffffu) < 0x7f800000u ? __fadd_rn(s, c) : s;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Up to ROUTE_TOKENS tokens a task is one expert, and S warps share its columns; a CTA has NW / S experts at
// a time, so 64 experts at H >= 1024 lie on 16 SMs, 256 on 64.  S goes by sizes alone: the logits are the
// same bits in any grid.
constexpr int ROUTE_TOKENS = 4;
__device__ __forceinline__ int router_split(int H) { return H >= 1024 ? 4 : H >= 512 ? 2 : 1; }

// This warp's share of one task: columns of chunks (8 each) first, first + step, ...  Lane 8 * j
// ends with token j's pair.
template <int TT>
__device__ __forceinline__ void router_dot(const uint16_t* __restrict__ x, const uint16_t* __restrict__ wr, int T,
                                           int H, int first, int step, int lane, float& rs, float& rc) {
  float s[TT], c[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) s[j] = c[j] = 0.0f;
  const uint4* w4 = reinterpret_cast<const uint4*>(wr);
  // tokens past T read the last one; their sums are dropped
  const uint4* x4[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) x4[j] = reinterpret_cast<const uint4*>(x + (size_t)min(j, T - 1) * H);
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

// More than ROUTE_TOKENS tokens: a task is 16 tokens and 8 experts, its columns shared out in MMA_SLICES
// slices, 32 columns at a time in turn, and the slices between the CTA's warps (16 of them, whatever the
// warps: 12 in a 4-bit layer).  A tensor instruction (tokens as its 16 rows, experts as its 8 columns)
// starts from zero and gives sums of 16 products, which enter the pairs as above.  At H = 7168, E = 256:
// 11.2 us against 8.7 on the other path for 4 tokens, 12.8 against 20.2 for 32.
constexpr int MMA_TOKENS = 16, MMA_EXPERTS = 8, MMA_SLICES = 16;
__host__ __device__ __forceinline__ int mma_groups(int T) { return (T + MMA_TOKENS - 1) / MMA_TOKENS; }
__host__ __device__ __forceinline__ int mma_tasks(int T, int E) {
  return (E + MMA_EXPERTS - 1) / MMA_EXPERTS * mma_groups(T);
}
constexpr int ROUTE_SCRATCH = MMA_SLICES * MMA_TOKENS * MMA_EXPERTS;   // float2
template <int NW>
__device__ __forceinline__ void router_logits_mma(const uint16_t* __restrict__ x, const uint16_t* __restrict__ wr,
                                                  const float* bias, int T, int H, int E, float* logits,
                                                  float2* scratch, int cta, int ctas, int warp, int lane) {
  const int groups = mma_groups(T), tasks = mma_tasks(T, E), g = lane >> 2, t = lane & 3;
  for (int task = cta; task < tasks; task += ctas) {
    const int e0 = task / groups * MMA_EXPERTS, t0 = task % groups * MMA_TOKENS;
    // tokens past T read the last one, experts past E too; their sums are dropped
    const uint4* x0 = reinterpret_cast<const uint4*>(x + (size_t)min(t0 + g, T - 1) * H) + t;
    const uint4* x1 = reinterpret_cast<const uint4*>(x + (size_t)min(t0 + g + 8, T - 1) * H) + t;
    const uint4* w = reinterpret_cast<const uint4*>(wr + (size_t)min(e0 + g, E - 1) * H) + t;
    auto sums = [&](int slice, bool wait) {
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
      for (int i = slice; i < H / 32; i += MMA_SLICES) {
        const uint4 a = __ldg(x0 + i * 4), b = __ldg(x1 + i * 4), v = __ldg(w + i * 4);
        float d[2][4];
        mma16_first<false>(d[0], a.x, b.x, a.y, b.y, v.x, v.y);
        mma16_first<false>(d[1], a.z, b.z, a.w, b.w, v.z, v.w);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) add_pair(s[q], c[q], d[j][q]);
      }
      if (wait) __syncthreads();           // the task before is read
#pragma unroll
      for (int q = 0; q < 4; ++q) scratch[(slice * 4 + q) * 32 + lane] = make_float2(s[q], c[q]);
    };
    if constexpr (NW == MMA_SLICES) {
      sums(warp, true);
    } else {
#pragma unroll 1
      for (int slice = warp; slice < MMA_SLICES; slice += NW) sums(slice, slice < NW);
    }
    __syncthreads();
    const int i = warp * 32 + lane;
    if (i < 128) {
      const int q = warp, tok = t0 + g + (q >> 1) * 8, e = e0 + 2 * t + (q & 1);
      float rs = scratch[i].x, rc = scratch[i].y;
#pragma unroll 4
      for (int j = 1; j < MMA_SLICES; ++j) join_pair(rs, rc, scratch[j * 128 + i].x, scratch[j * 128 + i].y);
      if (tok < T && e < E) {
        if (bias) add_pair(rs, rc, __ldg(bias + e));
        logits[(size_t)tok * E + e] = pair_value(rs, rc);
      }
    }
  }
}

// All logits, by every CTA of a grid (NW warps each, all threads call; NW need not be a multiple of
// the split).  scratch: ROUTE_SCRATCH of shared memory.
template <int NW>
__device__ __forceinline__ void router_logits(const uint16_t* x, const uint16_t* wr, const float* bias, int T, int H,
                                              int E, float* logits, float2* scratch, int cta, int ctas, int warp,
                                              int lane) {
  if (T > ROUTE_TOKENS) {
    router_logits_mma<NW>(x, wr, bias, T, H, E, logits, scratch, cta, ctas, warp, lane);
    return;
  }
  const int tasks = E, S = router_split(H), per = NW / S;
  const int slice = warp % S, mine = warp / S;
  for (int r = cta * per; r < tasks; r += ctas * per) {
    const int task = r + mine;
    const int e = task;
    float s = 0.0f, c = 0.0f;
    if (mine < per && task < tasks) {
      const uint16_t* row = wr + (size_t)e * H;
      if (T == 1) router_dot<1>(x, row, T, H, slice * 32 + lane, 32 * S, lane, s, c);
      else router_dot<ROUTE_TOKENS>(x, row, T, H, slice * 32 + lane, 32 * S, lane, s, c);
    }
    const int j = lane >> 3;       // this lane's token
    if (S > 1) {
      __syncthreads();
      if (mine < per && (lane & 7) == 0) scratch[warp * ROUTE_TOKENS + j] = make_float2(s, c);
      __syncthreads();
      if (slice != 0) continue;
      for (int q = 1; q < S; ++q) {
        const float2 v = scratch[(warp + q) * ROUTE_TOKENS + j];
        join_pair(s, c, v.x, v.y);
      }
    }
    if (mine < per && task < tasks && (lane & 7) == 0 && j < T) {
      if (bias) add_pair(s, c, __ldg(bias + e));
      logits[(size_t)j * E + e] = pair_value(s, c);
    }
  }
}

// A logit's place in the float order of route_key, from 1 on (0: no logit): that order has a value to spare, as -0 is
// keyed as +0.
__device__ __forceinline__ uint32_t logit_place(float v) {
  const uint32_t o = (uint32_t)(route_key(v, 0) >> 32);
  return o & 0x80000000u ? o : o + 1;
}
__device__ __forceinline__ float place_logit(uint32_t p) {
  return key_logit((unsigned long long)(p & 0x80000000u ? p : p - 1) << 32);
}

// One warp: the selection of route_topk_warp (its order, ties and weights, bit for bit) by warp-wide
// integer reductions; `load` reads a logit.
template <int EPL, class Load>
__device__ __forceinline__ void select_topk_warp(Load load, int E, int K, int lane, int& my_id, float& my_w) {
  uint32_t key[EPL];             // 0 when taken
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 32 * j;
    key[j] = e < E ? logit_place(load(e)) : 0u;
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
    const float v = place_logit(m);
    if (lane == k) {
      my_id = (int)id;
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
