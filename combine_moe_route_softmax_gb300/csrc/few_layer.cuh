// The whole MoE layer for a few tokens in one cooperative launch (moe_layer_few): router
// product (optional), top-k, gate/up + SwiGLU, down, fixed-order combine.  Included by
// one .cu file per weight format.  Internal header.
//
//   0  the router logits (with w_router), and for 4- and 8-bit weights the tokens as FP16 (below);
//      one grid barrier.  Every SM then selects the top-k itself (T x E logits from L2) and
//      lists the experts met with their columns.
//   1  tiles of 16 gate + 16 up rows of an expert: h = silu(g) * u of a (token, slot), kept as
//      two 16-bit terms h = hi + lo (one BF16 term would cost half of the layer's error
//      budget).
//   2  tiles of 32 output rows of an expert: y = W2 (hi + lo) in float32, hi and lo as two
//      columns of the same tensor instruction up to 4 tokens, two instructions above; the
//      SM that completes a row tile's last expert sums its rows over the slots in the
//      combine's order.
// All tiles, phase 1 then phase 2, expert by expert, are one queue.  A scheduler warp per SM takes
// the next tile when its workers are about to need it, so SMs stay level whatever the experts
// cost, and phase 2 begins on the first experts while phase 1 ends on the last: a tile of phase 2
// waits for its expert's h alone (its weights are loaded meanwhile).  Tiles in the queue are
// taken by running CTAs only, in order, so what a tile waits for is always being worked on.
//
// 16-bit operands: BF16 weights take BF16 activations.  E4M3 and 4-bit weights become FP16 in
// fewer instructions than BF16 (the conversion unit gives FP16 pairs), so their activations
// are FP16, scaled by a power of two per token (x) or per slot (h) that brings the largest
// value to 2^14: FP16 then holds every BF16 value above 2^-28 of the largest exactly, and the
// rest to 2^-39 of it.
#pragma once

#include "few.cuh"
#include "route_few.cuh"

namespace moe {
namespace few {

constexpr int WARPS = 16;
constexpr int THREADS = WARPS * 32;
constexpr int WORKERS = WARPS - 1;          // the last warp schedules
constexpr int STAGES = 2;
constexpr int PARTS_BYTES = 40 * 1024;      // slots of the joins
constexpr int kMaxSlots = kMaxTokens * kMaxTopK;
// one entry = up to COLS columns of one expert; at most one per routed slot, plus the shared ones
constexpr int kMaxEntries = kMaxSlots + kMaxTokens / COLS;
constexpr int kMaxWidth = 1 << 17;          // H and I
constexpr int SEQ = 128;                    // places of a CTA's tile sequence kept at a time
constexpr int AHEAD = 48;                   // units scheduled past the slowest worker's

struct LayerArgs {
  int T, H, I, E, K;
  int shared, tiled;
  const uint8_t *w13, *w2, *sw13, *sw2;
  const void *w13_s, *w2_s, *sw13_s, *sw2_s;
  const void *w13_z, *w2_z, *sw13_z, *sw2_z;
  const uint16_t* w_router;    // [E, H] or null
  const float* router_bias;    // [E] or null
  const float* logits_in;      // [T, E] or null
  const int32_t* num_tokens;
  float* logits;               // phase 0 writes [T, E]
  int32_t* topk_idx;
  float* topk_w;
  const uint16_t* x;
  uint16_t* out;
  int32_t* dev_status;
  // workspace, zero between launches
  uint32_t* ctl;               // barrier arrivals, barrier generation, next tile, CTAs done
  int32_t* tile_count;         // [H / 32] experts done of a row tile
  int32_t* entry_done;         // [kMaxEntries] row tiles done of an expert's h, plus one when it is ready
  uint32_t* h_max;             // [T*K + T] largest finite |h| of a slot, as bits
  // workspace
  uint16_t* x16;               // [T, H] FP16
  float* x_unit;               // [T] what 1 in x16 stands for
  float* h32;                  // [T*K + T, I]
  float* h_unit;               // [T*K + T]
  uint16_t *h_hi, *h_lo;       // [T*K + T, I]
  float* y;                    // [T*K + T, H]
};

struct LayerShared {
  int n_entries;
  int max_cols;
  int n1, n_all;               // tiles of phase 1, of both phases
  int tiles1, tiles2;          // row tiles of one expert
  Strides st[2];
  long long mat_bytes[2], mat_sc[2];   // one matrix's weights (bytes) and scales (elements)
  int seq[SEQ];                // tile numbers of the CTA's sequence
  int published;               // places filled
  int ready;                   // leading entries whose h is ready
  int use[WORKERS];            // unit each worker is at
  int go;
  float block[WARPS];
  short expert[kMaxEntries];   // E for the shared expert
  short first[kMaxEntries];    // first column in cols
  int ncols[kMaxEntries];
  short cols[kMaxSlots + kMaxTokens];   // slot ids t*K + k, or T*K + t for the shared expert
  short count[kMaxExperts];    // listing: slots of the expert so far
  short open[kMaxExperts];     // listing: its entry being filled
  short slot_entry[kMaxSlots];
  uint8_t slot_rank[kMaxSlots];
  short id[kMaxSlots];         // expert of each slot, -1 padding
  float w[kMaxSlots];
  uint8_t alive[kMaxTokens];   // token has a valid slot
  JoinShared join;
  float2 scratch[WARPS][ROUTE_TOKENS];
};

// Grid barrier in two halves (thread 0; the CTA synchronises around them).  The generation word
// is read before arriving, so only the arrival count has to be zero when the launch starts,
// and the last CTA leaves it zero.
__device__ __forceinline__ uint32_t barrier_arrive(uint32_t* bar) {
  uint32_t gen;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(gen) : "l"(bar + 1) : "memory");
  __threadfence();
  if (atomicAdd(&bar[0], 1u) == gridDim.x - 1) {
    bar[0] = 0;
    __threadfence();
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(bar + 1), "r"(gen + 1) : "memory");
  }
  return gen;
}
__device__ __forceinline__ bool barrier_wait(uint32_t* bar, uint32_t gen, int32_t* dev_status) {
  const bool ok = wait_for(
      [&] {
        uint32_t now;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(bar + 1) : "memory");
        return now != gen;
      },
      dev_status);
  __threadfence();
  return ok;
}

// The power of two that brings a positive finite float (bits m) to [2^14, 2^15), as far as float32
// can hold it and its inverse (2^-113 .. 2^120).
__device__ __forceinline__ float to_half_scale(uint32_t m) {
  const int e = (int)(m >> 23);                            // biased exponent, 0 for 0 and subnormals
  return __uint_as_float((uint32_t)min(127 + 14 - (e - 127), 127 + 120) << 23);
}
__device__ __forceinline__ uint16_t half_bits(float v) { return __half_as_ushort(__float2half_rn(v)); }

// Token t as FP16 (all threads of one CTA).
__device__ __forceinline__ void token_to_half(const LayerArgs& a, LayerShared& s, int t, int tid) {
  const uint4* src = reinterpret_cast<const uint4*>(a.x + (size_t)t * a.H);
  uint32_t m = 0;
  for (int i = tid; i < a.H / 8; i += THREADS) {
    const uint4 v = __ldg(src + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = (w[j] << 16) & 0x7fffffffu, hi = w[j] & 0x7fff0000u;
      if (lo < 0x7f800000u) m = max(m, lo);
      if (hi < 0x7f800000u) m = max(m, hi);
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) s.block[tid >> 5] = __uint_as_float(m);
  __syncthreads();
  m = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) m = max(m, __float_as_uint(s.block[i]));
  const float sc = to_half_scale(m);
  for (int i = tid; i < a.H / 8; i += THREADS) {
    const uint4 v = __ldg(src + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = half_bits(bf_lo(w[j]) * sc) | (uint32_t)half_bits(bf_hi(w[j]) * sc) << 16;
    reinterpret_cast<uint4*>(a.x16 + (size_t)t * a.H)[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (tid == 0) a.x_unit[t] = 1.0f / sc;
  __syncthreads();
}

// Lists the experts met -- the shared one, then in the order of their first slots -- and their
// columns (all threads; every CTA gets the same lists).  Loops are kept rolled: the code runs
// once per launch and is bound by fetching it.
__device__ __forceinline__ void list_entries(const LayerArgs& a, LayerShared& s) {
  const int n = a.T * a.K, tid = threadIdx.x, lane = tid & 31;
  for (int e = tid; e < a.E; e += THREADS) s.count[e] = 0;
  if (tid < a.T) {
    bool any = false;
#pragma unroll 1
    for (int k = 0; k < a.K; ++k) any |= s.id[tid * a.K + k] >= 0;
    s.alive[tid] = any;
  }
  __syncthreads();
  if (tid >= 32) return;
  int ent = 0, col = 0, most = 0;
  if (a.shared) {
    // first: with the most columns, its h takes longest to be ready
    const bool v = lane < a.T && s.alive[lane];
    const unsigned m = __ballot_sync(0xffffffffu, v);
    if (v) s.cols[__popc(m & lanemask_lt())] = (short)(n + lane);
    const int c = __popc(m);
#pragma unroll 1
    for (; col < c; col += COLS, ++ent) {
      if (lane == 0) {
        s.expert[ent] = (short)a.E;
        s.first[ent] = (short)col;
        s.ncols[ent] = min(COLS, c - col);
      }
      most = max(most, min(COLS, c - col));
    }
    col = c;
  }
  const int routed = ent;      // first routed entry
#pragma unroll 1
  for (int b = 0; b < n; b += 32) {
    const int i = b + lane;
    const int e = i < n ? s.id[i] : -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int rank = (e >= 0 ? s.count[e] : 0) + __popc(same & lanemask_lt());
    const bool lead = e >= 0 && rank % COLS == 0;        // first column of an entry
    const unsigned leads = __ballot_sync(0xffffffffu, lead);
    const int my_entry = ent + __popc(leads & lanemask_lt());
    const unsigned before = same & leads & (lanemask_lt() | 1u << lane);
    const int from_lane = __shfl_sync(0xffffffffu, my_entry, before ? 31 - __clz(before) : 0);
    const int entry = before ? from_lane : e >= 0 ? s.open[e] : 0;
    __syncwarp();
    if (lead) {
      s.expert[my_entry] = (short)e;
      s.ncols[my_entry] = 0;
    }
    __syncwarp();
    if (e >= 0) {
      s.slot_entry[i] = (short)entry;
      s.slot_rank[i] = (uint8_t)(rank % COLS);
      atomicAdd(&s.ncols[entry], 1);
      if ((same >> lane) == 1u) {                        // the expert's last slot of these 32
        s.count[e] = (short)(rank + 1);
        s.open[e] = (short)entry;
      }
    }
    __syncwarp();
    ent += __popc(leads);
  }
#pragma unroll 1
  for (int b = routed; b < ent; b += 32) {
    const int c = b + lane < ent ? s.ncols[b + lane] : 0;
    int sum = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    if (b + lane < ent) s.first[b + lane] = (short)(col + sum - c);
    col += __shfl_sync(0xffffffffu, sum, 31);
    most = max(most, (int)__reduce_max_sync(0xffffffffu, (unsigned)c));
  }
  __syncwarp();
#pragma unroll 1
  for (int i = lane; i < n; i += 32)
    if (s.id[i] >= 0) s.cols[s.first[s.slot_entry[i]] + s.slot_rank[i]] = (short)i;
  if (lane == 0) {
    s.n_entries = ent;
    s.max_cols = most;
  }
}

// The CTA's tile sequence as the stream's source of items.
template <int FMT, int GROUP>
struct LayerSrc {
  const LayerArgs& a;
  LayerShared& s;

  __device__ __forceinline__ int tile(int q) const {
    volatile int* published = &s.published;
    if (!wait_for([&] { return *published > q; }, a.dev_status)) return -1;
    __threadfence_block();
    return s.seq[q & (SEQ - 1)];
  }
  __device__ __forceinline__ bool down(int tile_) const { return tile_ >= s.n1; }
  __device__ __forceinline__ const Strides& strides(int tile_) const { return s.st[down(tile_)]; }
  __device__ __forceinline__ bool zeros() const { return a.w13_z != nullptr; }
  // tile number -> entry and row tile
  __device__ __forceinline__ void split(int tile_, int& entry, int& row) const {
    const int n = down(tile_) ? s.tiles2 : s.tiles1, i = down(tile_) ? tile_ - s.n1 : tile_;
    entry = i / n;
    row = i - entry * n;
  }
  __device__ __forceinline__ Tile where(int tile_, int s0) const {
    const bool d = down(tile_);
    const Strides& st = s.st[d];
    int entry, row;
    split(tile_, entry, row);
    const int e = s.expert[entry];
    const bool sh = e == a.E;
    const uint8_t* w = d ? (sh ? a.sw2 : a.w2) : (sh ? a.sw13 : a.w13);
    const long long m = sh ? 0 : e;
    w += m * s.mat_bytes[d];
    Tile r;
    r.sc = r.zp = nullptr;
    if constexpr (FMT == F_W4) {
      constexpr int NG = Format<FMT, GROUP>::NG;
      const void* sc = d ? (sh ? a.sw2_s : a.w2_s) : (sh ? a.sw13_s : a.w13_s);
      const void* zp = d ? (sh ? a.sw2_z : a.w2_z) : (sh ? a.sw13_z : a.w13_z);
      const long long blk = (long long)row * (d ? 2 : 1) * st.nsl + s0;
      w += blk * 2048;
      r.sc = static_cast<const uint32_t*>(sc) + m * s.mat_sc[d] + blk * 8 * NG;
      if (zp) r.zp = static_cast<const uint16_t*>(zp) + m * s.mat_sc[d] + blk * 8 * NG;
    } else {
      const long long bytes = FMT == F_BF16 ? 2ll * st.k : st.k;
      const int r0 = row * (d ? 32 : 16);
      if (a.tiled)
        w += (long long)(r0 >> 7) * (bytes * 128) + (long long)s0 * 16384 + (r0 & 127) * 128;
      else
        w += r0 * bytes + (long long)s0 * 128;
      if constexpr (FMT == F_E4M3) {
        const void* sc = d ? (sh ? a.sw2_s : a.w2_s) : (sh ? a.sw13_s : a.w13_s);
        r.sc = static_cast<const float*>(sc) + m * s.mat_sc[d] + (long long)(r0 >> 7) * (st.k / 128) + s0;
      }
    }
    r.w = w;
    return r;
  }
};

// Strides and cuts of both phases (one thread).
template <int FMT, int GROUP>
__device__ __forceinline__ void plan_phases(const LayerArgs& a, LayerShared& s) {
#pragma unroll 1
  for (int d = 0; d < 2; ++d) {
    Strides& st = s.st[d];
    const int rows = d ? a.H : 2 * a.I, half_rows = d ? 16 : a.I;
    st.k = d ? a.I : a.H;
    if constexpr (FMT == F_W4) {
      st.nsl = (int)w4_slices(st.k);
      st.step = 2048;
      st.pitch = 128;
      st.half = (long long)(half_rows / 16) * st.nsl * 2048;
      st.sc_half = (long long)(half_rows / 16) * st.nsl * 8 * Format<FMT, GROUP>::NG;
      s.mat_bytes[d] = (long long)(rows / 16) * st.nsl * 2048;
      s.mat_sc[d] = (long long)(rows / 16) * st.nsl * 8 * Format<FMT, GROUP>::NG;
    } else {
      const long long bytes = FMT == F_BF16 ? 2ll * st.k : st.k;
      st.nsl = (int)(bytes / 128);
      st.step = a.tiled ? 16384 : 128;
      st.pitch = a.tiled ? 128 : bytes;
      // 16 rows on inside a 128-row box, or I (a multiple of 128) rows on in either layout
      st.half = d ? 16 * st.pitch : a.I * bytes;
      st.sc_half = d ? 0 : (long long)(a.I / 128) * (st.k / 128);
      s.mat_bytes[d] = rows * bytes;
      s.mat_sc[d] = (long long)(rows / 128) * (st.k / 128);
    }
    const int n = rows / 32 * s.n_entries;
    st.cut(WORKERS, n <= (int)gridDim.x);
  }
  s.tiles1 = a.I / 16;
  s.tiles2 = a.H / 32;
  s.n1 = s.n_entries * s.tiles1;
  s.n_all = s.n1 + s.n_entries * s.tiles2;
  s.published = 0;
  s.ready = 0;
}

// The scheduler warp: keeps the sequence AHEAD units past the slowest worker, and passes on which
// entries' h are ready.  The first two tiles of a CTA are its own, the rest come off the queue.
__device__ __forceinline__ void schedule(const LayerArgs& a, LayerShared& s, int h_ready, int lane) {
  volatile int* use = s.use;
  int q = 0, units = 0, ready = 0;
  bool end = false;
  unsigned long long t0 = clock_ns();
  while (!end || ready < s.n_entries) {
    bool moved = false;
    if (ready < s.n_entries) {
      const int e = ready + lane;
      int v = 0;
      if (e < s.n_entries) asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(a.entry_done + e) : "memory");
      const unsigned m = __ballot_sync(0xffffffffu, e < s.n_entries && v == h_ready);
      const int n = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
      if (n > 0) {
        ready += n;
        __threadfence();
        __syncwarp();
        if (lane == 0) *static_cast<volatile int*>(&s.ready) = ready;
        moved = true;
      }
    }
    if (!end) {
      const int slowest = __reduce_min_sync(0xffffffffu, lane < WORKERS ? use[lane] : 0x7fffffff);
      if (units < slowest + AHEAD) {
        int t = 0;
        if (lane == 0) {
          t = q < 2 ? (int)(blockIdx.x + q * gridDim.x) : (int)(2 * gridDim.x + atomicAdd(&a.ctl[2], 1u));
          if (t >= s.n_all) t = -1;
          s.seq[q & (SEQ - 1)] = t;
          __threadfence_block();
          *static_cast<volatile int*>(&s.published) = q + 1;
        }
        t = __shfl_sync(0xffffffffu, t, 0);
        end = t < 0;
        if (!end) units += s.st[t >= s.n1].parts;
        ++q;
        moved = true;
      }
    }
    if (moved) {
      t0 = clock_ns();
    } else if (__any_sync(0xffffffffu, clock_ns() - t0 > TIMEOUT_NS)) {   // nothing for two seconds: let the workers go
      if (lane == 0) {
        if (a.dev_status) atomicOr(a.dev_status, MOE_DEV_PIPELINE_TIMEOUT);
        s.seq[q & (SEQ - 1)] = -1;
        __threadfence_block();
        if (!end) *static_cast<volatile int*>(&s.published) = q + 1;
        *static_cast<volatile int*>(&s.ready) = s.n_entries;
      }
      return;
    }
  }
}

// Phase 1's result for one tile: h of 16 intermediate rows; two BF16 terms, or float32 with the
// largest magnitude of each slot kept (its FP16 terms are made when the expert is complete).
template <bool HALF, int NT>
__device__ __forceinline__ void store_h(const LayerArgs& a, const LayerShared& s, const Sums<NT>& sums, int entry,
                                        int tile, int lane) {
  const int g = lane >> 2, t = lane & 3, nc = s.ncols[entry], c0 = s.first[entry];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = n * 8 + 2 * t + j;
      const int slot = c < nc ? s.cols[c0 + c] : -1;
      float unit = 1.0f;
      if (HALF && slot >= 0) unit = __ldcg(&a.x_unit[slot < a.T * a.K ? slot / a.K : slot - a.T * a.K]);
      uint32_t most = 0;
#pragma unroll
      for (int i = j; i < 4; i += 2) {
        const float gate = sums.v[n][0][i] * unit, up = sums.v[n][1][i] * unit;
        const float h = gate / (1.0f + expf(-gate)) * up;
        const size_t o = (size_t)slot * a.I + tile * 16 + g + (i >> 1) * 8;
        if (slot >= 0) {
          if (HALF) {
            __stcg(&a.h32[o], h);
            const uint32_t b = __float_as_uint(h) & 0x7fffffffu;
            if (b < 0x7f800000u) most = max(most, b);
          } else {
            const uint16_t hi = f32_to_bf16(h);
            a.h_hi[o] = hi;
            a.h_lo[o] = f32_to_bf16((hi & 0x7fffu) >= 0x7f80u ? 0.0f : h - bf16_to_f32(hi));   // inf, NaN: hi alone
          }
        }
      }
      if (HALF) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        if (g == 0 && slot >= 0) atomicMax(&a.h_max[slot], most);
      }
    }
}

// The h of a complete entry as two FP16 terms per value (one warp).
__device__ __forceinline__ void entry_to_half(const LayerArgs& a, const LayerShared& s, int entry, int lane) {
#pragma unroll 1
  for (int c = 0; c < s.ncols[entry]; ++c) {
    const int slot = s.cols[s.first[entry] + c];
    const float sc = to_half_scale(__ldcg(&a.h_max[slot]));
    const float4* src = reinterpret_cast<const float4*>(a.h32 + (size_t)slot * a.I);
    uint2* hi = reinterpret_cast<uint2*>(a.h_hi + (size_t)slot * a.I);
    uint2* lo = reinterpret_cast<uint2*>(a.h_lo + (size_t)slot * a.I);
#pragma unroll 4
    for (int i = lane; i < a.I / 4; i += 32) {
      const float4 v = __ldcg(src + i);
      const float f[4] = {v.x * sc, v.y * sc, v.z * sc, v.w * sc};
      uint16_t p[4], r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = half_bits(f[j]);
        r[j] = (p[j] & 0x7fffu) >= 0x7c00u ? 0 : half_bits(f[j] - __half2float(__ushort_as_half(p[j])));
      }
      hi[i] = make_uint2(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16);
      lo[i] = make_uint2(r[0] | (uint32_t)r[1] << 16, r[2] | (uint32_t)r[3] << 16);
    }
    __syncwarp();
    if (lane == 0) {
      a.h_unit[slot] = 1.0f / sc;
      a.h_max[slot] = 0;
    }
  }
}

// Phase 2's result for one (row tile, expert): y rows; up to 4 columns come as hi and lo columns
// of one group (hi in columns 0-3, lanes t = 0, 1; lo in 4-7, t = 2, 3).
template <bool HALF, int NT>
__device__ __forceinline__ void store_y(const LayerArgs& a, const LayerShared& s, Sums<NT>& sums, int entry, int tile,
                                        int lane) {
  const int g = lane >> 2, t = lane & 3, nc = s.ncols[entry], c0 = s.first[entry];
  if (nc <= 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) sums.v[0][h][i] += __shfl_down_sync(0xffffffffu, sums.v[0][h][i], 2);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = n * 8 + 2 * t + (i & 1);
      if (c < nc) {
        const int slot = s.cols[c0 + c];
        const float unit = HALF ? __ldcg(&a.h_unit[slot]) : 1.0f;
        float* p = a.y + (size_t)slot * a.H + tile * 32 + g + (i >> 1) * 8;
        __stcg(p, sums.v[n][0][i] * unit);
        __stcg(p + 16, sums.v[n][1][i] * unit);
      }
    }
}

// One row tile's outputs, lane = row, in the combine's order: ascending slot, float32 product and
// sum from +0, the shared row last, one BF16 rounding.
__device__ __forceinline__ void combine_tile(const LayerArgs& a, const LayerShared& s, int tile, int lane) {
  const int row = tile * 32 + lane;
#pragma unroll 2
  for (int t = 0; t < a.T; ++t) {
    float acc = 0.0f;
    const bool sh = a.shared && s.alive[t];
    const float sv = sh ? __ldcg(a.y + (size_t)(a.T * a.K + t) * a.H + row) : 0.0f;
#pragma unroll 1
    for (int k0 = 0; k0 < a.K; k0 += 8) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = k0 + j;
        v[j] = k < a.K && s.id[t * a.K + k] >= 0 ? __ldcg(&a.y[(size_t)(t * a.K + k) * a.H + row]) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = k0 + j;
        if (k < a.K && s.id[t * a.K + k] >= 0) acc = __fadd_rn(acc, __fmul_rn(v[j], s.w[t * a.K + k]));
      }
    }
    if (sh) acc = __fadd_rn(acc, sv);
    a.out[(size_t)t * a.H + row] = f32_to_bf16(acc);
  }
}

template <int FMT, int GROUP>
using LayerStream = Stream<FMT, GROUP, FMT != F_BF16, STAGES, WORKERS, LayerSrc<FMT, GROUP>>;

// The unit at in.usec with NT column groups: columns, sums, join, result.
template <int FMT, int GROUP, int NT, int PASSES>
__device__ __forceinline__ void do_unit(const LayerSrc<FMT, GROUP>& src, LayerStream<FMT, GROUP>& in, bool down,
                                        int entry, int row, float4* parts, int slots, int stride) {
  constexpr bool HALF = FMT != F_BF16;
  const LayerArgs& a = src.a;
  LayerShared& s = src.s;
  const int lane = in.lane, g = lane >> 2;
  const int nc = s.ncols[entry], c0 = s.first[entry];
  const uint16_t* x[PASSES][NT];
#pragma unroll
  for (int p = 0; p < PASSES; ++p)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      x[p][i] = nullptr;
      const bool pairs = down && PASSES == 1;              // hi and lo as columns of one group
      const int c = pairs ? (g & 3) : i * 8 + g;
      if (c < nc) {
        const int slot = s.cols[c0 + c];
        if (!down)
          x[p][i] = (HALF ? a.x16 : a.x) + (size_t)(slot < a.T * a.K ? slot / a.K : slot - a.T * a.K) * a.H;
        else
          x[p][i] = ((pairs ? g >= 4 : p == 1) ? a.h_lo : a.h_hi) + (size_t)slot * a.I;
      }
    }
  const Strides& st = s.st[down];
  Sums<NT> sums;
  in.template run<NT, PASSES>(sums, st, x);
  if (!join<NT>(sums, s.join, parts, slots, stride, in.usec.u, in.usec.u - in.usec.part, st.parts, lane, a.dev_status))
    return;
  if (!down) {
    store_h<HALF, NT>(a, s, sums, entry, row, lane);
    __threadfence();
    __syncwarp();
    int old = 0;
    if (lane == 0) old = atomicAdd(&a.entry_done[entry], 1);
    if (HALF && __shfl_sync(0xffffffffu, old, 0) == s.tiles1 - 1) {
      __threadfence();
      entry_to_half(a, s, entry, lane);
      __threadfence();
      __syncwarp();
      if (lane == 0) atomicAdd(&a.entry_done[entry], 1);
    }
    return;
  }
  store_y<HALF, NT>(a, s, sums, entry, row, lane);
  __threadfence();
  __syncwarp();
  int old = 0;
  if (lane == 0) old = atomicAdd(&a.tile_count[row], 1);
  if (__shfl_sync(0xffffffffu, old, 0) != s.n_entries - 1) return;
  __threadfence();
  if (lane == 0) a.tile_count[row] = 0;
  combine_tile(a, s, row, lane);
}

template <int FMT, int GROUP>
__global__ void __launch_bounds__(THREADS, 1) layer_kernel(const LayerArgs a) {
  constexpr bool HALF = FMT != F_BF16;
  __shared__ LayerShared s;
  extern __shared__ __align__(128) uint8_t rings[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.T * a.K;
  const bool sync = HALF || a.w_router;
  uint32_t gen = 0;
  if (HALF)
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) token_to_half(a, s, t, tid);
  if (a.w_router)
    router_logits<WARPS>(a.x, a.w_router, a.router_bias, a.T, a.H, a.E, a.logits, s.scratch, blockIdx.x, gridDim.x,
                         warp, lane);
  if (sync) {
    __syncthreads();
    if (tid == 0) gen = barrier_arrive(a.ctl);
  }
  if (a.w_router) {
    if (tid == 0) s.go = barrier_wait(a.ctl, gen, a.dev_status);
    __syncthreads();
  }
  const float* logits = a.w_router ? a.logits : a.logits_in;
  if (logits) {
    const int nt = a.num_tokens ? *a.num_tokens : a.T;
    for (int t = warp; t < a.T; t += WARPS) {
      int id = -1;
      float w = 0.0f;
      if (t < nt) select_topk(logits + (size_t)t * a.E, a.E, a.K, lane, id, w);
      if (lane < a.K) {
        s.id[t * a.K + lane] = (short)id;
        s.w[t * a.K + lane] = w;
        if (blockIdx.x == 0) {
          a.topk_idx[t * a.K + lane] = id;
          a.topk_w[t * a.K + lane] = w;
        }
      }
    }
  } else {
    for (int i = tid; i < n; i += THREADS) {
      int id = a.topk_idx[i];
      if (id < -1 || id >= a.E) {
        if (blockIdx.x == 0 && a.dev_status) atomicOr(a.dev_status, MOE_DEV_BAD_EXPERT);
        id = -1;
      }
      s.id[i] = (short)id;
      s.w[i] = a.topk_w[i];
    }
  }
  __syncthreads();
  list_entries(a, s);
  if (tid == 0) {
    plan_phases<FMT, GROUP>(a, s);
    if (!sync) s.go = 1;
    else if (!a.w_router) s.go = barrier_wait(a.ctl, gen, a.dev_status);
  }
  join_init(s.join);
  if (tid < WORKERS) s.use[tid] = tid;
  __syncthreads();
  if (!s.go) return;
  if (s.n_entries == 0) {   // no valid slot in the batch: every output is +0
    for (size_t i = (size_t)blockIdx.x * THREADS + tid; i < (size_t)a.T * a.H; i += (size_t)gridDim.x * THREADS)
      a.out[i] = 0;
    return;
  }
  if (warp == WORKERS) {
    schedule(a, s, s.tiles1 + (HALF ? 1 : 0), lane);
  } else {
    constexpr int RING = STAGES * Format<FMT, GROUP>::STAGE;
    float4* parts = reinterpret_cast<float4*>(rings + WORKERS * RING);
    const int stride = s.max_cols <= 8 ? 64 : 128;       // a slot is 1 KB for each 8 columns
    const int slots = min(MAX_SLOTS, PARTS_BYTES / (stride * 16));
    const LayerSrc<FMT, GROUP> src{a, s};
    LayerStream<FMT, GROUP> in(src, rings + warp * RING, warp, lane);
    volatile int* ready = &s.ready;
    while (in.usec.tile >= 0) {
      if (lane == 0) *static_cast<volatile int*>(&s.use[warp]) = in.usec.u;
      const bool down = src.down(in.usec.tile);
      int entry, row;
      src.split(in.usec.tile, entry, row);
      const int nc = s.ncols[entry];
      if (!down) {
        if (nc <= 8) do_unit<FMT, GROUP, 1, 1>(src, in, down, entry, row, parts, slots, stride);
        else do_unit<FMT, GROUP, 2, 1>(src, in, down, entry, row, parts, slots, stride);
      } else {
        wait_for([&] { return *ready > entry; }, a.dev_status);
        __threadfence_block();
        __syncwarp();
        if (nc <= 4) do_unit<FMT, GROUP, 1, 1>(src, in, down, entry, row, parts, slots, stride);
        else if (nc <= 8) do_unit<FMT, GROUP, 1, 2>(src, in, down, entry, row, parts, slots, stride);
        else do_unit<FMT, GROUP, 2, 2>(src, in, down, entry, row, parts, slots, stride);
      }
      in.hop(in.usec);
    }
    cp_wait<0>();
    if (lane == 0) *static_cast<volatile int*>(&s.use[warp]) = 0x7fffff00;
  }
  // the last CTA leaves the counters zero for the next launch
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s.go = atomicAdd(&a.ctl[3], 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s.go) return;
  __threadfence();
  for (int i = tid; i < s.n_entries; i += THREADS) a.entry_done[i] = 0;
  if (tid < 2) a.ctl[2 + tid] = 0;
}

template <int FMT, int GROUP>
cudaError_t launch_layer(const LayerArgs& a, cudaStream_t stream) {
  constexpr int smem = WORKERS * STAGES * Format<FMT, GROUP>::STAGE + PARTS_BYTES;
  static std::atomic<unsigned long long> done{0};
  if (!once_per_device(done, [] {
        return cudaFuncSetAttribute(layer_kernel<FMT, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) ==
               cudaSuccess;
      }))
    return cudaErrorUnknown;
  void* args[] = {const_cast<LayerArgs*>(&a)};
  return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(&layer_kernel<FMT, GROUP>), dim3(num_sms()),
                                     dim3(THREADS), args, smem, stream);
}

cudaError_t launch_layer_bf16(const LayerArgs& a, cudaStream_t stream);
cudaError_t launch_layer_e4m3(const LayerArgs& a, cudaStream_t stream);
cudaError_t launch_layer_w4(const LayerArgs& a, int group, cudaStream_t stream);

}  // namespace few
}  // namespace moe
