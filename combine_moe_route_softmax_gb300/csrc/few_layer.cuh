// The whole MoE layer for a few tokens in one cooperative launch (moe_layer_few): router
// product (optional), top-k, gate/up + SwiGLU, down, fixed-order combine.  Included by
// one .cu file per weight format.  Internal header.
//
// Phases, with a grid barrier between them:
//   0  (only with w_router) the router logits, one warp per (expert, few tokens);
//   1  every SM selects the top-k itself (T x E logits from L2) and lists the experts met
//      with their columns; then items (expert, 16 gate + 16 up rows, K slice):
//      h = silu(g) * u of a (token, slot), kept as two BF16 terms h = hi + lo (16 bits of
//      mantissa: one BF16 term would cost half of the layer's error budget);
//   2  items (32 output rows, expert, K slice): y = W2 (hi + lo), hi and lo as two columns of
//      the same tensor instruction, y in float32; the warp that completes a row tile's last
//      expert sums its rows over the slots in the combine's order.
// The workers (few.cuh) run one stream of items per phase; the first item of phase 2 is
// loaded before the barrier.
#pragma once

#include "few.cuh"
#include "route_few.cuh"

namespace moe {
namespace few {

constexpr int kMaxSlots = kMaxTokens * kMaxTopK;
// one entry = up to COLS columns of one expert; at most one per routed slot, plus the shared ones
constexpr int kMaxEntries = kMaxSlots + kMaxTokens / COLS;

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
  float* logits;               // phase 0 writes, phase 1 reads [T, E]
  int32_t* topk_idx;
  float* topk_w;
  const uint16_t* x;
  uint16_t* out;
  int32_t* dev_status;
  // workspace
  uint32_t* bar;               // {arrivals, generation}
  int32_t* part_count;         // [workers]
  int32_t* tile_count;         // [H / 32]
  uint16_t *h_hi, *h_lo;       // [T*K + T, I]
  float* y;                    // [T*K + T, H]
  float* part;                 // [workers][2][PART_FLOATS]
};

struct LayerShared {
  int n_entries;
  int routed;                  // valid routed slots
  int expert[kMaxEntries];     // E for the shared expert
  int first[kMaxEntries];      // first column in cols
  int ncols[kMaxEntries];
  int cols[kMaxSlots + kMaxTokens];   // slot ids t*K + k, or T*K + t for the shared expert
  int count[kMaxExperts];
  short id[kMaxSlots];         // expert of each slot, -1 padding
  float w[kMaxSlots];
  uint8_t alive[kMaxTokens];   // token has a valid slot
};

// All CTAs of the launch arrive; false if the wait ran out (the status bit is then set).
// The generation word is read before arriving, so only the arrival count has to be zero when
// the launch starts, and the last CTA leaves it zero.
__device__ __forceinline__ bool grid_barrier(uint32_t* bar, int32_t* dev_status, int* ok) {
  __syncthreads();
  if (threadIdx.x == 0) {
    *ok = 1;
    uint32_t gen, now;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(gen) : "l"(bar + 1) : "memory");
    __threadfence();
    if (atomicAdd(&bar[0], 1u) == gridDim.x - 1) {
      bar[0] = 0;
      __threadfence();
      asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(bar + 1), "r"(gen + 1) : "memory");
    } else {
      unsigned long long t0 = 0, t1;
      for (;;) {
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(bar + 1) : "memory");
        if (now != gen) break;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t1));
        if (t0 == 0) t0 = t1;
        if (t1 - t0 > TIMEOUT_NS) {
          if (dev_status) atomicOr(dev_status, MOE_DEV_PIPELINE_TIMEOUT);
          *ok = 0;
          break;
        }
      }
    }
    __threadfence();
  }
  __syncthreads();
  return *ok != 0;
}

// Lists the experts met and their columns (all threads; every CTA gets the same lists).
__device__ __forceinline__ void list_entries(const LayerArgs& a, LayerShared& s) {
  const int n = a.T * a.K, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int e = tid; e < a.E; e += THREADS) s.count[e] = 0;
  if (tid < a.T) {
    bool any = false;
    for (int k = 0; k < a.K; ++k) any |= s.id[tid * a.K + k] >= 0;
    s.alive[tid] = any;
  }
  __syncthreads();
  if (warp != 0) return;
  // rank of each slot within its expert, 32 slots at a time; kept in cols for the moment
  for (int b = 0; b < n; b += 32) {
    const int i = b + lane;
    const int e = i < n ? s.id[i] : -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int before = __popc(same & lanemask_lt());
    const int base = e >= 0 ? s.count[e] : 0;
    __syncwarp();
    if (e >= 0 && before == 0) s.count[e] = base + __popc(same);
    __syncwarp();
    if (i < n) s.first[i] = base + before;   // first is rewritten below, after every rank is used
  }
  // columns and entries of each expert, ascending
  int col = 0, ent = 0;
  int my_first[kMaxSlots / 32];
#pragma unroll
  for (int j = 0; j < kMaxSlots / 32; ++j)
    if (j * 32 < n) my_first[j] = j * 32 + lane < n ? s.first[j * 32 + lane] : 0;
  __syncwarp();
  for (int b = 0; b < a.E; b += 32) {
    const int e = b + lane;
    const int c = e < a.E ? s.count[e] : 0;
    const int ne = (c + COLS - 1) / COLS;
    int pc = c, pe = ne;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, pc, o), v = __shfl_up_sync(0xffffffffu, pe, o);
      if (lane >= o) { pc += u; pe += v; }
    }
    const int c0 = col + pc - c, e0 = ent + pe - ne;
    for (int j = 0; j < ne; ++j) {
      s.expert[e0 + j] = e;
      s.first[e0 + j] = c0 + j * COLS;
      s.ncols[e0 + j] = min(COLS, c - j * COLS);
    }
    if (e < a.E) s.count[e] = c0;   // now: the expert's first column
    col += __shfl_sync(0xffffffffu, pc, 31);
    ent += __shfl_sync(0xffffffffu, pe, 31);
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < kMaxSlots / 32; ++j) {
    const int i = j * 32 + lane;
    if (i < n && s.id[i] >= 0) s.cols[s.count[s.id[i]] + my_first[j]] = i;
  }
  const int routed = col;
  if (a.shared) {
    const bool v = lane < a.T && s.alive[lane];
    const unsigned m = __ballot_sync(0xffffffffu, v);
    if (v) s.cols[col + __popc(m & lanemask_lt())] = n + lane;
    const int c = __popc(m);
    for (int j = 0; j * COLS < c; ++j) {
      if (lane == 0) {
        s.expert[ent] = a.E;
        s.first[ent] = col + j * COLS;
        s.ncols[ent] = min(COLS, c - j * COLS);
      }
      ++ent;
    }
  }
  if (lane == 0) {
    s.n_entries = ent;
    s.routed = routed;
  }
}

// Phase 1 or 2 of the layer as a stream of items.
template <int FMT, int GROUP>
struct Phase {
  const LayerArgs& a;
  const LayerShared& s;
  const bool down;
  Strides st;
  int tiles;                   // row tiles of one matrix
  long long F;                 // items of the phase
  int W, me, lane;
  long long f1;                // end of this worker's run
  long long mat_bytes, mat_sc; // one matrix's weights (bytes) and scales (elements of its lane pointer)

  __device__ __forceinline__ Phase(const LayerArgs& a_, const LayerShared& s_, bool down_, int warp, int lane_)
      : a(a_), s(s_), down(down_), lane(lane_) {
    const int rows = down ? a.H : 2 * a.I;
    const int half_rows = down ? 16 : a.I;
    st.k = down ? a.I : a.H;
    tiles = rows / 32;
    if constexpr (FMT == F_W4) {
      st.nsl = (int)w4_slices(st.k);
      st.step = 2048;
      st.row8 = 1024;
      st.half = (long long)(half_rows / 16) * st.nsl * 2048;
      st.sc_half = (long long)(half_rows / 16) * st.nsl * 8 * Item<FMT, GROUP>::NG;
      mat_bytes = (long long)(rows / 16) * st.nsl * 2048;
      mat_sc = (long long)(rows / 16) * st.nsl * 8 * Item<FMT, GROUP>::NG;
    } else {
      const long long pitch = FMT == F_BF16 ? 2ll * st.k : st.k;
      st.nsl = (int)(pitch / 128);
      st.step = a.tiled ? 16384 : 128;
      st.row8 = a.tiled ? 1024 : 8 * pitch;
      // 16 rows on inside a 128-row box, or I (a multiple of 128) rows on in either layout
      st.half = down ? (a.tiled ? 2048 : 16 * pitch) : a.I * pitch;
      st.sc_half = down ? 0 : (long long)(a.I / 128) * (st.k / 128);
      mat_bytes = rows * pitch;
      mat_sc = (long long)(rows / 128) * (st.k / 128);
    }
    F = (long long)s.n_entries * tiles * st.nsl;
    W = workers_for(F, gridDim.x * WARPS, 2);
    me = F > 0 ? my_worker(W, blockIdx.x, gridDim.x, warp) : -1;
    f1 = me >= 0 ? run_start(F, me + 1, W) : 0;
  }
  __device__ __forceinline__ void split(long long f, int& entry, int& tile, int& s0) const {
    const long long q = f / st.nsl;
    s0 = (int)(f - q * st.nsl);
    if (down) {
      tile = (int)(q / s.n_entries);
      entry = (int)(q - (long long)tile * s.n_entries);
    } else {
      entry = (int)(q / tiles);
      tile = (int)(q - (long long)entry * tiles);
    }
  }
  // the tile at item f, as far as this worker's run goes
  __device__ __forceinline__ Tile tile_at(long long f, int entry, int tile, int s0) const {
    Tile r;
    r.s0 = s0;
    r.n = (int)min((long long)(st.nsl - s0), f1 - f);
    const int e = s.expert[entry];
    const bool sh = e == a.E;
    const uint8_t* w = down ? (sh ? a.sw2 : a.w2) : (sh ? a.sw13 : a.w13);
    const void* sc = down ? (sh ? a.sw2_s : a.w2_s) : (sh ? a.sw13_s : a.w13_s);
    const void* zp = down ? (sh ? a.sw2_z : a.w2_z) : (sh ? a.sw13_z : a.w13_z);
    const long long m = sh ? 0 : e;
    const int g = lane >> 2, t = lane & 3;
    w += m * mat_bytes;
    r.sc = r.zp = nullptr;
    if constexpr (FMT == F_W4) {
      const long long blk = (long long)tile * (down ? 2 : 1) * st.nsl + s0;
      w += blk * 2048 + lane * 32;
      r.sc = static_cast<const uint32_t*>(sc) + m * mat_sc + (blk * 8 + g) * Item<FMT, GROUP>::NG;
      if (zp) r.zp = static_cast<const uint16_t*>(zp) + m * mat_sc + (blk * 8 + g) * Item<FMT, GROUP>::NG;
    } else {
      const long long pitch = FMT == F_BF16 ? 2ll * st.k : st.k;
      const int r0 = tile * (down ? 32 : 16);
      if (a.tiled)
        w += (long long)(r0 >> 7) * (pitch * 128) + (long long)s0 * 16384 + ((r0 & 127) + g) * 128 + t * 32;
      else
        w += (r0 + g) * pitch + (long long)s0 * 128 + t * 32;
      if constexpr (FMT == F_E4M3)
        r.sc = static_cast<const float*>(sc) + m * mat_sc + (long long)(r0 >> 7) * (st.k / 128) + s0;
    }
    r.w = w;
    return r;
  }
};

// Phase 1's result for one tile: h of 16 intermediate rows, two BF16 terms per value.
template <int NT>
__device__ __forceinline__ void store_h(const LayerArgs& a, const LayerShared& s, const Sums<NT>& sums, int entry,
                                        int tile, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = n * 8 + 2 * t + (i & 1);
      if (c < s.ncols[entry]) {
        const float gate = sums.v[n][0][i], up = sums.v[n][1][i];
        const float h = gate / (1.0f + expf(-gate)) * up;
        const uint16_t hi = f32_to_bf16(h);
        const float lo = (hi & 0x7fffu) >= 0x7f80u ? 0.0f : h - bf16_to_f32(hi);   // inf, NaN: hi alone
        const size_t o = (size_t)s.cols[s.first[entry] + c] * a.I + tile * 16 + g + (i >> 1) * 8;
        a.h_hi[o] = hi;
        a.h_lo[o] = f32_to_bf16(lo);
      }
    }
}

// Phase 2's result for one (row tile, expert): y rows, hi and lo columns added.
template <int NT>
__device__ __forceinline__ void store_y(const LayerArgs& a, const LayerShared& s, Sums<NT>& sums, int entry, int tile,
                                        int lane) {
  const int g = lane >> 2, t = lane & 3, nc = s.ncols[entry];
  if constexpr (NT == 1) {   // hi in columns 0-3 (lanes t = 0, 1), lo in 4-7 (t = 2, 3)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) sums.v[0][h][i] += __shfl_down_sync(0xffffffffu, sums.v[0][h][i], 2);
    if (t >= 2) return;
  } else {
#pragma unroll
    for (int n = 0; n < NT / 2; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums.v[n][h][i] += sums.v[n + NT / 2][h][i];
  }
#pragma unroll
  for (int n = 0; n < (NT + 1) / 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = n * 8 + 2 * t + (i & 1);
      if (c < nc) {
        float* p = a.y + (size_t)s.cols[s.first[entry] + c] * a.H + tile * 32 + g + (i >> 1) * 8;
        __stcg(p, sums.v[n][0][i]);
        __stcg(p + 16, sums.v[n][1][i]);
      }
    }
}

// One row tile's outputs: the combine's order -- ascending slot, float32 product and sum from
// +0, the shared row last, one BF16 rounding.
__device__ __forceinline__ void combine_tile(const LayerArgs& a, const LayerShared& s, int tile, int lane) {
  const int row = tile * 32 + lane;
  for (int t = 0; t < a.T; ++t) {
    float acc = 0.0f;
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
    if (a.shared && s.alive[t]) acc = __fadd_rn(acc, __ldcg(&a.y[(size_t)(a.T * a.K + t) * a.H + row]));
    a.out[(size_t)t * a.H + row] = f32_to_bf16(acc);
  }
}

// One tile of a phase with NT column groups: columns, sums, join, result.  True if this warp
// completed the tile.
template <int FMT, int GROUP, int NT>
__device__ __forceinline__ bool do_tile(const Phase<FMT, GROUP>& ph, Item<FMT, GROUP>& it, const Tile& cur,
                                        const Tile& next, int entry, int tile, long long f) {
  const LayerArgs& a = ph.a;
  const LayerShared& s = ph.s;
  const int lane = ph.lane, g = lane >> 2, t = lane & 3;
  const int nc = s.ncols[entry], c0 = s.first[entry];
  const uint16_t* x[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    x[n] = nullptr;
    if (!ph.down) {
      const int c = n * 8 + g;
      if (c < nc) {
        const int slot = s.cols[c0 + c];
        const int tok = slot < a.T * a.K ? slot / a.K : slot - a.T * a.K;
        x[n] = a.x + (size_t)tok * a.H;
      }
    } else {
      // the lower half of the columns is hi, the upper half lo
      const int c = NT == 1 ? (g & 3) : (n % (NT == 1 ? 1 : NT / 2)) * 8 + g;
      const bool lo = NT == 1 ? g >= 4 : n >= NT / 2;
      if (c < nc) x[n] = (lo ? a.h_lo : a.h_hi) + (size_t)s.cols[c0 + c] * a.I;
    }
    if constexpr (FMT != F_W4) {
      // a lane's columns start at t * 16 (BF16) or t * 32 (E4M3), added in item_mma
    }
  }
  Sums<NT> sums;
  run_tile<FMT, GROUP, NT>(sums, it, cur, next, ph.st, x, t);
  if (cur.n < ph.st.nsl) {
    const long long a0 = f - cur.s0;
    const int w0 = worker_of(a0, ph.F, ph.W), w1 = worker_of(a0 + ph.st.nsl - 1, ph.F, ph.W);
    if (!join_parts<NT>(sums, a.part, a.part_count, ph.me, cur.s0 == 0 ? 1 : 0, w0, w1, lane)) return false;
  }
  if (!ph.down) {
    if constexpr (NT <= 2) store_h<NT>(a, s, sums, entry, tile, lane);
  } else {
    store_y<NT>(a, s, sums, entry, tile, lane);
  }
  return true;
}

template <int FMT, int GROUP>
__device__ __forceinline__ void first_load(const Phase<FMT, GROUP>& ph, Item<FMT, GROUP>& it) {
  if (ph.me < 0) return;
  const long long f = run_start(ph.F, ph.me, ph.W);
  int entry, tile, s0;
  ph.split(f, entry, tile, s0);
  const Tile c = ph.tile_at(f, entry, tile, s0);
  it.load(c.w, c.sc, c.zp, ph.st);
}

// This worker's run of a phase; `it` holds its first item.
template <int FMT, int GROUP>
__device__ __forceinline__ void run_phase(const Phase<FMT, GROUP>& ph, Item<FMT, GROUP>& it) {
  if (ph.me < 0) return;
  const LayerShared& s = ph.s;
  long long f = run_start(ph.F, ph.me, ph.W);
  int entry, tile, s0, done = 0;
  ph.split(f, entry, tile, s0);
  Tile cur = ph.tile_at(f, entry, tile, s0);
  while (true) {
    const long long fn = f + cur.n;
    Tile next;
    next.n = 0;
    int entry_n = entry, tile_n = tile;
    if (fn < ph.f1) {
      if (ph.down) {
        if (++entry_n == s.n_entries) { entry_n = 0; ++tile_n; }
      } else {
        if (++tile_n == ph.tiles) { tile_n = 0; ++entry_n; }
      }
      next = ph.tile_at(fn, entry_n, tile_n, 0);
    }
    const int nc = s.ncols[entry];
    bool whole;
    if (ph.down) {
      if (nc <= 4) whole = do_tile<FMT, GROUP, 1>(ph, it, cur, next, entry, tile, f);
      else if (nc <= 8) whole = do_tile<FMT, GROUP, 2>(ph, it, cur, next, entry, tile, f);
      else whole = do_tile<FMT, GROUP, 4>(ph, it, cur, next, entry, tile, f);
      done += whole;
      // leaving the row tile: count its completed experts; the last one combines
      if (done && (next.n == 0 || tile_n != tile)) {
        __threadfence();
        __syncwarp();
        int old = 0;
        if (ph.lane == 0) old = atomicAdd(&ph.a.tile_count[tile], done);
        old = __shfl_sync(0xffffffffu, old, 0);
        if (old + done == s.n_entries) {
          __threadfence();
          if (ph.lane == 0) ph.a.tile_count[tile] = 0;
          combine_tile(ph.a, s, tile, ph.lane);
        }
        done = 0;
      }
    } else {
      if (nc <= 8) do_tile<FMT, GROUP, 1>(ph, it, cur, next, entry, tile, f);
      else do_tile<FMT, GROUP, 2>(ph, it, cur, next, entry, tile, f);
    }
    if (next.n == 0) break;
    f = fn;
    cur = next;
    entry = entry_n;
    tile = tile_n;
  }
}

template <int FMT, int GROUP>
__global__ void __launch_bounds__(THREADS, 1) layer_kernel(const LayerArgs a) {
  __shared__ LayerShared s;
  __shared__ int ok;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.T * a.K;
  const float* logits = a.logits_in;
  if (a.w_router) {
    router_logits(a.x, a.w_router, a.router_bias, a.T, a.H, a.E, a.logits, blockIdx.x * WARPS + warp,
                  gridDim.x * WARPS, lane);
    if (!grid_barrier(a.bar, a.dev_status, &ok)) return;
    logits = a.logits;
  }
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
  __syncthreads();
  Item<FMT, GROUP> it;
  {
    const Phase<FMT, GROUP> ph(a, s, false, warp, lane);
    first_load(ph, it);
    run_phase(ph, it);
  }
  const Phase<FMT, GROUP> ph(a, s, true, warp, lane);
  first_load(ph, it);
  if (!grid_barrier(a.bar, a.dev_status, &ok)) return;
  if (s.n_entries == 0) {   // no valid slot in the batch: every output is +0
    for (size_t i = (size_t)blockIdx.x * THREADS + tid; i < (size_t)a.T * a.H; i += (size_t)gridDim.x * THREADS)
      a.out[i] = 0;
    return;
  }
  run_phase(ph, it);
}

template <int FMT, int GROUP>
cudaError_t launch_layer(const LayerArgs& a, cudaStream_t stream) {
  void* args[] = {const_cast<LayerArgs*>(&a)};
  return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(&layer_kernel<FMT, GROUP>), dim3(num_sms()),
                                     dim3(THREADS), args, 0, stream);
}

cudaError_t launch_layer_bf16(const LayerArgs& a, cudaStream_t stream);
cudaError_t launch_layer_e4m3(const LayerArgs& a, cudaStream_t stream);
cudaError_t launch_layer_w4(const LayerArgs& a, int group, cudaStream_t stream);

}  // namespace few
}  // namespace moe
