// The whole MoE layer for a few tokens in one cooperative launch (moe_layer_few): router
// product (optional), top-k, gate/up + SwiGLU, down, fixed-order combine.  Included by
// one .cu file per weight format.  Internal header.
//
//   0  the router logits (with w_router), and for 4- and 8-bit weights the tokens as FP16 (below);
//      one grid barrier.  Every SM then selects the top-k itself (T x E logits from L2) and
//      lists the experts met with their columns.
//   1  tiles of 16 gate + 16 up rows of an expert: h = silu(g) * u of a (token, slot).
//   2  tiles of 32 output rows of an expert: y = W2 h in float32; the SM that completes a row
//      tile's last expert sums its rows over the slots in the combine's order.
// All tiles, phase 1 then phase 2, expert by expert, are one queue.  The scheduler warp of an SM takes
// the next tile when its workers are about to need it, so SMs stay level whatever the experts
// cost, and phase 2 begins on the first experts while phase 1 ends on the last: a tile of phase 2
// waits for its expert's h alone (its weights are loaded meanwhile).  Tiles in the queue are
// taken by running CTAs only, in order, so what a tile waits for is always being worked on.
//
// 16-bit operands: BF16 weights take BF16 activations.  E4M3 and 4-bit weights become FP16 in
// fewer instructions than BF16 (the conversion unit gives FP16 pairs), so their activations
// are FP16, scaled by powers of two: x per token, so that its largest value comes to 2^14 (FP16
// then holds every BF16 value above 2^-28 of the largest exactly, and the rest to 2^-39 of it);
// h per slot and tile of phase 1 (16 values, whose largest comes to 2^14), as each tile is
// finished.  Phase 2 brings these to the slot's largest scale as it reads them, by a product with a
// power of two, so nothing has to wait for the whole of h but the largest exponent.
//
// Bound: reading the weights of the experts met once.  Measured (6.68 TB/s is the copy bandwidth):
//   E4M3, 16 tokens at H = 7168, I = 2048, E = 256, top-8 + shared: 655-710 us with where the weights lie in
//     memory, 6.4-6.9 TB/s (reads alone may pass the copy bandwidth)
//   E4M3, one token at those sizes: 84 us for 400 MB -- 10 until the experts are known, 60
//     streaming at the copy bandwidth, 8 from the average warp's last unit to the last combine, launch
//   BF16, 5 tokens at H = 2048, I = 1408, E = 64, top-8: 85 us, 5.9 TB/s
//   4 bits, one token at the E4M3 sizes: 75 us, 2.8 TB/s; 32 tokens at the BF16 sizes, groups of 32 with
//     zero points: 141 us, 2.3 TB/s (126 with one term of h) -- latency of an item (few.cuh)
//   BF16, one token at H = 256, I = 512, E = 8, top-2: 19 us, latency throughout
// An expert's weights are read once for each 16 columns: a shared expert of 17 to 32 tokens twice.
// An L2 prefetch of the shared expert while the routing is found out changed none of these.
//
// Roundings of h: one FP16 term keeps 11 bits, an error of 1.4e-4 of the output that moves one BF16
// output in thirty to its neighbour (9e-4 of the outputs' size); one BF16 term 1.2e-3.  So h is
// kept in two terms, h = hi + lo (BF16: 16 bits, FP16: 22): side by side as two columns of one tensor
// instruction up to 4 columns of an expert, as two instructions above.
#pragma once

#include "few.cuh"
#include "route_few.cuh"

namespace moe {
namespace few {

constexpr int MAX_WARPS = 16;
// Warps of a CTA, the last of which schedules.  W4's unpacking wants more than the 128 registers a
// thread has with 16 warps: 144 us with 12 warps, 157 with 14, 168 with 16 on 32 tokens at H = 2048,
// I = 1408, E = 64, top-8, groups of 32; E4M3's does not: 720 us with 16 against 796 on 16 tokens at H = 7168, I = 2048,
// E = 256, top-8 (both measured with one term of h).  At these limits 36 to 56 bytes of a thread's registers are
// kept in local memory (W4, E4M3), around the variants of a unit.
template <int FMT>
__host__ __device__ constexpr int warps_of() { return FMT == F_W4 ? 12 : MAX_WARPS; }
constexpr int PARTS_BYTES = 40 * 1024;      // slots of the joins
constexpr int kMaxSlots = kMaxTokens * kMaxTopK;
// one entry = up to COLS columns of one expert; at most one per routed slot, plus the shared ones
constexpr int kMaxEntries = kMaxSlots + kMaxTokens / COLS;
constexpr int kMaxWidth = 1 << 17;          // H and I

// Exponents of h are kept as 121 + log2(what 1 in a FP16 term stands for), 1 .. 234; a slot's row of
// them is padded to 16 bytes.
constexpr int EXP_BIAS = 121;
__host__ __device__ __forceinline__ int exp_pitch(int i) { return (i / 16 + 15) / 16 * 16; }
// Rows of FP16 activations reach to whole W4 items.
__host__ __device__ __forceinline__ int half_pitch(int k) { return (k + 255) / 256 * 256; }

struct LayerArgs {
  CUtensorMap map[4];          // BF16, E4M3: w13, w2, shared w13, shared w2 (boxes of 16 rows x 128 bytes)
  int T, H, I, E, K;
  int shared, tiled, zeros;
  const uint8_t* w[4];         // the same four, for W4
  const float* scales[4];      // E4M3
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
  unsigned long long limit_ns; // of each wait
  // workspace, zero between launches
  uint32_t* ctl;               // barrier arrivals, barrier generation, next tile, CTAs done
  int32_t* tile_count;         // [H / 32] experts done of a row tile
  int32_t* entry_done;         // [kMaxEntries] row tiles done of an expert's h
  int32_t* h_top;              // [T*K + T] largest exponent of a slot's h (FP16)
  // workspace
  uint16_t* x16;               // [T, half_pitch(H)] FP16
  float* x_unit;               // [T] what 1 in x16 stands for
  uint16_t* h_hi;              // [T*K + T, I]; FP16: rows of half_pitch(I)
  int h_lo;                    // elements from h_hi to the second terms
  uint8_t* h_exp;              // [T*K + T, ex_pitch] exponent of each 16 values of h (FP16)
  float* y;                    // [T*K + T, H]
};

struct LayerShared {
  int n_entries;
  int max_cols;
  int n1, n_all;               // tiles of phase 1, of both phases
  int tiles1, tiles2;          // row tiles of one expert
  int own;                     // tiles of each CTA that do not come off the queue
  Cut cut[2];
  Feed<MAX_WARPS - 1> feed;
  int ready;                   // leading entries whose h is ready
  int go;
  int gave_up;                 // a wait of this CTA ran out
  float block[MAX_WARPS];
  short expert[kMaxEntries];   // E for the shared expert
  short first[kMaxEntries];    // first column in cols
  int ncols[kMaxEntries];
  short cols[kMaxSlots + kMaxTokens];   // slot ids t*K + k, or T*K + t for the shared expert
  short toks[kMaxSlots + kMaxTokens];   // and their tokens
  short count[kMaxExperts];    // listing: slots of the expert so far
  short open[kMaxExperts];     // listing: its entry being filled
  short slot_entry[kMaxSlots];
  uint8_t slot_rank[kMaxSlots];
  short id[kMaxSlots];         // expert of each slot, -1 padding
  float w[kMaxSlots];
  uint8_t alive[kMaxTokens];   // token has a valid slot
  JoinShared join;
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
__device__ __forceinline__ bool barrier_wait(uint32_t* bar, uint32_t gen, const Patience& patience) {
  const bool ok = wait_for(
      [&] {
        uint32_t now;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(bar + 1) : "memory");
        return now != gen;
      },
      patience);
  __threadfence();
  return ok;
}

// Token t as FP16 (all threads of one CTA).
template <int WARPS>
__device__ __forceinline__ void token_to_half(const LayerArgs& a, LayerShared& s, int t, int tid) {
  const uint4* src = reinterpret_cast<const uint4*>(a.x + (size_t)t * a.H);
  uint32_t m = 0;
  for (int i = tid; i < a.H / 8; i += WARPS * 32) {
    m = max(m, bf16_max(__ldg(src + i)));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) s.block[tid >> 5] = __uint_as_float(m);
  __syncthreads();
  m = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) m = max(m, __float_as_uint(s.block[i]));
  const float sc = to_half_scale(m);
  for (int i = tid; i < a.H / 8; i += WARPS * 32) {
    reinterpret_cast<uint4*>(a.x16 + (size_t)t * half_pitch(a.H))[i] = bf16_to_half8(__ldg(src + i), sc);
  }
  for (int i = a.H / 8 + tid; i < half_pitch(a.H) / 8; i += WARPS * 32)
    reinterpret_cast<uint4*>(a.x16 + (size_t)t * half_pitch(a.H))[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) a.x_unit[t] = 1.0f / sc;
  __syncthreads();
}

// Lists the experts met -- the shared one, then in the order of their first slots -- and their
// columns (all threads; every CTA gets the same lists).  Loops are kept rolled: the code runs
// once per launch and is bound by fetching it.
template <int WARPS>
__device__ __forceinline__ void list_entries(const LayerArgs& a, LayerShared& s) {
  const int n = a.T * a.K, tid = threadIdx.x, lane = tid & 31;
  for (int e = tid; e < a.E; e += WARPS * 32) s.count[e] = 0;
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
    if (v) {
      s.cols[__popc(m & lanemask_lt())] = (short)(n + lane);
      s.toks[__popc(m & lanemask_lt())] = (short)lane;
    }
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
    if (s.id[i] >= 0) {
      const int c = s.first[s.slot_entry[i]] + s.slot_rank[i];
      s.cols[c] = (short)i;
      s.toks[c] = (short)(i / a.K);
    }
  if (lane == 0) {
    s.n_entries = ent;
    s.max_cols = most;
  }
}

// The scheduler's side: tiles off the queue (the first s.own of a CTA are its own; the others are
// asked for one run ahead), and which entries' h are ready, as far as tiles of phase 2 need them.
template <int FMT, int GROUP>
struct LayerSched {
  const LayerArgs& a;
  LayerShared& s;
  int q, pending, run, ready, want;

  __device__ __forceinline__ bool next(int lane, int& t, int& n) {
    // runs of a few (smaller) tiles in phase 2 as long as there are plenty, about 32 items of small ones: a
    // look at the queue takes about as long as an SM needs for 32 KB (16 tokens, E4M3 as above: 685 us,
    // 699 with two at most; 32 tokens in 4 bits, H = 1024, I = 512, E = 128: 67.7, 74.4 with four)
    if (q < s.own) {
      t = blockIdx.x + q * gridDim.x;
      n = 1;
    } else {
      t = __shfl_sync(0xffffffffu, pending, 0);
      n = run;
    }
    if (++q >= s.own) {
      const int left = (s.n_all - t) / (int)gridDim.x;
      run = t < s.n1 || left < 3 ? 1 : min(left / 2, max(left < 20 ? 2 : 4, 32 / s.cut[1].nsl));
      if (lane == 0) pending = (int)(s.own * gridDim.x + atomicAdd(&a.ctl[2], (unsigned)run));
    }
    n = min(n, s.n_all - t);
    if (n <= 0) return false;
    if (t + n > s.n1) want = max(want, (t + n - 1 - s.n1) / s.tiles2 + 1);
    return true;
  }
  __device__ __forceinline__ Cut cut(int t) const { return s.cut[t >= s.n1]; }
  __device__ __forceinline__ int same(int t) const { return t < s.n1 ? s.n1 - t : s.n_all - t; }
  __device__ __forceinline__ bool done() const { return ready >= want; }
  __device__ __forceinline__ bool idle(int lane) {
    if (ready >= want) return false;
    const int e = ready + lane;
    int v = 0;
    if (e < want) asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(a.entry_done + e) : "memory");
    const unsigned m = __ballot_sync(0xffffffffu, e < want && v == s.tiles1);
    const int n = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
    if (n == 0) return false;
    ready += n;
    __threadfence();
    __syncwarp();
    if (lane == 0) *static_cast<volatile int*>(&s.ready) = ready;
    return true;
  }
  __device__ __forceinline__ void describe(int t, int part, const Cut& c, Unit& u) const {
    const bool d = t >= s.n1;
    const int tiles = d ? s.tiles2 : s.tiles1, i = d ? t - s.n1 : t;
    const int entry = i / tiles, row = i - entry * tiles;
    const int e = s.expert[entry];
    const bool sh = e == a.E;
    const int which = (sh ? 2 : 0) + d;
    const long long m = sh ? 0 : e;
    const int s0 = part * c.len;
    const int rows = d ? a.H : 2 * a.I, k = d ? a.I : a.H;
    u.entry = entry;
    u.row = row;
    u.s0 = (short)s0;
    u.n = (short)min(c.len, c.nsl - s0);
    u.part = (short)part;
    u.parts = (short)c.parts;
    u.down = d;
    // the half tiles: 16 rows each, side by side in phase 2, gate and up rows in phase 1
    const int r0 = d ? row * 32 : row * 16, r1 = d ? r0 + 16 : a.I + r0;
    if constexpr (FMT == F_W4) {
      const int block = w4_block(GROUP, a.zeros);
      const uint8_t* w = a.w[which] + m * (rows / 16) * c.nsl * block;
      u.p0 = w + ((long long)(r0 / 16) * c.nsl + s0) * block;
      u.p1 = w + ((long long)(r1 / 16) * c.nsl + s0) * block;
    } else {
      u.map = &a.map[which];
      if (a.tiled) {
        // boxes of 128 rows x 128 bytes, one after the other along K: row y of 128-byte lines
        u.x = 0;
        u.y0 = (int)(((m * (rows / 128) + r0 / 128) * c.nsl + s0) * 128 + r0 % 128);
        u.y1 = (int)(((m * (rows / 128) + r1 / 128) * c.nsl + s0) * 128 + r1 % 128);
      } else {
        u.x = s0 * 128;
        u.y0 = (int)(m * rows + r0);
        u.y1 = (int)(m * rows + r1);
      }
      if constexpr (FMT == F_E4M3) {
        const float* sc = a.scales[which] + m * (rows / 128) * (k / 128) + s0;
        u.p0 = reinterpret_cast<const uint8_t*>(sc + (long long)(r0 / 128) * (k / 128));
        u.p1 = reinterpret_cast<const uint8_t*>(sc + (long long)(r1 / 128) * (k / 128));
      }
    }
  }
};

// Cuts of both phases (one warp, a lane per number of parts): the least rounds of a unit per worker, times
// what a unit takes.
template <int FMT>
__device__ __forceinline__ void plan_phases(const LayerArgs& a, LayerShared& s, int lane) {
  constexpr int WORKERS = warps_of<FMT>() - 1;
  const int tiles1 = a.I / 16, tiles2 = a.H / 32, workers = gridDim.x * WORKERS;
#pragma unroll 1
  for (int d = 0; d < 2; ++d) {
    const int k = d ? a.I : a.H;
    const int items = FMT == F_W4 ? w4_slices(k) : FMT == F_BF16 ? k / 64 : k / 128;
    const int tiles = s.n_entries * (d ? tiles2 : tiles1);
    // Longer units cost less per item, shorter ones level the end of the layer.  One token at the
    // decode sizes (E4M3), 4 / 8 items in phase 1: 86.4 / 82.6 us, then 4 / 8 in phase 2: 82.6 / 83.3;
    // 16 tokens: 719 / 698 and 698 / 689.
    const int longest = d == 0 || tiles >= 20 * (int)gridDim.x ? 8 : 4;
    const int n = min(lane + 1, min(WORKERS, items)), len = (items + n - 1) / n;
    const unsigned rounds = (unsigned)((tiles * n + workers - 1) / workers);
    const unsigned cost = len <= longest || n == min(WORKERS, items) ? rounds * (len + UNIT_COST) * 32 + n : 0xffffffffu;
    const int best = (int)(__reduce_min_sync(0xffffffffu, cost) & 31u);
    if (lane == 0) s.cut[d].set(items, best);
  }
  if (lane == 0) {
    s.tiles1 = tiles1;
    s.tiles2 = tiles2;
    s.n1 = s.n_entries * tiles1;
    s.n_all = s.n1 + s.n_entries * tiles2;
    // Phase 1 but for its rest is handed out evenly: an SM gets through small tiles faster than the queue
    // gives them one by one (32 tokens in 4 bits, H = 1024, I = 512, E = 128: 81.1 us with two, 74.4).
    s.own = max(2, s.n1 / (int)gridDim.x);
    s.ready = 0;
  }
}

// Phase 1's result for one tile: h of 16 intermediate rows as two BF16 or two scaled FP16 terms.
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
      float unit = 1.0f, h[2];
      if (HALF && slot >= 0) unit = __ldcg(&a.x_unit[s.toks[c0 + c]]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float gate = sums.v[n][0][2 * i + j] * unit, up = sums.v[n][1][2 * i + j] * unit;
        h[i] = gate / (1.0f + expf(-gate)) * up;
      }
      float sc = 1.0f;
      if (HALF) {
        // infinities and NaN count as the largest finite value: their block sets the slot's scale, so phase 2
        // takes them times 1, never times a power of two that FP16 has no room for (infinity times 0)
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) most = max(most, min(__float_as_uint(h[i]) & 0x7fffffffu, 0x7f7fffffu));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        sc = to_half_scale(most);
        if (g == 0 && slot >= 0) {
          const int e = EXP_BIAS + 127 - (int)(__float_as_uint(sc) >> 23);
          a.h_exp[(size_t)slot * exp_pitch(a.I) + tile] = (uint8_t)e;
          atomicMax(&a.h_top[slot], e);
        }
      }
      if (slot < 0) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const size_t o = (size_t)slot * (HALF ? half_pitch(a.I) : a.I) + tile * 16 + g + i * 8;
        if (HALF) {
          const float v = h[i] * sc;
          const uint16_t hi = half_bits(v);
          a.h_hi[o] = hi;
          a.h_hi[o + a.h_lo] = (hi & 0x7fffu) >= 0x7c00u ? 0 : half_bits(v - __half2float(__ushort_as_half(hi)));   // inf, NaN: hi alone
          // the last tile also clears the rows' ends
          if (tile == s.tiles1 - 1 && i == 0)
            for (int z = a.I + g * 8; z < half_pitch(a.I); z += 64) {
              uint16_t* p = a.h_hi + (size_t)slot * half_pitch(a.I) + z;
              *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(p + a.h_lo) = make_uint4(0, 0, 0, 0);
            }
        } else {
          const uint16_t hi = f32_to_bf16(h[i]);
          a.h_hi[o] = hi;
          a.h_hi[o + a.h_lo] = f32_to_bf16((hi & 0x7fffu) >= 0x7f80u ? 0.0f : h[i] - bf16_to_f32(hi));   // inf, NaN: hi alone
        }
      }
    }
}

// Phase 2's result for one (row tile, expert): y rows.  Up to 4 columns come as hi and lo columns of
// one group (hi in columns 0-3, lanes t = 0, 1; lo in 4-7, t = 2, 3).
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
        const float unit = HALF ? __uint_as_float((uint32_t)(127 - EXP_BIAS + __ldcg(&a.h_top[slot])) << 23) : 1.0f;
        float* p = a.y + (size_t)slot * a.H + tile * 32 + g + (i >> 1) * 8;
        __stcg(p, sums.v[n][0][i] * unit);
        __stcg(p + 16, sums.v[n][1][i] * unit);
      }
    }
}

// One row tile's outputs in the combine's order: ascending slot, float32 product and sum from +0,
// the shared row last, one BF16 rounding.  Lane = (token of four, four rows), G such tokens at a time:
// a warp has up to 8 G 16-byte loads in flight per lane, since this is the tail of the layer.  Not
// inlined: its registers are not the streaming loop's.  G = 2 beyond 8 tokens: 139.9 -> 135.9 us for 32
// (4 bits, H = 2048), 670.6 -> 667.2 for 16 (E4M3, H = 7168); with 5, 83.6 -> 85.8 (BF16, H = 2048).
template <int G>
static __device__ __noinline__ void combine_tile(const LayerArgs& a, const LayerShared& s, int tile, int lane) {
  const int row = tile * 32 + (lane & 7) * 4;
#pragma unroll 1
  for (int t0 = lane >> 3; t0 < a.T; t0 += 4 * G) {
    float acc[G][4];
    float4 sv[G];
    int tok[G];
    bool sh[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      tok[g] = min(t0 + 4 * g, a.T - 1);         // past the end: the last one again, not stored
      sh[g] = a.shared && s.alive[tok[g]];
      acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.0f;
      sv[g] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (sh[g]) sv[g] = __ldcg(reinterpret_cast<const float4*>(a.y + (size_t)(a.T * a.K + tok[g]) * a.H + row));
    }
#pragma unroll 1
    for (int k0 = 0; k0 < a.K; k0 += 8) {
      // every row is read, used or not (they all exist): a load behind a condition waits for the one before
      float4 v[G][8];
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[g][j] = __ldcg(reinterpret_cast<const float4*>(a.y + (size_t)(tok[g] * a.K + min(k0 + j, a.K - 1)) * a.H + row));
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = tok[g] * a.K + min(k0 + j, a.K - 1);
          const bool use = k0 + j < a.K && s.id[i] >= 0;
          const float w = s.w[i];
          acc[g][0] = use ? __fadd_rn(acc[g][0], __fmul_rn(v[g][j].x, w)) : acc[g][0];
          acc[g][1] = use ? __fadd_rn(acc[g][1], __fmul_rn(v[g][j].y, w)) : acc[g][1];
          acc[g][2] = use ? __fadd_rn(acc[g][2], __fmul_rn(v[g][j].z, w)) : acc[g][2];
          acc[g][3] = use ? __fadd_rn(acc[g][3], __fmul_rn(v[g][j].w, w)) : acc[g][3];
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (sh[g]) {
        acc[g][0] = __fadd_rn(acc[g][0], sv[g].x);
        acc[g][1] = __fadd_rn(acc[g][1], sv[g].y);
        acc[g][2] = __fadd_rn(acc[g][2], sv[g].z);
        acc[g][3] = __fadd_rn(acc[g][3], sv[g].w);
      }
      const uint32_t lo = f32_to_bf16(acc[g][0]) | (uint32_t)f32_to_bf16(acc[g][1]) << 16;
      const uint32_t hi = f32_to_bf16(acc[g][2]) | (uint32_t)f32_to_bf16(acc[g][3]) << 16;
      if (t0 + 4 * g < a.T) *reinterpret_cast<uint2*>(a.out + (size_t)tok[g] * a.H + row) = make_uint2(lo, hi);
    }
  }
}

template <int FMT, int GROUP>
using LayerStream = Stream<FMT, GROUP, FMT != F_BF16, false, FeedSource<MAX_WARPS - 1>>;

// The unit in use with NT column groups: columns, sums, join, result.
template <int FMT, int GROUP, int NT, int PASSES>
__device__ __forceinline__ void do_unit(const LayerArgs& a, LayerShared& s, LayerStream<FMT, GROUP>& in, bool down,
                                        float4* parts, int slots, int stride) {
  constexpr bool HALF = FMT != F_BF16;
  const int lane = in.lane, g = lane >> 2;
  const Unit& un = in.src.unit(in.cur);
  const int entry = un.entry, row = un.row, part = un.part, n = un.parts;
  const int nc = s.ncols[entry], c0 = s.first[entry];
  int off[PASSES][NT];
  const uint8_t* ex[NT];
  int top[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const bool pairs = down && PASSES == 1;              // hi and lo as columns of one group
    const int c = pairs ? (g & 3) : i * 8 + g;
    const int at = c0 + (c < nc ? c : 0);                // no such column: the first one again
    const int slot = s.cols[at];
    ex[i] = nullptr;
    top[i] = 0;
    if (HALF && down) {
      ex[i] = a.h_exp + (size_t)slot * exp_pitch(a.I);
      top[i] = __ldcg(&a.h_top[slot]);
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if (!down)
        off[p][i] = s.toks[at] * (HALF ? half_pitch(a.H) : a.H);
      else
        off[p][i] = slot * (HALF ? half_pitch(a.I) : a.I) + ((pairs ? g >= 4 : p == 1) ? a.h_lo : 0);
    }
  }
  Sums<NT> sums;
  const Acts<false> from{down ? a.h_hi : HALF ? a.x16 : a.x, 0};
  if (!in.template run<NT, PASSES>(sums, from, off, HALF && down, ex, top)) return;
  if (!join<NT>(sums, s.join, parts, slots, stride, in.cur, in.cur - part, n, lane, in.patience)) return;
  if (!down) {
    store_h<HALF, NT>(a, s, sums, entry, row, lane);
    __syncwarp();
    if (lane == 0) atom_add_release(&a.entry_done[entry], 1);
    return;
  }
  store_y<HALF, NT>(a, s, sums, entry, row, lane);
  __syncwarp();
  int old = 0;
  if (lane == 0) old = atom_add_release(&a.tile_count[row], 1);
  if (__shfl_sync(0xffffffffu, old, 0) != s.n_entries - 1) return;
  __threadfence();
  if (lane == 0) a.tile_count[row] = 0;
  if (a.T > 8) combine_tile<2>(a, s, row, lane);
  else combine_tile<1>(a, s, row, lane);
}

template <int FMT, int GROUP>
__global__ void __launch_bounds__(warps_of<FMT>() * 32, 1) layer_kernel(const __grid_constant__ LayerArgs a) {
  constexpr bool HALF = FMT != F_BF16;
  constexpr int WARPS = warps_of<FMT>(), THREADS = WARPS * 32, WORKERS = WARPS - 1;
  __shared__ LayerShared s;
  extern __shared__ __align__(1024) uint8_t rings[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.T * a.K;
  const bool sync = HALF || a.w_router;
  // where the joins' slots will be
  float2* scratch = reinterpret_cast<float2*>(rings + WORKERS * 2 * Format<FMT, GROUP>::STAGE);
  static_assert(ROUTE_SCRATCH * 8 <= PARTS_BYTES, "");
  uint32_t gen = 0;
  const Patience patience{&s.gave_up, a.dev_status, a.limit_ns};
  if (tid == 0) s.gave_up = 0;
  if (HALF)
    // by the last CTAs, which have the fewest router rows
    for (int t = gridDim.x - 1 - blockIdx.x; t < a.T; t += gridDim.x) token_to_half<WARPS>(a, s, t, tid);
  if (a.w_router)
    router_logits<WARPS>(a.x, a.w_router, a.router_bias, a.T, a.H, a.E, a.logits, scratch, blockIdx.x, gridDim.x,
                         warp, lane);
  if (sync) {
    __syncthreads();
    if (tid == 0) gen = barrier_arrive(a.ctl);
  }
  if (a.w_router) {
    if (tid == 0) s.go = barrier_wait(a.ctl, gen, patience);
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
  list_entries<WARPS>(a, s);
  if (warp == 0) {
    __syncwarp();
    plan_phases<FMT>(a, s, lane);
  }
  if (tid == 0) {
    if (!sync) s.go = 1;
    else if (!a.w_router) s.go = barrier_wait(a.ctl, gen, patience);
  }
  join_init(s.join);
  feed_init(s.feed);
  __syncthreads();
  if (!s.go) return;
  if (s.n_entries == 0) {   // no valid slot in the batch: every output is +0
    for (size_t i = (size_t)blockIdx.x * THREADS + tid; i < (size_t)a.T * a.H; i += (size_t)gridDim.x * THREADS)
      a.out[i] = 0;
    return;
  }
  if (warp == WORKERS) {
    LayerSched<FMT, GROUP> src{a, s, 0, 0, 0, 0, 0};
    schedule<WORKERS>(s.feed, src, lane, patience);
  } else {
    constexpr int RING = 2 * Format<FMT, GROUP>::STAGE;
    float4* parts = reinterpret_cast<float4*>(rings + WORKERS * RING);
    const int stride = s.max_cols <= 8 ? 64 : 128;       // a slot is 1 KB for each 8 columns
    const int slots = min(MAX_SLOTS, PARTS_BYTES / (stride * 16));
    LayerStream<FMT, GROUP> in{{s.feed, warp}, rings + warp * RING};
    in.ring_addr = gg::smem_u32(in.ring);
    in.bars = gg::smem_u32(&s.feed.full[warp][0]);
    in.lane = lane;
    in.patience = patience;
    in.dx = a.tiled ? 0 : 128;
    in.dy = a.tiled ? 128 : 0;
    in.block = FMT == F_W4 ? w4_block(GROUP, a.zeros) : 0;
    in.zeros = a.zeros;
    in.start();
    volatile int* ready = &s.ready;
    while (in.take()) {
      const int entry = in.src.unit(in.cur).entry;
      const bool down = in.src.unit(in.cur).down;
      const int nc = s.ncols[entry];
      if (down) {
        if (!warp_wait_for([&] { return *ready > entry; }, patience)) {
          in.dead = 1;
          break;
        }
        __threadfence_block();
        __syncwarp();
      }
      // phase 2: hi and lo side by side in one group of 8 up to 4 columns, else one after the other
      if (down && nc > 4) {
        if (nc > 8) do_unit<FMT, GROUP, 2, 2>(a, s, in, down, parts, slots, stride);
        else do_unit<FMT, GROUP, 1, 2>(a, s, in, down, parts, slots, stride);
      } else if (nc > 8) {
        do_unit<FMT, GROUP, 2, 1>(a, s, in, down, parts, slots, stride);
      } else {
        do_unit<FMT, GROUP, 1, 1>(a, s, in, down, parts, slots, stride);
      }
    }
    in.finish();
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
  for (int i = tid; i < a.T * (a.K + 1); i += THREADS) a.h_top[i] = 0;
  if (tid < 2) a.ctl[2 + tid] = 0;
}

template <int FMT, int GROUP>
cudaError_t launch_layer(const LayerArgs& a, cudaStream_t stream) {
  constexpr int smem = (warps_of<FMT>() - 1) * 2 * Format<FMT, GROUP>::STAGE + PARTS_BYTES;
  static std::atomic<unsigned long long> done{0};
  if (!once_per_device(done, [] {
        return cudaFuncSetAttribute(layer_kernel<FMT, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) ==
               cudaSuccess;
      }))
    return cudaErrorUnknown;
  void* args[] = {const_cast<LayerArgs*>(&a)};
  return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(&layer_kernel<FMT, GROUP>), dim3(num_sms()),
                                     dim3(warps_of<FMT>() * 32), args, smem, stream);
}

cudaError_t launch_layer_bf16(const LayerArgs& a, cudaStream_t stream);
cudaError_t launch_layer_e4m3(const LayerArgs& a, cudaStream_t stream);
cudaError_t launch_layer_w4(const LayerArgs& a, int group, cudaStream_t stream);

}  // namespace few
}  // namespace moe
