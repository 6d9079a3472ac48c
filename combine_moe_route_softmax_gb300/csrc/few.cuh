// Weight streaming for products with a few columns (1 to 32 activation rows per weight
// matrix), shared by the few-token layer (few_layer.cuh) and the 4-bit product
// (few_linear.cu).  Internal header.
//
// The mathematics: y[n, c] = sum_k W[n, k] x[c, k] for a handful of columns c.  Every weight is
// used a few times only, so the bound is reading W once; the arithmetic rides along on
// mma.sync.m16n8k16 (16-bit operands, float32 sums), weights as the 16-row operand and activation
// rows as the 8 columns -- 2 to 8 tensor instructions per KB of weights, far below any
// tensor-core limit, which is why these kernels do not use the 128-row tcgen05 tiles.
//
// Work is cut into items: 32 weight rows (a row tile) x 128 bytes of K, 4 KB; a few neighbouring
// items of a tile are a unit.  A CTA (one per SM) takes whole tiles, one after the other,
// and its worker warps take the units of that sequence in turn, each running ahead on its own:
// a warp copies its items with cp.async into a ring of its own in shared memory, whole
// 128-byte lines, ahead of their use, across units and tiles.  The K order inside a line is
// whatever the lanes hold, since a dot product does not care and the activations are read in
// the same order.  The sums of a tile's units are joined in shared memory by the warp that
// finishes last, in unit order, so the result does not depend on who was last.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {
namespace few {

constexpr int kMaxTokens = MOE_FEW_MAX_TOKENS;
constexpr int COLS = 16;             // columns of one matrix handled in one pass over it (layer)
constexpr unsigned long long TIMEOUT_NS = 2000000000ull;

enum { F_BF16 = 0, F_E4M3 = 1, F_W4 = 2 };

__device__ __forceinline__ unsigned long long clock_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Bounded wait for done(): false (and the status bit) after TIMEOUT_NS.
template <class Done>
__device__ __forceinline__ bool wait_for(Done done, int32_t* dev_status) {
  if (done()) return true;
  const unsigned long long t0 = clock_ns();
  while (!done()) {
    if (clock_ns() - t0 > TIMEOUT_NS) {
      if (dev_status) atomicOr(dev_status, MOE_DEV_PIPELINE_TIMEOUT);
      return false;
    }
  }
  return true;
}

// HALF: operands are FP16, else BF16.
template <bool HALF>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if (HALF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four E4M3 codes -> two FP16 pairs, exactly (FP16 holds every E4M3 value).
__device__ __forceinline__ void e4m3x4_to_half(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

// Eight 4-bit codes of one word minus their zero point -> four pairs (columns 0 1, 2 3, 4 5, 6 7).
// Column 2i sits at nibble i and 2i + 1 at nibble i + 4, so a mask leaves a pair of codes in
// the low mantissa bits of two 16-bit halves.  BF16: 0x4300 | c is exactly 128 + c, and minus
// (128 + z) is exact.  FP16: 0x6400 | c is 1024 + c, and 0x6400 | 16 c is 1024 + 16 c, a
// sixteenth of which minus (64 + z) is exact in one multiply-add: two shifts fewer.
template <bool HALF>
struct W4Zero {
  uint32_t a, b;               // 128 + z; or 1024 + z and -(64 + z)
  // z in byte `sel` of the word
  __device__ __forceinline__ W4Zero(uint32_t z, int sel) {
    if (HALF) {
      const uint32_t p = __byte_perm(z, 0, 0x4040 | sel * 0x0101);
      a = p | 0x64006400u;
      b = (p << 4) | 0xd400d400u;
    } else {
      a = __byte_perm(z, 0x43u, 0x4040 | sel * 0x0101);
      b = 0;
    }
  }
};
template <bool HALF>
__device__ __forceinline__ void w4_pairs(uint32_t v, const W4Zero<HALF>& z, uint32_t (&p)[4]) {
  if (HALF) {
    const uint32_t w = v >> 8;
    const uint32_t c0 = (v & 0x000f000fu) | 0x64006400u, c1 = (v & 0x00f000f0u) | 0x64006400u;
    const uint32_t c2 = (w & 0x000f000fu) | 0x64006400u, c3 = (w & 0x00f000f0u) | 0x64006400u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p[0]) : "r"(c0), "r"(z.a));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[1]) : "r"(c1), "r"(0x2c002c00u), "r"(z.b));   // 0x2c00 = 1/16
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p[2]) : "r"(c2), "r"(z.a));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[3]) : "r"(c3), "r"(0x2c002c00u), "r"(z.b));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = ((v >> (4 * i)) & 0x000f000fu) | 0x43004300u;
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(c), "r"(z.a));
    }
  }
}

// --------------------------------------------------------------------------------- items
// Where one row tile's items begin in memory.
struct Tile {
  const uint8_t* w;    // first row of the first half tile, at the unit's first slice
  const void* sc;      // E4M3: scale of the first half tile's block; W4: scales of its row block
  const void* zp;      // W4 zero points, or null
};
// One phase's matrices: constant strides, and how its tiles are cut into units.
struct Strides {
  long long step;      // bytes from one slice to the next
  long long pitch;     // bytes from one row of a half tile to the next
  long long half;      // bytes from the first half tile (16 rows) to the second
  long long sc_half;   // scale elements (E4M3 floats; W4 two-row words) to the second half tile
  int k;               // columns
  int nsl;             // slices (items) per tile
  int len, parts;      // items per unit (fewer in the last), units per tile
  // at most `most` units, of at least two items unless there is little work
  __host__ __device__ __forceinline__ void cut(int most, bool little) {
    len = (nsl + most - 1) / most;
    if (len < 2 && !little && nsl > 1) len = 2;
    parts = (nsl + len - 1) / len;
  }
};

template <int FMT, int GROUP>
struct Format {
  static constexpr int KI = FMT == F_BF16 ? 64 : FMT == F_E4M3 ? 128 : 256;   // columns per item
  static constexpr int NG = FMT == F_W4 ? 256 / GROUP : 1;                    // W4 scale groups per slice
  static constexpr int SC = FMT == F_W4 ? 8 * NG * 4 : 16;                    // scale bytes of a half tile
  static constexpr int ZP = FMT == F_W4 ? 8 * NG * 2 : 0;                     // zero-point bytes of a half tile
  static constexpr int HALF_CHUNKS = FMT == F_BF16 ? 1 : FMT == F_E4M3 ? 2 : 4;
  static constexpr int STAGE = FMT == F_BF16 ? 4096 : 4096 + 2 * (SC + ZP);
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One warp copies one item into its stage: 32 rows x 128 bytes, each instruction four whole
// lines.  16-byte chunk c of row r goes to chunk c ^ (r & 1), so that the reads below (two rows x
// every other chunk per 8 lanes) touch every bank once.
template <int FMT, int GROUP>
__device__ __forceinline__ void copy_item(uint32_t stage, const Tile& c, long long pitch, long long half,
                                          long long sc_half, int lane) {
  using F = Format<FMT, GROUP>;
  const int r = lane >> 3, ch = lane & 7;
  const uint8_t* p = c.w + r * pitch + ch * 16;
  const uint32_t d = stage + r * 128 + ((ch ^ (r & 1)) << 4);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 4; ++q) cp16(d + h * 2048 + q * 512, p + h * half + q * 4 * pitch);
  if constexpr (FMT == F_E4M3) {
    if (lane < 2) cp4(stage + 4096 + lane * 16, static_cast<const float*>(c.sc) + lane * sc_half);
  }
  if constexpr (FMT == F_W4) {
    constexpr int N = F::SC / 16;   // chunks per half tile
    if (lane < 2 * N)
      cp16(stage + 4096 + lane * 16, reinterpret_cast<const uint8_t*>(static_cast<const uint32_t*>(c.sc) +
                                                                      (lane / N) * sc_half) + (lane % N) * 16);
    if (c.zp && lane < N)
      cp16(stage + 4096 + 2 * F::SC + lane * 16,
           reinterpret_cast<const uint8_t*>(static_cast<const uint16_t*>(c.zp) + (lane / (N / 2)) * sc_half) +
               (lane % (N / 2)) * 16);
  }
}

// Sums of one row tile: [8-column group][half tile][fragment: rows g, g (+1 column), g + 8, g + 8].
template <int NT>
struct Sums {
  float v[NT][2][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[n][h][i] = 0.0f;
  }
};

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// This lane's activations: 16-byte chunk I of half J of an item (an item's half is J's 16 of the
// lane's 32 bytes per weight row, HALF_CHUNKS chunks of activations); x[n] is the lane's column of
// group n at the item's first column (null: no such column, zeros).  kleft: columns to the
// row's end (W4 rows are padded to whole items, activations are not).  Activations are kept
// in L1, which the weights pass by; plain loads, since the layer writes some of them in the
// same launch.
template <int FMT, int NT>
__device__ __forceinline__ void load_acts(uint4 (&b)[NT], const uint16_t* const (&x)[NT], int J, int I, int t,
                                          int kleft) {
  const int k = FMT == F_BF16 ? t * 16 + 8 * J : FMT == F_E4M3 ? t * 32 + 16 * J + 8 * I : (4 * J + I) * 32 + t * 8;
#pragma unroll
  for (int n = 0; n < NT; ++n)
    b[n] = x[n] && (FMT != F_W4 || k < kleft) ? *reinterpret_cast<const uint4*>(x[n] + k) : make_uint4(0, 0, 0, 0);
}

template <bool HALF, int NT>
__device__ __forceinline__ void mma_step(Sums<NT>& acc, const uint32_t (&a)[4][4], const uint4 (&b)[NT]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mma16<HALF>(acc.v[n][h], a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], b[n].x, b[n].y);
      mma16<HALF>(acc.v[n][h], a[2 * h][2], a[2 * h + 1][2], a[2 * h][3], a[2 * h + 1][3], b[n].z, b[n].w);
    }
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Half an item: sums += weights x activations.  acc: E4M3 sums of the item so far, unscaled.
template <int FMT, int GROUP, bool HALF, int NT, int PASSES, int J, class Acts>
__device__ __forceinline__ void half_item(Sums<NT>& sums, Sums<NT>& acc, const uint8_t* stage, Acts acts, int g, int t,
                                          bool zeros) {
  using F = Format<FMT, GROUP>;
  uint4 q[4];                      // rows g, g + 8 of the first half tile, then of the second
  const uint8_t* base = stage + g * 128 + (((2 * t + J) ^ (g & 1)) << 4);
#pragma unroll
  for (int r = 0; r < 4; ++r) q[r] = *reinterpret_cast<const uint4*>(base + r * 1024);
  if constexpr (FMT == F_BF16) {
    uint32_t a[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) { a[r][0] = q[r].x; a[r][1] = q[r].y; a[r][2] = q[r].z; a[r][3] = q[r].w; }
    uint4 b[PASSES][NT];
    acts(b, J, 0);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) mma_step<HALF, NT>(sums, a, b[p]);
  } else if constexpr (FMT == F_E4M3) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 b[PASSES][NT];
      acts(b, J, i);
      uint32_t a[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int w = 0; w < 2; ++w) e4m3x4_to_half(word(q[r], 2 * i + w), a[r][2 * w], a[r][2 * w + 1]);
#pragma unroll
      for (int p = 0; p < PASSES; ++p) mma_step<HALF, NT>(acc, a, b[p]);
    }
  } else {
    // word j of the lane's 8 holds columns j*32 + t*8 .. + 8
    constexpr int WPG = GROUP / 32;   // words per scale group
    const uint32_t* scales = reinterpret_cast<const uint32_t*>(stage + 4096) + g * F::NG;
    const uint16_t* zps = reinterpret_cast<const uint16_t*>(stage + 4096 + 2 * F::SC) + g * F::NG;
#pragma unroll
    for (int i0 = 0; i0 < 4; i0 += WPG) {
      const int gi = (4 * J + i0) / WPG;
      const uint32_t za = zeros ? zps[gi] : 0x0808u, zb = zeros ? zps[F::ZP / 2 + gi] : 0x0808u;
      const W4Zero<HALF> z[4] = {{za, 0}, {za, 1}, {zb, 0}, {zb, 1}};
      Sums<NT> part;
      part.clear();
#pragma unroll
      for (int i = i0; i < i0 + WPG; ++i) {
        uint4 b[PASSES][NT];
        acts(b, J, i);
        uint32_t a[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) w4_pairs<HALF>(word(q[r], i), z[r], a[r]);
#pragma unroll
        for (int p = 0; p < PASSES; ++p) mma_step<HALF, NT>(part, a, b[p]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t sc = scales[h * (F::SC / 4) + gi];
        const float s0 = bf_lo(sc), s1 = bf_hi(sc);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          sums.v[n][h][0] = fmaf(s0, part.v[n][h][0], sums.v[n][h][0]);
          sums.v[n][h][1] = fmaf(s0, part.v[n][h][1], sums.v[n][h][1]);
          sums.v[n][h][2] = fmaf(s1, part.v[n][h][2], sums.v[n][h][2]);
          sums.v[n][h][3] = fmaf(s1, part.v[n][h][3], sums.v[n][h][3]);
        }
      }
    }
  }
}

// -------------------------------------------------------------------------------- stream
// A CTA's sequence of tiles, as one worker warp sees it.  Src says what the sequence is:
//   tile(q)            number of the CTA's q-th tile, negative past the end (may wait);
//   strides(tile)      the strides and the cut of its phase;
//   where(tile, s0)    where its items begin at slice s0;  zeros().
// Units are counted over the sequence; worker w of WORKERS takes units w, w + WORKERS, ...  Its ring
// of STAGES stages is filled STAGES - 1 items ahead of their use.
template <int FMT, int GROUP, bool HALF, int STAGES, int WORKERS, class Src>
struct Stream {
  using F = Format<FMT, GROUP>;
  const Src& src;
  uint8_t* ring;
  uint32_t ring_addr;
  int lane;
  int in, out;                 // stage to fill next, stage to use next
  struct Cursor {
    int u, q, part, tile;      // unit, its place in the sequence, its part of the tile (number < 0: the end)
  } fillc, usec;
  int left;                    // items left of the unit being filled
  Tile c;
  long long step, pitch, half, sc_half;

  __device__ __forceinline__ Stream(const Src& s, uint8_t* r, int worker, int lane_)
      : src(s), ring(r), lane(lane_), in(0), out(0) {
    ring_addr = static_cast<uint32_t>(__cvta_generic_to_shared(r));
    fillc.u = worker;
    fillc.q = 0;
    fillc.part = worker;
    settle(fillc);
    usec = fillc;
    open();
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fill();
  }
  // from a part that may be past its tile to the tile it falls to
  __device__ __forceinline__ void settle(Cursor& k) const {
    while (true) {
      k.tile = src.tile(k.q);
      if (k.tile < 0) return;
      const int n = src.strides(k.tile).parts;
      if (k.part < n) return;
      k.part -= n;
      ++k.q;
    }
  }
  __device__ __forceinline__ void hop(Cursor& k) const {
    k.u += WORKERS;
    k.part += WORKERS;
    settle(k);
  }
  __device__ __forceinline__ void open() {
    if (fillc.tile < 0) return;
    const Strides& st = src.strides(fillc.tile);
    const int s0 = fillc.part * st.len;
    left = min(st.len, st.nsl - s0);
    step = st.step;
    pitch = st.pitch;
    half = st.half;
    sc_half = st.sc_half;
    c = src.where(fillc.tile, s0);
  }
  __device__ __forceinline__ void fill() {
    if (fillc.tile >= 0) {
      copy_item<FMT, GROUP>(ring_addr + in * F::STAGE, c, pitch, half, sc_half, lane);
      if (--left > 0) {
        c.w += step;
        if constexpr (FMT == F_E4M3) c.sc = static_cast<const float*>(c.sc) + 1;
        if constexpr (FMT == F_W4) {
          c.sc = static_cast<const uint32_t*>(c.sc) + 8 * F::NG;
          if (c.zp) c.zp = static_cast<const uint16_t*>(c.zp) + 8 * F::NG;
        }
      } else {
        hop(fillc);
        open();
      }
    }
    cp_commit();
    in = in + 1 == STAGES ? 0 : in + 1;
  }
  // The items of the unit at usec: sums = weights x activations.  x0[p][n] is this lane's column
  // of group n, or null; PASSES sets of columns are added into the same sums.
  template <int NT, int PASSES>
  __device__ __forceinline__ void run(Sums<NT>& sums, const Strides& st, const uint16_t* const (&x0)[PASSES][NT]) {
    const int g = lane >> 2, t = lane & 3;
    const int s0 = usec.part * st.len, n = min(st.len, st.nsl - s0);
    const uint16_t* x[PASSES][NT];
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
#pragma unroll
      for (int i = 0; i < NT; ++i) x[p][i] = x0[p][i] ? x0[p][i] + (long long)s0 * F::KI : nullptr;
    int kleft = st.k - s0 * F::KI;
    const bool zeros = src.zeros();
    sums.clear();
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      fill();
      // few columns: the item's activations are on their way before its weights are waited for
      constexpr bool EARLY = F::HALF_CHUNKS * NT * PASSES <= 4;
      uint4 early[EARLY ? 2 * F::HALF_CHUNKS : 1][PASSES][NT];
      if constexpr (EARLY) {
#pragma unroll
        for (int q = 0; q < 2 * F::HALF_CHUNKS; ++q)
#pragma unroll
          for (int p = 0; p < PASSES; ++p)
            load_acts<FMT, NT>(early[q][p], x[p], q / F::HALF_CHUNKS, q % F::HALF_CHUNKS, t, kleft);
      }
      auto acts = [&](uint4(&b)[PASSES][NT], int J, int I) {
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          if constexpr (EARLY) {
#pragma unroll
            for (int q = 0; q < NT; ++q) b[p][q] = early[J * F::HALF_CHUNKS + I][p][q];
          } else {
            load_acts<FMT, NT>(b[p], x[p], J, I, t, kleft);
          }
        }
      };
      cp_wait<STAGES - 1>();
      __syncwarp();
      const uint8_t* stage = ring + out * F::STAGE;
      Sums<NT> acc;
      if constexpr (FMT == F_E4M3) acc.clear();
      half_item<FMT, GROUP, HALF, NT, PASSES, 0>(sums, acc, stage, acts, g, t, zeros);
      half_item<FMT, GROUP, HALF, NT, PASSES, 1>(sums, acc, stage, acts, g, t, zeros);
      if constexpr (FMT == F_E4M3) {
        // an item is one 128-column scale block
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float s = *reinterpret_cast<const float*>(stage + 4096 + h * 16);
#pragma unroll
          for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) sums.v[q][h][j] = fmaf(s, acc.v[q][h][j], sums.v[q][h][j]);
        }
      }
      __syncwarp();     // the stage may be filled again
      out = out + 1 == STAGES ? 0 : out + 1;
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
#pragma unroll
        for (int q = 0; q < NT; ++q)
          if (x[p][q]) x[p][q] += F::KI;
      kleft -= F::KI;
    }
  }
};

// ---------------------------------------------------------------------------------- join
constexpr int MAX_SLOTS = 48;
struct JoinShared {
  int turn[MAX_SLOTS];         // unit that may use the slot next
  int count[MAX_SLOTS];        // units done of the tile whose first unit has this slot
};

__device__ __forceinline__ void join_init(JoinShared& j) {
  if (threadIdx.x < MAX_SLOTS) {
    j.turn[threadIdx.x] = threadIdx.x;
    j.count[threadIdx.x] = 0;
  }
}

// Joins the units [u0, u0 + n) of one tile; unit u is this warp's.  Slot i % slots of `parts`
// (`stride` float4 each) belongs to unit i until its tile is summed; a warp that is `slots` units
// ahead waits for it (units are taken in order and a tile has at most `slots` of them, so the wait
// ends; it is bounded all the same).  True on the warp that has the tile's sums; false also
// after a timeout, which sets the status bit.
template <int NT>
__device__ __forceinline__ bool join(Sums<NT>& sums, JoinShared& j, float4* parts, int slots, int stride, int u, int u0,
                                     int n, int lane, int32_t* dev_status) {
  const int mine = u % slots;
  volatile int* turn = j.turn;
  if (!__all_sync(0xffffffffu, wait_for([&] { return turn[mine] == u; }, dev_status))) return false;
  if (n > 1) {
    float4* p = parts + mine * stride;
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        p[(q * 2 + h) * 32 + lane] = make_float4(sums.v[q][h][0], sums.v[q][h][1], sums.v[q][h][2], sums.v[q][h][3]);
    __threadfence_block();
    __syncwarp();
    int old = 0;
    if (lane == 0) old = atomicAdd(&j.count[u0 % slots], 1);
    old = __shfl_sync(0xffffffffu, old, 0);
    if (old != n - 1) return false;
    __threadfence_block();
    if (lane == 0) j.count[u0 % slots] = 0;
    sums.clear();
    int at = u0 % slots;
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const float4* v = parts + at * stride;
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 f = v[(q * 2 + h) * 32 + lane];
          sums.v[q][h][0] += f.x;
          sums.v[q][h][1] += f.y;
          sums.v[q][h][2] += f.z;
          sums.v[q][h][3] += f.w;
        }
      at = at + 1 == slots ? 0 : at + 1;
    }
    __threadfence_block();
    __syncwarp();
  }
  // the slots may be used again
  for (int i = u0 + lane; i < u0 + n; i += 32) turn[i % slots] = i + slots;
  return true;
}

// ---------------------------------------------------------------------- host-side layout
__host__ __device__ __forceinline__ long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// The packed 4-bit layout (moe_pack_w4): blocks of 16 rows x 256 columns, 2 KB of codes.
__host__ __device__ __forceinline__ long long w4_slices(int k) { return (k + 255) / 256; }

}  // namespace few
}  // namespace moe
