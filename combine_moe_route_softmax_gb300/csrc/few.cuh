// Weight streaming for products with a few columns (1 to 32 activation rows per weight
// matrix), shared by the few-token layer (few_layer.cuh) and the 4-bit product
// (few_linear.cu).  Internal header.
//
// The mathematics: y[n, c] = sum_k W[n, k] x[c, k] for a handful of columns c.  Every weight is
// used a few times only, so the bound is reading W once; the arithmetic rides along on
// mma.sync.m16n8k16 (16-bit operands, float32 sums), weights as the 16-row operand and activation
// rows as the 8 columns.  Per KB of weights and group of 8 columns these are 2 (BF16), 4 (E4M3) or 8 (4 bits)
// tensor instructions, twice that with two terms of more than 4 columns: the tensor pipe is 7 to 12 %
// busy in the layers, 29 % in the 24-row product, and a 128-row tcgen05 tile would have 1 to 32 columns of work.
//
// Work is cut into items: 32 weight rows (a row tile) x 128 bytes of K, 4 KB; a few neighbouring
// items of a tile are a unit.  A CTA (one per SM) takes whole tiles, one after the other.  Its
// scheduler warp writes down each unit (where it lies, whose it is) as its workers come near it,
// and the worker warps take units as they get free.  A worker's items arrive by TMA in a ring
// of its own in shared memory, one ahead of the one in use, across units and tiles.  The K
// order inside a 128-byte line is whatever the lanes hold, since a dot product does not care and
// the activations are read in the same order.  The sums of a tile's units are joined in shared
// memory by the warp that finishes last, in unit order, so the result does not depend on who
// was last.
//
// BF16 and E4M3 items keep up with the copies.  A 4-bit item holds four times the weights of a BF16 one and
// takes 700 to 900 instructions (with its share of joins and results), in one chain from the load of the codes to
// the scaling of a group's sums; three warps to a scheduler (their 168 registers allow no more) use 37 to 41 % of its
// issue slots, so 4-bit layers run at 40 % of the copies' rate, by latency before instructions.
//
// Measured with the copies alone (15 warps, two 4 KB stages each, two boxes of 16 rows an item):
// 7.1 TB/s over 1.6 GB and 6.8 over 0.4 GB, row-major or tiled; three stages no faster; per-warp
// cp.async of the same items 5.2 to 6.5 with three times the instructions; one warp feeding
// the SM with 512-byte bulk copies 2.1.
#pragma once

#include <cuda_fp16.h>

#include "gemm_common.cuh"

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
// How long the waits of a CTA last.  The first that runs out sets the status bit and gave_up, which ends
// all others, those still to come at their first look: a launch that cannot go on is over one limit later.
struct Patience {
  int* gave_up;                // shared, 0 at first
  int32_t* dev_status;         // nullable
  unsigned long long limit_ns;
  __device__ __forceinline__ bool over() const { return *static_cast<volatile int*>(gave_up) != 0; }
  __device__ __forceinline__ bool ran_out(unsigned long long t0) const {
    if (clock_ns() - t0 <= limit_ns) return false;
    *static_cast<volatile int*>(gave_up) = 1;
    if (dev_status) atomicOr(dev_status, MOE_DEV_PIPELINE_TIMEOUT);
    return true;
  }
};
// Bounded wait for done(): false if this or another wait of the CTA ran out.
template <class Done>
__device__ __forceinline__ bool wait_for(Done done, const Patience& p) {
  if (done()) return true;
  const unsigned long long t0 = clock_ns();
  while (!done()) {
    __nanosleep(40);     // a waiting warp leaves the issue slots to the others
    if (p.over() || p.ran_out(t0)) return false;
  }
  return true;
}

// The same for a whole warp: one answer for all lanes.
template <class Done>
__device__ __forceinline__ bool warp_wait_for(Done done, const Patience& p) {
  return __all_sync(0xffffffffu, wait_for(done, p));
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

// The same from zero: d = a b.
template <bool HALF>
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  if (HALF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Four E4M3 codes -> two FP16 pairs, exactly (FP16 holds every E4M3 value).
__device__ __forceinline__ void e4m3x4_to_half(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

// Eight 4-bit codes of one word minus their zero point -> four FP16 pairs (columns 0 1, 2 3, 4 5, 6 7).
// Column 2i sits at nibble i and 2i + 1 at nibble i + 4, so a mask leaves a pair of codes in
// the low mantissa bits of two 16-bit halves: 0x6400 | c is 1024 + c, and 0x6400 | 16 c is 1024 + 16 c, a
// sixteenth of which minus (64 + z) is exact in one multiply-add, for any byte z.  Integers placed under a
// fixed exponent and brought down by a subtraction are a published way of making floats of codes: Y. J.
// Kim, R. Henry, R. Fahim, H. H. Awadalla, "Who Says Elephants Can't Run: Bringing Large Scale MoE Models into Cloud
// Scale Production", 2022.
struct W4Zero {
  uint32_t a, b;               // 1024 + z and -(64 + z)
  // z in byte `sel` of the word
  __device__ __forceinline__ W4Zero(uint32_t z, int sel) {
    a = __byte_perm(z, 0x64u, 0x4040 | sel * 0x0101);
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(b) : "r"(a), "r"(0xbc00bc00u), "r"(0x63806380u));   // 960 - a
  }
};
// (v & mask) | magic in one instruction: the magic number comes in a register, which the compiler
// cannot see through (two constants would be two instructions).
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(v), "r"(mask), "r"(magic));
  return r;
}
__device__ __forceinline__ uint32_t w4_magic() {
  uint32_t r;
  asm volatile("mov.b32 %0, %1;" : "=r"(r) : "n"(0x64006400));
  return r;
}
__device__ __forceinline__ void w4_pairs(uint32_t v, const W4Zero& z, uint32_t magic, uint32_t (&p)[4]) {
  const uint32_t w = v >> 8;
  const uint32_t c0 = and_or(v, 0x000f000fu, magic), c1 = and_or(v, 0x00f000f0u, magic);
  const uint32_t c2 = and_or(w, 0x000f000fu, magic), c3 = and_or(w, 0x00f000f0u, magic);
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p[0]) : "r"(c0), "r"(z.a));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[1]) : "r"(c1), "r"(0x2c002c00u), "r"(z.b));   // 0x2c00 = 1/16
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p[2]) : "r"(c2), "r"(z.a));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[3]) : "r"(c3), "r"(0x2c002c00u), "r"(z.b));
}

// The power of two that brings a positive finite float (bits m) to [2^14, 2^15), as far as float32
// can hold it and its inverse (2^-113 .. 2^120).
__device__ __forceinline__ float to_half_scale(uint32_t m) {
  const int e = (int)(m >> 23);                            // biased exponent, 0 for 0 and subnormals
  return __uint_as_float((uint32_t)min(127 + 14 - (e - 127), 127 + 120) << 23);
}
__device__ __forceinline__ uint16_t half_bits(float v) { return __half_as_ushort(__float2half_rn(v)); }

// Largest finite magnitude of eight BF16 values, as float bits.
__device__ __forceinline__ uint32_t bf16_max(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = (w[j] << 16) & 0x7fffffffu, hi = w[j] & 0x7fff0000u;
    if (lo < 0x7f800000u) m = max(m, lo);
    if (hi < 0x7f800000u) m = max(m, hi);
  }
  return m;
}
// Eight BF16 values times sc as FP16.
__device__ __forceinline__ uint4 bf16_to_half8(const uint4& v, float sc) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = half_bits(__uint_as_float(w[j] << 16) * sc) |
           (uint32_t)half_bits(__uint_as_float(w[j] & 0xffff0000u) * sc) << 16;
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ int atom_add_release(int32_t* p, int v) {
  int old;
  asm volatile("atom.add.release.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// --------------------------------------------------------------------------------- items
// How tiles are cut: into `parts` units of `len` items (the last may have fewer).
struct Cut {
  int nsl, len, parts;
  __host__ __device__ __forceinline__ void set(int items, int n) {
    nsl = items;
    len = (items + n - 1) / n;
    parts = (items + len - 1) / len;
  }
};
// What a unit costs beside its items (join, result), in items.
constexpr int UNIT_COST = 4;

// One unit, as the scheduler writes it down.  BF16 and E4M3 items are boxes of a tensor map (128
// bytes of column, rows y0.. and y1.. for the two half tiles; per item x or the rows go on by dx,
// dy); W4 items are two blocks at p0 and p1.  E4M3: p0, p1 are the half tiles' scales.
struct __align__(16) Unit {
  const uint8_t *p0, *p1;
  const CUtensorMap* map;
  int x, y0, y1;
  int entry, row;
  short s0, n, part, parts;   // first item, items, place in the tile, units of the tile
  int down;            // layer: phase 2
};

template <int FMT, int GROUP>
struct Format {
  static constexpr int KI = FMT == F_BF16 ? 64 : FMT == F_E4M3 ? 128 : 256;   // columns per item
  static constexpr int NG = FMT == F_W4 ? 256 / GROUP : 1;                    // W4 scale groups per slice
  static constexpr int SC = 8 * NG * 4;                                       // W4 scale bytes of a block
  static constexpr int ZP = 8 * NG * 2;                                       // W4 zero-point bytes of a block
  static constexpr int HALF_CHUNKS = FMT == F_BF16 ? 1 : FMT == F_E4M3 ? 2 : 4;
  static constexpr int HALF = FMT == F_W4 ? 2048 + SC + ZP : 2048;            // bytes of a half tile in a stage
  static constexpr int STAGE = 2 * HALF;
};
// The packed 4-bit layout (moe_pack_w4): blocks of 16 rows x 256 columns -- 2 KB of codes, the
// scales, the zero points if there are any -- row block major.
__host__ __device__ __forceinline__ int w4_slices(int k) { return (k + 255) / 256; }
__host__ __device__ __forceinline__ int w4_block(int group, bool zeros) {
  return 2048 + 8 * (256 / group) * (zeros ? 6 : 4);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
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

// Where activations are: element offsets from one base, in global memory (kept in L1, which the
// weights pass by; plain loads, since the layer writes some of them in the same launch) or shared.
template <bool SMEM>
struct Acts {
  const uint16_t* base;              // global
  uint32_t addr;                     // shared
  __device__ __forceinline__ uint4 load(int off) const {
    uint4 v;
    if (SMEM)
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "r"(addr + off * 2));
    else
      v = *reinterpret_cast<const uint4*>(base + off);
    return v;
  }
};
// This lane's part of an item's columns starts at acts_lane; 16-byte chunk I of half J (J's 16 of the
// lane's 32 bytes per weight row, HALF_CHUNKS chunks of activations) is acts_chunk further on.
template <int FMT>
__device__ __forceinline__ int acts_lane(int t) { return FMT == F_BF16 ? t * 16 : FMT == F_E4M3 ? t * 32 : t * 8; }
template <int FMT>
__device__ __forceinline__ constexpr int acts_chunk(int J, int I) {
  return FMT == F_BF16 ? 8 * J : FMT == F_E4M3 ? 16 * J + 8 * I : (4 * J + I) * 32;
}

template <bool HALF, int NT>
__device__ __forceinline__ void mma_step(Sums<NT>& acc, const uint32_t (&a)[4][4], const uint4 (&b)[NT],
                                         bool first = false) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (first) mma16_first<HALF>(acc.v[n][h], a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], b[n].x, b[n].y);
      else mma16<HALF>(acc.v[n][h], a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], b[n].x, b[n].y);
      mma16<HALF>(acc.v[n][h], a[2 * h][2], a[2 * h + 1][2], a[2 * h][3], a[2 * h + 1][3], b[n].z, b[n].w);
    }
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Half an item: sums += weights x activations.  acc: E4M3 sums of the item so far, unscaled.
template <int FMT, int GROUP, bool HALF, int NT, int PASSES, class Acts>
__device__ __forceinline__ void half_item(Sums<NT>& sums, Sums<NT>& acc, const uint8_t* stage, int J, Acts acts, int lane,
                                          bool zeros) {
  using F = Format<FMT, GROUP>;
  const int g = lane >> 2, t = lane & 3;
  uint4 q[4];                      // rows g, g + 8 of the first half tile, then of the second
  // boxes come with TMA's 128-byte swizzle (16-byte chunk c of row r at c ^ (r & 7)), packed
  // blocks in lane order: 8 lanes touch every bank once either way
  const uint8_t* base = stage + (FMT == F_W4 ? J * 512 + lane * 16 : g * 128 + (((2 * t + J) ^ g) << 4));
#pragma unroll
  for (int r = 0; r < 4; ++r)
    q[r] = *reinterpret_cast<const uint4*>(base + (r >> 1) * F::HALF + (r & 1) * 1024);
  if constexpr (FMT == F_BF16) {
    uint32_t a[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) { a[r][0] = q[r].x; a[r][1] = q[r].y; a[r][2] = q[r].z; a[r][3] = q[r].w; }
    uint4 b[PASSES][NT];
    acts(b, 0);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) mma_step<HALF, NT>(sums, a, b[p]);
  } else if constexpr (FMT == F_E4M3) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 b[PASSES][NT];
      acts(b, i);
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
    constexpr int HG = F::NG / 2;     // groups of half an item
    static_assert(HALF, "codes become FP16");
    const uint32_t magic = w4_magic();
    uint32_t scs[2][HG], zps[2][(HG + 1) / 2];     // by half tile: BF16 pairs; bytes, two groups a word
    const uint8_t* par = stage + 2048 + (g * F::NG + J * HG) * 4;
    const uint8_t* zpar = stage + 2048 + F::SC + (g * F::NG + J * HG) * 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (HG == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(par + h * F::HALF);
        scs[h][0] = v.x; scs[h][1] = v.y; scs[h][2] = v.z; scs[h][3] = v.w;
        const uint2 z = zeros ? *reinterpret_cast<const uint2*>(zpar + h * F::HALF) : make_uint2(0x08080808u, 0x08080808u);
        zps[h][0] = z.x; zps[h][1] = z.y;
      } else if constexpr (HG == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(par + h * F::HALF);
        scs[h][0] = v.x; scs[h][1] = v.y;
        zps[h][0] = zeros ? *reinterpret_cast<const uint32_t*>(zpar + h * F::HALF) : 0x08080808u;
      } else {
        scs[h][0] = *reinterpret_cast<const uint32_t*>(par + h * F::HALF);
        zps[h][0] = zeros ? *reinterpret_cast<const uint16_t*>(zpar + h * F::HALF) : 0x0808u;
      }
    }
#pragma unroll
    for (int i0 = 0; i0 < 4; i0 += WPG) {
      const int gi = i0 / WPG, zb = (gi & 1) * 2;
      const W4Zero z[4] = {{zps[0][gi >> 1], zb}, {zps[0][gi >> 1], zb + 1}, {zps[1][gi >> 1], zb},
                           {zps[1][gi >> 1], zb + 1}};
      Sums<NT> part;
#pragma unroll
      for (int i = i0; i < i0 + WPG; ++i) {
        uint4 b[PASSES][NT];
        acts(b, i);
        uint32_t a[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) w4_pairs(word(q[r], i), z[r], magic, a[r]);
#pragma unroll
        for (int p = 0; p < PASSES; ++p) mma_step<HALF, NT>(part, a, b[p], i == i0 && p == 0);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float s0 = bf_lo(scs[h][gi]), s1 = bf_hi(scs[h][gi]);
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

// -------------------------------------------------------------------------------- feed
constexpr int FEED = 64;             // units written down at a time
constexpr int AHEAD = 40;            // ... past the slowest worker's
constexpr int STOCK = 4;             // ... that no worker has taken
template <int WORKERS>
struct Feed {
  Unit unit[FEED];
  int published;                     // units written down so far
  int total;                         // units of the CTA, once known
  int next;                          // unit to take next
  int use[WORKERS];                  // unit each worker is at
  unsigned long long full[WORKERS][2];
};
template <int WORKERS>
__device__ __forceinline__ void feed_init(Feed<WORKERS>& f) {
  if (threadIdx.x == 0) {
    f.published = 0;
    f.total = 0x7fffffff;
    f.next = 0;
    for (int i = 0; i < WORKERS; ++i)
      for (int j = 0; j < 2; ++j) gg::mbar_init(gg::smem_u32(&f.full[i][j]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x < WORKERS) f.use[threadIdx.x] = 0;
}

// Units off the feed, as one worker takes them.
template <int WORKERS>
struct FeedSource {
  Feed<WORKERS>& feed;
  int worker;
  __device__ __forceinline__ int claim(int lane) {
    int u = 0;
    if (lane == 0) u = atomicAdd(&feed.next, 1);
    return __shfl_sync(0xffffffffu, u, 0);
  }
  // 1: unit u is written down, 2: there is no such unit, 0: not known yet
  __device__ __forceinline__ int state(int u, int lane) const {
    int go = 0;
    if (lane == 0) {
      volatile int *published = &feed.published, *total = &feed.total;
      go = *published > u ? 1 : *total <= u ? 2 : 0;
    }
    go = __shfl_sync(0xffffffffu, go, 0);
    __threadfence_block();
    return go;
  }
  __device__ __forceinline__ const Unit& unit(int u) const { return feed.unit[u & (FEED - 1)]; }
  __device__ __forceinline__ void at(int u, int lane) const {
    if (lane == 0) *static_cast<volatile int*>(&feed.use[worker]) = u;
  }
};

// A worker warp's stream of units: take() moves to the next one (false at the end), run() multiplies
// it.  The item after the one in use is always on its way.  Src gives the units (FeedSource, or one
// that works them out).
template <int FMT, int GROUP, bool HALF, bool SMEM, class Src>
struct Stream {
  using F = Format<FMT, GROUP>;
  Src src;
  uint8_t* ring;               // two stages
  uint32_t ring_addr, bars;    // shared addresses of the ring and of its two barriers
  int lane;
  Patience patience;
  int dx, dy;                  // tensor maps: from one item to the next
  int block;                   // W4: bytes of a block
  bool zeros;
  int stage;                   // of the item in use: bit 0, and its barriers' phase above
  static constexpr int END = 0x7fffffff;
  int filled;                  // unit of the item on its way; END past the last
  bool pending;                // ... which is not written down yet
  int left, x, y0, y1;         // its items still to be asked for, and where they are
  const uint8_t *p0, *p1;
  const CUtensorMap* map;
  int cur;                     // unit in use
  // Set when a wait gave up: 1 with at most the item after the last one run on its way (filled, pending), 2
  // with the item that was waited for, 3 with that and the next.
  int dead;

  // Asks for the next item, into stage st.  It never waits while a unit is in use: the scheduler waits
  // for the slowest worker, which must not wait for it in turn.  If the next unit is not written
  // down yet, take() waits for it, when this worker holds nothing up.
  __device__ __forceinline__ void fill(int st) {
    if (left == 0) {
      if (filled == END) return;
      if (!pending) {            // the next unit
        filled = src.claim(lane);
        pending = true;
      }
      const int go = src.state(filled, lane);
      if (go == 0) return;
      pending = false;
      if (go == 2) {
        filled = END;
        return;
      }
      const Unit& k = src.unit(filled);
      left = k.n;
      p0 = k.p0;
      p1 = k.p1;
      if constexpr (FMT != F_W4) {
        x = k.x;
        y0 = k.y0;
        y1 = k.y1;
        map = k.map;
      }
    }
    if (lane == 0) {
      const uint32_t d = ring_addr + st * F::STAGE, bar = bars + st * 8;
      if constexpr (FMT == F_W4) {
        gg::mbar_expect_tx(bar, 2 * block);
        bulk_load(d, p0, block, bar);
        bulk_load(d + F::HALF, p1, block, bar);
      } else {
        gg::mbar_expect_tx(bar, 4096);
        gg::tma_load_2d(d, map, x, y0, bar);
        gg::tma_load_2d(d + 2048, map, x, y1, bar);
      }
    }
    if constexpr (FMT == F_W4) {
      p0 += block;
      p1 += block;
    } else {
      x += dx;
      y0 += dy;
      y1 += dy;
    }
    --left;
  }
  __device__ __forceinline__ void start() {
    stage = 0;
    left = 0;
    filled = 0;
    pending = false;
    dead = 0;
    fill(0);
  }
  __device__ __forceinline__ bool take() {
    if (dead) return false;
    if (filled != END) src.at(filled, lane);
    if (pending) {
      const unsigned long long t0 = clock_ns();
      while (true) {             // the lanes stay together: fill() is the whole warp's
        fill(stage & 1);
        if (!pending) break;
        __nanosleep(40);
        if (__any_sync(0xffffffffu, patience.over() || patience.ran_out(t0))) {
          dead = 1;
          return false;
        }
      }
    }
    cur = filled;
    return cur != END;
  }
  __device__ __forceinline__ void finish() {
    // given up: the items on their way arrive before the block ends
    if (dead >= 2 || (dead && !pending && filled != END)) gg::mbar_drain(bars + (stage & 1) * 8, (stage >> 1) & 1);
    if (dead == 3) gg::mbar_drain(bars + ((stage + 1) & 1) * 8, ((stage + 1) >> 1) & 1);
    src.at(0x7ffff000, lane);    // far past any unit
  }

  // sums = weights x activations over the unit in use.  off[p][n] is where this lane's column of group n
  // (any column, if it has none: its sums are dropped) begins; PASSES sets of columns are added
  // into the same sums.  With scaled (FP16 only), 16 values of a column share an exponent: ex[n] are those
  // of the lane's column, and they count from top[n].  Rows of activations reach to whole items (W4: 256
  // columns), with zeros.  False if a wait gave up.
  template <int NT, int PASSES>
  __device__ __forceinline__ bool run(Sums<NT>& sums, const Acts<SMEM>& from, const int (&off)[PASSES][NT],
                                      bool scaled = false, const uint8_t* const* ex = nullptr,
                                      const int* top = nullptr) {
    const int t = lane & 3;
    const Unit& un = src.unit(cur);
    const int s0 = un.s0, n = un.n;
    int at[PASSES][NT];
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
#pragma unroll
      for (int i = 0; i < NT; ++i) at[p][i] = off[p][i] + s0 * F::KI + acts_lane<FMT>(t);
    const float *sc0 = nullptr, *sc1 = nullptr;
    if constexpr (FMT == F_E4M3) {
      sc0 = reinterpret_cast<const float*>(un.p0);
      sc1 = reinterpret_cast<const float*>(un.p1);
    }
    sums.clear();
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      // the first half's activations are on their way before the weights are waited for
      uint4 b[F::HALF_CHUNKS][PASSES][NT];
      uint2 e8[NT];
      auto ask = [&](int J) {
#pragma unroll
        for (int q = 0; q < F::HALF_CHUNKS; ++q)
#pragma unroll
          for (int p = 0; p < PASSES; ++p)
#pragma unroll
            for (int c = 0; c < NT; ++c) b[q][p][c] = from.load(at[p][c] + acts_chunk<FMT>(J, q));
      };
      // exponents of half J: E4M3 one (the lane's 16 columns), W4 eight (words 4J.. of two blocks each)
      auto ask_exps = [&](int J) {
        if constexpr (HALF) {
          if (!scaled) return;
          const int e0 = (s0 + i) * (F::KI / 16) + (FMT == F_E4M3 ? t * 2 + J : 8 * J);
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            if constexpr (FMT == F_E4M3) e8[q].x = ex[q][e0];
            else e8[q] = *reinterpret_cast<const uint2*>(ex[q] + e0);
          }
        }
      };
      constexpr bool EARLY = F::HALF_CHUNKS * NT * PASSES <= 8;   // else as they are used: registers
      if constexpr (EARLY) ask(0);
      ask_exps(0);
      fill((stage ^ 1) & 1);
      float f0 = 1.0f, f1 = 1.0f;
      if constexpr (FMT == F_E4M3) {
        f0 = __ldg(sc0 + i);
        f1 = __ldg(sc1 + i);
      }
      const uint32_t bar = bars + (stage & 1) * 8, phase = (stage >> 1) & 1;
      if (!warp_wait_for([&] { return gg::mbar_try_wait(bar, phase); }, patience)) {
        dead = i + 1 < n || (!pending && filled != END) ? 3 : 2;
        return false;
      }
      const uint8_t* st = ring + (stage & 1) * F::STAGE;
      Sums<NT> acc;
      if constexpr (FMT == F_E4M3) acc.clear();
      // rolled: one copy of the arithmetic, which several variants of this function share the
      // instruction cache with
#pragma unroll 1
      for (int J = 0; J < 2; ++J) {
        auto acts = [&](uint4(&v)[PASSES][NT], int I) {
#pragma unroll
          for (int p = 0; p < PASSES; ++p) {
            if constexpr (EARLY) {
#pragma unroll
              for (int q = 0; q < NT; ++q) v[p][q] = b[I][p][q];
            } else {
#pragma unroll
              for (int q = 0; q < NT; ++q) v[p][q] = from.load(at[p][q] + acts_chunk<FMT>(J, I));
            }
          }
          if constexpr (HALF) {
            if (scaled) {
#pragma unroll
              for (int q = 0; q < NT; ++q) {
                // bytes 2 I + (t >> 1) of the eight; 2^(exponent - top), 0 where FP16 ends
                const int e = FMT == F_E4M3 ? e8[q].x : ((I < 2 ? e8[q].x : e8[q].y) >> (16 * (I & 1) + 8 * (t >> 1))) & 255;
                const float f = __uint_as_float((uint32_t)(127 + max(min(e - top[q], 0), -30)) << 23);
                const __half2 h = __float2half2_rn(f);
#pragma unroll
                for (int p = 0; p < PASSES; ++p) {
                  __half2* w = reinterpret_cast<__half2*>(&v[p][q]);
#pragma unroll
                  for (int j = 0; j < 4; ++j) w[j] = __hmul2(w[j], h);
                }
              }
            }
          }
        };
        half_item<FMT, GROUP, HALF, NT, PASSES>(sums, acc, st, J, acts, lane, zeros);
        if (J == 0) {
          if constexpr (EARLY) ask(1);
          ask_exps(1);
        }
      }
      if constexpr (FMT == F_E4M3) {
        // an item is one 128-column scale block
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) sums.v[q][h][j] = fmaf(h ? f1 : f0, acc.v[q][h][j], sums.v[q][h][j]);
      }
      __syncwarp();     // the stage may be filled again
      ++stage;          // bit 0: the stage; bit 1: its phase
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
#pragma unroll
        for (int q = 0; q < NT; ++q) at[p][q] += F::KI;
    }
    return true;
  }
};

// The scheduler warp.  Src says what the CTA's sequence of tiles is: next(t, n) the next run of tiles
// t, t + 1, ... (false past the end), cut(t), same(t) (how many from t on are cut alike),
// describe(t, part, cut, unit), and idle(), called every time round (true if it got something done).
constexpr int BATCH = 16;            // units written down at a time
template <int WORKERS, int SIZE, class Src>
__device__ __forceinline__ void schedule(Feed<SIZE>& f, Src& src, int lane, const Patience& patience) {
  volatile int* use = f.use;
  int units = 0, t = 0, n = 0;
  bool end = false;
  unsigned long long t0 = clock_ns();
  while (!end || !src.done()) {
    bool moved = src.idle(lane);
    // few units in stock: what an SM holds ready at the end, the others do without
    volatile int* next = &f.next;
    const int most = __reduce_min_sync(
        0xffffffffu, lane < WORKERS ? use[lane] + AHEAD : lane == WORKERS ? *next + STOCK : 0x7fffffff);
    if (!end && units < most) {
      if (n == 0 && !src.next(lane, t, n)) {
        end = true;
        if (lane == 0) *static_cast<volatile int*>(&f.total) = units;
      } else {
        const Cut c = src.cut(t);
        const int m = min(min(n, src.same(t)), max(1, BATCH / c.parts));
        const int i = lane / c.parts;
        if (i < m) src.describe(t + i, lane - i * c.parts, c, f.unit[(units + lane) & (FEED - 1)]);
        __threadfence_block();
        __syncwarp();
        units += m * c.parts;
        if (lane == 0) *static_cast<volatile int*>(&f.published) = units;
        t += m;
        n -= m;
      }
      moved = true;
    }
    if (moved) {
      t0 = clock_ns();
    } else {
      if (__any_sync(0xffffffffu, patience.over() || patience.ran_out(t0))) return;   // the workers leave too
      __nanosleep(60);
    }
  }
}

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
// ends; it is bounded all the same).  It also waits for the first unit's slot, whose count the tile
// uses: where tiles of more parts follow ones of fewer, the tile that had that slot before may
// not be the one that had this unit's.  True on the warp that has the tile's sums; false also when a
// wait gave up: the tile is never summed, and what else the CTA waits for gives up at once.
template <int NT>
__device__ __forceinline__ bool join(Sums<NT>& sums, JoinShared& j, float4* parts, int slots, int stride, int u, int u0,
                                     int n, int lane, const Patience& patience) {
  const int mine = u % slots, head = u0 % slots;
  volatile int* turn = j.turn;
  if (!warp_wait_for([&] { return turn[mine] == u && turn[head] == u0; }, patience)) return false;
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
    if (lane == 0) old = atomicAdd(&j.count[head], 1);
    old = __shfl_sync(0xffffffffu, old, 0);
    if (old != n - 1) return false;
    __threadfence_block();
    if (lane == 0) j.count[head] = 0;
    sums.clear();
    int at = head;
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

}  // namespace few
}  // namespace moe
