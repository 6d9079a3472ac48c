// Weight streaming for products with a few columns (1 to 16 activation rows per weight
// matrix), shared by the few-token layer (few_layer.cuh) and the 4-bit product
// (few_linear.cu).  Internal header.
//
// The mathematics: y[n, c] = sum_k W[n, k] x[c, k] for a handful of columns c.  Every weight is
// used a few times only, so the bound is reading W once; the arithmetic rides along on
// mma.sync.m16n8k16 (BF16 in, float32 sums), weights as the 16-row operand and activation
// rows as the 8 columns -- 2 to 4 tensor instructions per KB of weights, far below any
// tensor-core limit, which is why these kernels do not use the 128-row tcgen05 tiles.
//
// Work is cut into items: 32 weight rows x 128 bytes of K, 4 KB.  The items of a launch
// phase, in the order (matrix, row tile, K slice) or (row tile, matrix, K slice), are
// divided evenly over the workers (16 warps per SM), each taking one contiguous run, so every
// SM reads the same number of bytes whatever the shapes (to one item).  A warp reads an
// item as four 256-bit loads per lane, each 8 rows x one whole 128-byte line, straight into
// the registers the tensor instruction takes them from: the K order inside a line is
// whatever the lanes hold, since a dot product does not care and the activations are read
// in the same order.  Measured with loads alone, 1.6 GB row-major: 7.0 TB/s so; 5.5 with
// 128-bit loads (8 rows x 64 bytes); 6.5 without the 256-byte L2 prefetch hint; 5.5 through
// 16-byte cp.async into shared memory by four warps; 2.1 through 512-byte bulk copies.
//
// A row tile whose slices fall to several workers is joined by the one that finishes last:
// each writes its partial sums, fences and counts; the last adds all parts in worker
// order, so the result does not depend on who was last.  Nobody waits.
#pragma once

#include "common.cuh"

namespace moe {
namespace few {

constexpr int WARPS = 16;
constexpr int THREADS = WARPS * 32;
constexpr int kMaxTokens = MOE_FEW_MAX_TOKENS;
constexpr int COLS = 16;             // columns of one matrix handled in one pass over it
constexpr int PART_FLOATS = 1024;    // one worker's partial sums: 32 rows x 32 columns
constexpr unsigned long long TIMEOUT_NS = 2000000000ull;

enum { F_BF16 = 0, F_E4M3 = 1, F_W4 = 2 };

struct V8 {
  uint32_t x[8];
};
// Read-once weights: not kept in L1, the neighbouring 128 bytes fetched into L2 with them.
__device__ __forceinline__ V8 ld_weights(const uint8_t* p) {
  V8 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v.x[0]), "=r"(v.x[1]), "=r"(v.x[2]), "=r"(v.x[3]), "=r"(v.x[4]), "=r"(v.x[5]), "=r"(v.x[6]),
                 "=r"(v.x[7])
               : "l"(p));
  return v;
}
// Activations: kept in L1 (the warps of an SM read the same rows); not .nc, since the layer
// writes some of them in the same launch.
__device__ __forceinline__ uint4 ld_act(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two E4M3 codes in the low byte of each half of h -> two BF16, exactly: the sign to bit 15,
// the other 7 bits behind a zeroed upper exponent give the value times 2^-120 (a subnormal
// BF16 for a subnormal code), and the product with 2^120 is exact.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t h) {
  const uint32_t m = ((h >> 4) & 0x07f007f0u) | (h & 0x80008000u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(0x7b807b80u));   // 0x7b80 = 2^120
  return r;
}

// ------------------------------------------------------------------------- work division
// Worker w of W takes items [F*w/W, F*(w+1)/W).
__host__ __device__ __forceinline__ long long run_start(long long F, long long w, long long W) { return F * w / W; }
__host__ __device__ __forceinline__ int worker_of(long long f, long long F, long long W) {
  return (int)(((f + 1) * W - 1) / F);
}
// Workers used for F items: all, unless that leaves them less than `least` items each.
__host__ __device__ __forceinline__ int workers_for(long long F, int all, int least) {
  const long long n = (F + least - 1) / least;
  return n < all ? (int)n : all;
}
// The worker this warp is: neighbouring warps of an SM take neighbouring runs when all
// workers are used; fewer are spread over the SMs first.
__device__ __forceinline__ int my_worker(int W, int cta, int ctas, int warp) {
  if (W >= ctas * WARPS) return cta * WARPS + warp;
  const int w = warp * ctas + cta;
  return w < W ? w : -1;
}

// Where a lane finds one row tile's items.
struct Tile {
  const uint8_t* w;    // this lane's 32 bytes of row g of the first half tile, at slice s0
  const void* sc;      // scales at slice s0 (E4M3: first half tile's block; W4: this lane's)
  const void* zp;      // W4 zero points at slice s0, or null
  int s0, n;           // slices [s0, s0 + n) of the tile
};
// Constant strides of a phase's matrices.
struct Strides {
  long long step;      // bytes from one slice to the next
  long long row8;      // bytes from row r to row r + 8
  long long half;      // bytes from the first half tile (16 rows) to the second
  long long sc_half;   // scale elements from the first half tile to the second
  int k;               // columns
  int nsl;             // slices per row
};

// One item's weights with their scales.
template <int FMT, int GROUP>
struct Item {
  static constexpr int NG = FMT == F_W4 ? 256 / GROUP : 1;   // scale groups per slice
  V8 q[4];                 // rows g, g + 8 of the first half tile, then of the second
  uint32_t sc[2][NG];      // E4M3: float bits; W4: BF16 pair (row g, row g + 8)
  uint32_t zp[2][(NG + 1) / 2];   // W4: byte pairs (row g, row g + 8), two groups per word

  __device__ __forceinline__ void load(const uint8_t* w, const void* scales, const void* zeros, const Strides& st) {
    q[0] = ld_weights(w);
    q[1] = ld_weights(w + st.row8);
    q[2] = ld_weights(w + st.half);
    q[3] = ld_weights(w + st.half + st.row8);
    if constexpr (FMT == F_E4M3) {
      const uint32_t* s = static_cast<const uint32_t*>(scales);
      sc[0][0] = __ldg(s);
      sc[1][0] = __ldg(s + st.sc_half);
    }
    if constexpr (FMT == F_W4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t* s = static_cast<const uint32_t*>(scales) + h * st.sc_half;
        if constexpr (NG == 2) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(s));
          sc[h][0] = v.x; sc[h][1] = v.y;
        } else {
#pragma unroll
          for (int i = 0; i < NG / 4; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(s) + i);
            sc[h][4 * i] = v.x; sc[h][4 * i + 1] = v.y; sc[h][4 * i + 2] = v.z; sc[h][4 * i + 3] = v.w;
          }
        }
        if (zeros) {
          const uint16_t* z = static_cast<const uint16_t*>(zeros) + h * st.sc_half;
          if constexpr (NG == 2) {
            zp[h][0] = __ldg(reinterpret_cast<const uint32_t*>(z));
          } else if constexpr (NG == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(z));
            zp[h][0] = v.x; zp[h][1] = v.y;
          } else {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(z));
            zp[h][0] = v.x; zp[h][1] = v.y; zp[h][2] = v.z; zp[h][3] = v.w;
          }
        }
      }
    }
  }
  // bytes / elements from one slice's scales to the next, per lane pointer
  static __device__ __forceinline__ const void* next_scales(const void* p) {
    if constexpr (FMT == F_E4M3) return static_cast<const uint32_t*>(p) + 1;
    if constexpr (FMT == F_W4) return static_cast<const uint32_t*>(p) + 8 * NG;
    return p;
  }
  static __device__ __forceinline__ const void* next_zeros(const void* p) {
    if constexpr (FMT == F_W4) return p ? static_cast<const uint16_t*>(p) + 8 * NG : p;
    return p;
  }
};

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

// sums += (weights of one item) x (activations); x[n] is this lane's column of group n at
// column k0 of the item (null: no such column, zeros); kleft: columns from k0 to the end of
// the row (W4 rows are padded to whole items, activations are not).
template <int FMT, int GROUP, int NT>
__device__ __forceinline__ void item_mma(Sums<NT>& sums, const Item<FMT, GROUP>& it, const uint16_t* const (&x)[NT],
                                         int t, int kleft, bool zeros) {
  const uint4 zero4 = make_uint4(0, 0, 0, 0);
  if constexpr (FMT == F_BF16) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {   // 8 of this lane's 16 columns: two k-steps
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = x[n] ? ld_act(x[n] + t * 16 + 8 * j) : zero4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const V8 &lo = it.q[2 * h], &hi = it.q[2 * h + 1];
          mma_bf16(sums.v[n][h], lo.x[4 * j], hi.x[4 * j], lo.x[4 * j + 1], hi.x[4 * j + 1], b.x, b.y);
          mma_bf16(sums.v[n][h], lo.x[4 * j + 2], hi.x[4 * j + 2], lo.x[4 * j + 3], hi.x[4 * j + 3], b.z, b.w);
        }
      }
    }
  } else if constexpr (FMT == F_E4M3) {
    // an item is one 128-column scale block: unscaled sums first, then one multiply-add each
    Sums<NT> acc;
    acc.clear();
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // 8 of this lane's 32 columns: two k-steps
      uint32_t a[4][4];             // [row][pair of columns]
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t q = it.q[r].x[2 * j + i];
          a[r][2 * i] = e4m3x2_to_bf16x2(__byte_perm(q, 0, 0x1404));       // bytes 0, 1 to the top of each half
          a[r][2 * i + 1] = e4m3x2_to_bf16x2(__byte_perm(q, 0, 0x3424));   // bytes 2, 3
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = x[n] ? ld_act(x[n] + t * 32 + 8 * j) : zero4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma_bf16(acc.v[n][h], a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], b.x, b.y);
          mma_bf16(acc.v[n][h], a[2 * h][2], a[2 * h + 1][2], a[2 * h][3], a[2 * h + 1][3], b.z, b.w);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float s = __uint_as_float(it.sc[h][0]);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums.v[n][h][i] = fmaf(s, acc.v[n][h][i], sums.v[n][h][i]);
    }
  } else {
    // Word j of the lane's 8 holds columns j*32 + t*8 .. + 8, column 2i at nibble i and 2i + 1
    // at nibble i + 4: a mask leaves a pair of codes in the low mantissa bits of two BF16
    // halves, 0x4300 | c is exactly 128 + c, and minus (128 + zero point) is exact.
    constexpr int WPG = GROUP / 32;   // words per scale group
#pragma unroll
    for (int gi = 0; gi < Item<FMT, GROUP>::NG; ++gi) {
      Sums<NT> acc;
      acc.clear();
      uint32_t off[4];               // 128 + zero point, per row, as a BF16 pair
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (zeros) {
          const uint32_t z = it.zp[r >> 1][gi >> 1];
          off[r] = __byte_perm(z, 0x43u, ((gi & 1) * 2 + (r & 1)) * 0x0101 | 0x4040);
        } else {
          off[r] = 0x43084308u;
        }
      }
#pragma unroll
      for (int jj = 0; jj < WPG; ++jj) {
        const int j = gi * WPG + jj;
        uint32_t a[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t c = ((it.q[r].x[j] >> (4 * i)) & 0x000f000fu) | 0x43004300u;
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(a[r][i]) : "r"(c), "r"(off[r]));
          }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 b = x[n] && j * 32 + t * 8 < kleft ? ld_act(x[n] + j * 32 + t * 8) : zero4;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            mma_bf16(acc.v[n][h], a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], b.x, b.y);
            mma_bf16(acc.v[n][h], a[2 * h][2], a[2 * h + 1][2], a[2 * h][3], a[2 * h + 1][3], b.z, b.w);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float s0 = bf_lo(it.sc[h][gi]), s1 = bf_hi(it.sc[h][gi]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          sums.v[n][h][0] = fmaf(s0, acc.v[n][h][0], sums.v[n][h][0]);
          sums.v[n][h][1] = fmaf(s0, acc.v[n][h][1], sums.v[n][h][1]);
          sums.v[n][h][2] = fmaf(s1, acc.v[n][h][2], sums.v[n][h][2]);
          sums.v[n][h][3] = fmaf(s1, acc.v[n][h][3], sums.v[n][h][3]);
        }
      }
    }
  }
}

// Items [cur.s0, cur.s0 + cur.n) of one tile.  `it` holds the first item's weights on entry
// and the first of the next tile's (next, if it has any) on return: the next item's loads are
// in flight while this one's are used.
template <int FMT, int GROUP, int NT>
__device__ __forceinline__ void run_tile(Sums<NT>& sums, Item<FMT, GROUP>& it, const Tile& cur, const Tile& next,
                                         const Strides& st, const uint16_t* const (&x0)[NT], int t) {
  constexpr int KI = FMT == F_BF16 ? 64 : FMT == F_E4M3 ? 128 : 256;   // columns per item
  const uint8_t* w = cur.w;
  const void* sc = cur.sc;
  const void* zp = cur.zp;
  const uint16_t* x[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) x[n] = x0[n] ? x0[n] + (long long)cur.s0 * KI : nullptr;
  int kleft = st.k - cur.s0 * KI;
  const bool zeros = cur.zp != nullptr;
  sums.clear();
  for (int i = 0; i < cur.n; ++i) {
    const Item<FMT, GROUP> use = it;
    if (i + 1 < cur.n) {
      w += st.step;
      sc = Item<FMT, GROUP>::next_scales(sc);
      zp = Item<FMT, GROUP>::next_zeros(zp);
      it.load(w, sc, zp, st);
    } else if (next.n > 0) {
      it.load(next.w, next.sc, next.zp, st);
    }
    item_mma<FMT, GROUP, NT>(sums, use, x, t, kleft, zeros);
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (x[n]) x[n] += KI;
    kleft -= KI;
  }
}

// This worker's part of a tile whose items belong to workers w0..w1: true on the warp that
// completes it, with the whole sums.  slot: 1 if the part starts the tile, else 0 (a worker has
// at most one of each in flight).  count: one word per worker, zero between launches.
template <int NT>
__device__ __forceinline__ bool join_parts(Sums<NT>& sums, float* part, int32_t* count, int worker, int slot, int w0,
                                           int w1, int lane) {
  float4* mine = reinterpret_cast<float4*>(part + ((size_t)worker * 2 + slot) * PART_FLOATS);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      __stcg(&mine[(n * 2 + h) * 32 + lane],
             make_float4(sums.v[n][h][0], sums.v[n][h][1], sums.v[n][h][2], sums.v[n][h][3]));
  __threadfence();
  __syncwarp();
  int old = 0;
  if (lane == 0) old = atomicAdd(&count[w0], 1);
  old = __shfl_sync(0xffffffffu, old, 0);
  if (old != w1 - w0) return false;
  __threadfence();
  if (lane == 0) count[w0] = 0;
  sums.clear();
  for (int w = w0; w <= w1; ++w) {
    const float4* p = reinterpret_cast<const float4*>(part + ((size_t)w * 2 + (w == w0 ? 1 : 0)) * PART_FLOATS);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 v = __ldcg(&p[(n * 2 + h) * 32 + lane]);
        sums.v[n][h][0] += v.x;
        sums.v[n][h][1] += v.y;
        sums.v[n][h][2] += v.z;
        sums.v[n][h][3] += v.w;
      }
  }
  return true;
}

// ---------------------------------------------------------------------- host-side layout
__host__ __device__ __forceinline__ long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// The packed 4-bit layout (moe_pack_w4): blocks of 16 rows x 256 columns, 2 KB of codes.
__host__ __device__ __forceinline__ long long w4_slices(int k) { return (k + 255) / 256; }

}  // namespace few
}  // namespace moe
