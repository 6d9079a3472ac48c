// moe_linear_e4m3: out[t, n] = sum_b xs[t, b] * ws[n / 128, b] * (sum over the 128 columns k of block b of
// x[t, k] * w[n, k]) (+ bias[n]), x and w E4M3, every sum in float32, one rounding at the end.
//
// The weights are the 16-row operand of mma.sync and the rows of x its 8 columns.  A 128-column block is four
// instructions of 32 columns; which column sits where inside a block does not matter as long as both operands agree, so a
// lane loads 16 consecutive bytes of a row and uses them as the operands of two instructions.
#include "gemm_common.cuh"
#include "linear_e4m3.cuh"

namespace moe {
namespace lin8 {

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int FEW_WARPS = 16, FEW_COLS = 16;
constexpr int ITEM = 4096, RING = 2;               // bytes of an item; items that a warp has in flight
template <int NT, int MT>
constexpr int few_smem() { return FEW_WARPS * RING * ITEM + 2 * FEW_WARPS * NT * MT * 512 + FEW_WARPS * RING * 8 + 1024; }

// Up to 8 NT rows of x.  A warp's unit is an item: 16 MT weight rows x 2 / MT K blocks, 4 KB by one TMA copy into the warp's ring,
// RING items in flight per warp (131 KB an SM), on across tiles, so that the memory never waits for a tile to be finished.
// A CTA's round is `tiles` row tiles (more than one where K has fewer than eight items): warp w takes item w, and of long
// rows w + 16, w + 32, ..  The warps' sums of a tile meet in shared memory and are added in their order.
template <int NT, int MT>
__global__ void __launch_bounds__(FEW_WARPS * 32, 1)
    linear_few_kernel(const __grid_constant__ CUtensorMap tm, const Args a, int tiles) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int ROWS = 16 * MT, CHUNK = 2 / MT, SUMS = NT * MT * 128;         // SUMS: of a warp
  float* part = reinterpret_cast<float*>(smem + FEW_WARPS * RING * ITEM);     // [2][warp][MT][NT][4][32]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int kblocks = a.K / 128, chunks = (kblocks + CHUNK - 1) / CHUNK;
  const int rounds = (a.N + ROWS * tiles - 1) / (ROWS * tiles);
  uint8_t* ring = smem + warp * RING * ITEM;
  const uint32_t bars = gg::smem_u32(smem + FEW_WARPS * RING * ITEM + 2 * FEW_WARPS * SUMS * 4) + warp * RING * 8;
  if (lane < RING) gg::mbar_init(bars + 8 * lane, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();

  // this warp's items in order: round, chunk of the row
  const bool busy = warp < tiles * chunks;
  const int first = tiles > 1 ? warp % chunks : warp, tile = tiles > 1 ? warp / chunks : 0;
  int load_round = busy && !a.mute ? (int)blockIdx.x : rounds, load_chunk = first;
  uint32_t armed = 0;          // stages with a copy that was not waited for
  auto load = [&](int stage) {
    if (load_round >= rounds) return;
    if (lane == 0) {
      const uint32_t bar = bars + 8 * stage;
      gg::mbar_expect_tx(bar, ITEM);     // rows past N and blocks past K arrive as zeros
      asm volatile(
          "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
              gg::smem_u32(ring + stage * ITEM)),
          "l"(reinterpret_cast<uint64_t>(&tm)), "r"(0), "r"((load_round * tiles + tile) * ROWS), "r"(load_chunk * CHUNK), "r"(bar)
          : "memory");
    }
    armed |= 1u << stage;
    load_chunk += FEW_WARPS;
    if (load_chunk >= chunks) {
      load_chunk = first;
      load_round += gridDim.x;
    }
  };
  for (int i = 0; i < RING; ++i) load(i);

  const uint8_t* x[NT];
  const float* xs[NT][2];      // rows past the last one repeat it; their sums are not stored
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    x[i] = a.x + (size_t)min(8 * i + g, a.T - 1) * a.K + 16 * c;
#pragma unroll
    for (int h = 0; h < 2; ++h) xs[i][h] = a.x_scales + (size_t)min(8 * i + 2 * c + h, a.T - 1) * kblocks;
  }
  int stage = 0, side = 0;
  uint32_t phase = 0;
  bool dead = false;           // a wait ran out: nothing more is loaded or added, the rounds are still walked through
  for (int round = blockIdx.x; round < rounds; round += gridDim.x, side ^= 1) {
    const int t0 = (round * tiles + tile) * ROWS;
    float acc[MT][NT][4] = {};
    if (busy) {
      const float* ws = a.w_scales + (size_t)(min(t0, a.N - 1) / 128) * kblocks;
      for (int chunk = first; chunk < chunks; chunk += FEW_WARPS) {
        const int kb = chunk * CHUNK, n = min(CHUNK, kblocks - kb);
        uint4 b[CHUNK][NT][2];
        float sw[CHUNK], sx[CHUNK][NT][2];
#pragma unroll
        for (int j = 0; j < CHUNK; ++j) {
          const int k = kb + min(j, n - 1);
          sw[j] = __ldg(ws + k);
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              b[j][i][h] = __ldg(reinterpret_cast<const uint4*>(x[i] + (size_t)k * 128 + 64 * h));
              sx[j][i][h] = __ldg(xs[i][h] + k);
            }
        }
        if (!dead) {
          const uint32_t bar = bars + 8 * stage;
          if (!gg::mbar_try_wait(bar, phase)) {
            const unsigned long long since = gg::globaltimer();
            bool got = false;
            while (!(got = gg::mbar_try_wait(bar, phase)) && gg::globaltimer() - since <= a.limit_ns) {
            }
            dead = !got;
          }
          dead = __any_sync(0xffffffffu, dead);
        }
        if (dead) continue;
        const uint8_t* w0 = ring + stage * ITEM + g * 128;
#pragma unroll
        for (int j = 0; j < CHUNK; ++j) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint4 p[2], q[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // 16-byte pieces of a row lie where the copy's 128-byte swizzle put them
              const uint8_t* from = w0 + (j * ROWS + 16 * m) * 128 + (((c + 4 * h) ^ g) << 4);
              p[h] = *reinterpret_cast<const uint4*>(from);
              q[h] = *reinterpret_cast<const uint4*>(from + 1024);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              float d[4] = {};
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                mma_e4m3(d, p[h].x, q[h].x, p[h].y, q[h].y, b[j][i][h].x, b[j][i][h].y);
                mma_e4m3(d, p[h].z, q[h].z, p[h].w, q[h].w, b[j][i][h].z, b[j][i][h].w);
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float s = j < n ? __fmul_rn(sx[j][i][h], sw[j]) : 0.0f;   // past K: zeros
                acc[m][i][h] = fmaf(d[h], s, acc[m][i][h]);
                acc[m][i][2 + h] = fmaf(d[2 + h], s, acc[m][i][2 + h]);
              }
            }
          }
        }
        __syncwarp();          // every lane has read the item
        armed &= ~(1u << stage);
        load(stage);
        if (++stage == RING) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    float* mine = part + (side * FEW_WARPS + warp) * SUMS + lane;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) mine[((m * NT + i) * 4 + v) * 32] = acc[m][i][v];
    __syncthreads();           // the other side was read before the barrier of the round before
    for (int e = threadIdx.x; e < tiles * ROWS * a.T; e += FEW_WARPS * 32) {
      // element: row r of the round's rows, column t
      const int t = e / (ROWS * tiles), r = e - t * ROWS * tiles, row = round * tiles * ROWS + r;
      if (row >= a.N) continue;
      const int l = (r & 7) * 4 + ((t & 7) >> 1), v = ((r >> 3) & 1) * 2 + (t & 1);
      const int of = r / ROWS, m = (r / 16) % MT;
      const int w0 = tiles > 1 ? of * chunks : 0, w1 = tiles > 1 ? w0 + chunks : min(FEW_WARPS, chunks);
      const float* from = part + side * FEW_WARPS * SUMS + (m * NT + (t >> 3)) * 128 + v * 32 + l;
      float s = from[w0 * SUMS];
      for (int w = w0 + 1; w < w1; ++w) s = __fadd_rn(s, from[w * SUMS]);
      if (a.bias) s = __fadd_rn(s, a.bias[row]);
      const long long o = (long long)t * a.out_stride + row;
      if (a.out_f32)
        static_cast<float*>(a.out)[o] = s;
      else
        static_cast<uint16_t*>(a.out)[o] = f32_to_bf16(s);
    }
  }
  if (dead) {
    // copies still in flight land before the shared memory goes away
    if (lane == 0 && a.dev_status) atomicOr(a.dev_status, MOE_DEV_PIPELINE_TIMEOUT);
    for (int i = 0; i < RING; ++i)
      if (armed & (1u << i)) gg::mbar_drain(bars + 8 * i, i < stage ? phase ^ 1 : phase);
  }
}

template <int NT, int MT>
moe_status_t launch_few(const Args& a, cudaStream_t s) {
  auto kern = linear_few_kernel<NT, MT>;
  static std::atomic<unsigned long long> attr_done{0};
  if (!once_per_device(attr_done, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, few_smem<NT, MT>()) == cudaSuccess;
      }))
    return MOE_ERR_CUDA;
  // as many row tiles to a round as keep the warps busy, as long as every SM has a round
  constexpr int ROWS = 16 * MT, CHUNK = 2 / MT;
  const int kblocks = a.K / 128, chunks = (kblocks + CHUNK - 1) / CHUNK, all = (a.N + ROWS - 1) / ROWS;
  const int tiles = std::max(1, std::min(FEW_WARPS / chunks, all / num_sms()));
  const int rounds = (all + tiles - 1) / tiles;
  // the weights as K blocks of 128 bytes x rows
  const auto encode = gg::encode_fn();
  if (!encode) return MOE_ERR_CUDA;
  CUtensorMap tm;
  const cuuint64_t dims[3] = {128, (cuuint64_t)a.N, (cuuint64_t)kblocks}, strides[2] = {(cuuint64_t)a.K, 128};
  const cuuint32_t box[3] = {128, ROWS, CHUNK}, unit[3] = {1, 1, 1};
  if (encode(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(a.w), dims, strides, box, unit,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return MOE_ERR_CUDA;
  kern<<<std::min(rounds, num_sms()), FEW_WARPS * 32, few_smem<NT, MT>(), s>>>(tm, a, tiles);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

// Units of 32 weight rows (MT = 2) for up to 16 rows of x, or of 16: those fill a last round of the SMs better, but cost more a byte
// and a round.  Modelled as rounds times (a start, and the rows' bytes); one row, units of 16 / 32: 7168 x 16384 21.1 / 22.3 us,
// 40960 x 4096 35.4 / 29.8, 4096 x 7168 8.7 / 8.0, 2048 x 2048 3.0 / 3.3, 16384 x 7168 22.7 / 22.9, 5000 x 4096 8.5 / 8.3.
bool few_wide(int N, int K) {
  auto us = [&](int rows, double start, double byte) {
    const int units = (N + rows - 1) / rows, rounds = (units + num_sms() - 1) / num_sms();
    return rounds * (start + byte * rows * K);
  };
  return us(32, 0.07, 1.88e-5) <= us(16, 0.18, 2.30e-5);
}

// rows and tiles of rows are counted in 32 bits
inline bool shape_ok(int T, int N, int K) {
  return T >= 0 && T <= (1 << 30) && N > 0 && N <= (1 << 24) && K > 0 && K <= (1 << 22) && K % 128 == 0;
}

struct Plan {
  int variant;     // -1: linear_few_kernel
  Split split;
};

int tiles_of(Variant v, int T, int N) {
  const int cols = v == TC_64 ? 64 : v == TC_256 ? 256 : 128;
  const long long t = (v == SWAP ? 1 : ((long long)T + 127) / 128) * (((long long)N + cols - 1) / cols);
  return (int)std::min<long long>(t, 0x7fffffff);
}

// The cut of a variant: whole tiles in full rounds of the SMs, and the rest, each shared by `parts` CTAs as far as there are
// SMs and K blocks (not the 256-column tiles, which are for many rows).
Split cut(Variant v, int T, int N, int kblocks, int parts) {
  const int tiles = tiles_of(v, T, N), most = num_sms(), rest = tiles % most;
  parts = v == TC_256 || rest == 0 ? 1 : std::min(parts, std::min(most / rest, kblocks));
  if (parts <= 1) return Split{std::min(most, tiles), tiles, 1};
  return Split{tiles > rest ? most : rest * parts, tiles - rest, parts};
}

moe_status_t launch_variant(Variant v, const Args& a, const Split& split, cudaStream_t s) {
  return v == SWAP ? launch_swap(a, split, s) : launch_tc(v, a, split, s);
}

// By rows and weights, then the tile width and the parts of K whose time, modelled from measured calls, is least.
//   Up to 8 rows, and up to 16 where the weights are below 32 MB: the kernel for few rows (1 x 40960 x 4096 30.0 us, with weight
//   rows as M 32.5; 8 x 40960 x 4096 31.0 / 31.3, but 8 x 16384 x 7168 24.5 / 22.2).  9 and 16 rows, weights from memory:
//   2048 x 2048 4.1, 4.3 / 6.5; 2112 x 7168 7.2, 7.5 / 8.9; 4096 x 4096 7.8, 8.1 / 8.7; 4096 x 7168 10.2, 10.5 / 10.2; from here on
//   behind: 8192 x 3584 10.9, 11.9 / 9.9; 8191 x 4096 11.6, 12.7 / 10.7; 8192 x 4096 (32 MB) 11.7, 12.8 / 10.7; 40960 x 4096 37.8, 44.3 /
//   31.4.  So 24 MB would be the better border by up to a tenth; 7168 x 2048 (8.3, 9.2 / 7.6) goes by the shape, not the bytes.
//   Up to 32: weight rows as M (32 x 4096 x 7168 10.7, with 128 x 64 tiles 12.0; 32 x 7168 x 2048 7.0 / 9.6).
//   More, 64 / 128 / 256 columns: 64 x 4096 x 7168 12.5 / 14.9 / 31, 512 x 4096 x 7168 26.8 / 21.0 / 31.7, 3000 x 576 x 7168 24.3 /
//   20.6 / 31.5, 2048 x 2048 x 2048 19.4 / 18.0 / 14.8, 8192 x 4096 x 7168 304 / 239 / 200.
//   Parts 1 / 2 / 4 / 8: 64 x 576 x 7168 14.0 / 10.7 / 8.8 / 8.8, 700 x 576 x 7168 14.7 / 11.8, 32 x 4096 x 7168 14.3 / 11.7 / 10.7; of a
//   last round (128 x 40960 x 4096) 43.4 / 42.5 / 42.0 / 41.9.
Plan plan(int T, int N, int K) {
  if (T <= 8 || (T <= FEW_COLS && (long long)N * K < (32 << 20))) return Plan{-1, {}};
  // microseconds of a K block, of a tile's start and store, of a join and of each of its parts; a block takes at least its
  // weights' share of the memory (41 bytes a nanosecond and SM), read once for all row tiles
  struct Cost {
    Variant v;
    double block, bytes, tile, join, part;
  };
  static constexpr Cost kCosts[] = {{TC_64, 0.205, 8192, 0.6, 2.2, 0.45},
                                    {TC_128, 0.30, 16384, 2.0, 4.0, 0.75},
                                    {TC_256, 0.49, 32768, 2.3, 0.0, 0.0},
                                    {SWAP, 0.21, 16384, 0.6, 1.7, 0.8}};
  const int kblocks = K / 128, most = num_sms();
  const double row_tiles = (T + 127) / 128;
  Plan best{-1, {}};
  double least = 0.0;
  for (const Cost& c : kCosts) {
    if ((c.v == SWAP) != (T <= SWAP_ROWS)) continue;
    const double k = kblocks * std::max(c.block, c.bytes / 41e3 / row_tiles);
    const int tiles = tiles_of(c.v, T, N), rest = tiles % most;
    for (int p = 1; p <= 8; ++p) {
      if (p > 1 && (c.v == TC_256 || rest == 0 || p * rest > most || p > kblocks)) break;
      const double t = tiles / most * (k + c.tile) + (rest ? k / p + c.tile : 0.0) + (p > 1 ? c.join + c.part * p : 0.0);
      if (best.variant < 0 || t < least) {
        least = t;
        best = Plan{c.v, cut(c.v, T, N, kblocks, p)};
      }
    }
  }
  return best;
}

}  // namespace lin8
}  // namespace moe

// Only calls whose K is shared use a workspace.  One size for all of them, so that what was made for T rows serves fewer.
extern "C" size_t moe_linear_e4m3_workspace_bytes(int T, int N, int K) {
  using namespace moe::lin8;
  if (!shape_ok(T, N, K)) return 0;
  return T <= 8 ? 256 : count_bytes() + sum_bytes();
}

static moe_status_t linear_e4m3_impl(const uint8_t* x, const float* x_scales, int T, int K, const uint8_t* w,
                                     const float* w_scales, int N, const float* bias, void* out, int out_f32,
                                     long long out_stride, void* ws, size_t ws_bytes, int32_t* dev_status,
                                     const moe::lin8::Plan* forced, unsigned long long limit_ns, int mute, void* stream) {
  using namespace moe;
  using namespace moe::lin8;
  auto bits = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  if (!shape_ok(T, N, K) || out_stride < N || (out_f32 != 0 && out_f32 != 1)) return MOE_ERR_ARG;
  if (!ws || ws_bytes < moe_linear_e4m3_workspace_bytes(T, N, K)) return MOE_ERR_WORKSPACE;
  if (bits(ws) & 255) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !x_scales || !w || !w_scales || !out) return MOE_ERR_ARG;
  if (((bits(x) | bits(w)) & 15) || ((bits(x_scales) | bits(w_scales) | bits(bias) | bits(dev_status)) & 3) ||
      (bits(out) & (out_f32 ? 3 : 1)))
    return MOE_ERR_ARG;
  const Args a{x, x_scales, w, w_scales, bias, out, out_stride, T, N, K, out_f32, static_cast<int32_t*>(ws),
               reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + count_bytes()), dev_status, limit_ns,
               mute};
  const Plan p = forced ? *forced : plan(T, N, K);
  if (p.variant >= 0) return launch_variant((Variant)p.variant, a, p.split, as_stream(stream));
  const bool wide = few_wide(N, K);
  if (T <= 8) return wide ? launch_few<1, 2>(a, as_stream(stream)) : launch_few<1, 1>(a, as_stream(stream));
  return wide ? launch_few<2, 2>(a, as_stream(stream)) : launch_few<2, 1>(a, as_stream(stream));
}

extern "C" moe_status_t moe_linear_e4m3(const uint8_t* x, const float* x_scales, int T, int K, const uint8_t* w,
                                        const float* w_scales, int N, const float* bias, void* out, int out_f32,
                                        long long out_stride, void* ws, size_t ws_bytes, int32_t* dev_status,
                                        void* stream) {
  return linear_e4m3_impl(x, x_scales, T, K, w, w_scales, N, bias, out, out_f32, out_stride, ws, ws_bytes, dev_status,
                          nullptr, moe::lin8::LIMIT_NS, 0, stream);
}

// Test hook, deliberately absent from the public header: moe_linear_e4m3 by one variant whatever the sizes (-1: the
// kernel for few rows, 0.. a Variant), with the K of the tiles of a last round shared by up to `parts` CTAs (not
// the 256-column tiles'), and with the limit of each wait in nanoseconds.  mute: copies (few rows) or MMAs are
// never issued, so that a test can make the waits for them run out.
extern "C" moe_status_t moe_testing_linear_e4m3(const uint8_t* x, const float* x_scales, int T, int K, const uint8_t* w,
                                                const float* w_scales, int N, const float* bias, void* out, int out_f32,
                                                long long out_stride, void* ws, size_t ws_bytes, int32_t* dev_status,
                                                int variant, int parts, unsigned long long limit_ns, int mute,
                                                void* stream) {
  using namespace moe::lin8;
  if (!shape_ok(T, N, K) || variant < -1 || variant >= VARIANTS || (variant == -1 && T > FEW_COLS) ||
      (variant == SWAP && T > SWAP_ROWS))
    return MOE_ERR_ARG;
  Plan p{variant, {}};
  if (variant >= 0 && T > 0) p.split = cut((Variant)variant, T, N, K / 128, std::max(1, parts));
  return linear_e4m3_impl(x, x_scales, T, K, w, w_scales, N, bias, out, out_f32, out_stride, ws, ws_bytes, dev_status,
                          &p, limit_ns, mute, stream);
}
