// moe_linear_w4: y = x W^T (+ bias) for a few rows of BF16 x and 4-bit weights with a BF16
// scale (and optionally a zero point) per group of 32, 64 or 128 columns.  The weight
// stream and the arithmetic are those of few.cuh, with one matrix and the rows of x as columns,
// 32 at a time (each pass over the weights serves 32 rows of x).
//
// A CTA keeps its rows of x in shared memory as FP16, scaled by a power of two per row that brings
// the largest value to 2^14 (exact for values above 2^-28 of it): FP16 codes unpack in fewer
// instructions than BF16 ones, and 24 rows read from L2 beside every item are three times the
// weights' bytes.  Where the rows are too long for that, K is shared between CTAs, whose sums the
// last of them adds up in order.
//
// Bound: reading W once; in fact the latency of an item's unpacking (few.cuh) and, with 24 columns, the tensor
// instructions (pipe 29 % busy).  Measured (group 128 unless said otherwise): 24 x 40960 x 4096, float32 out
// 42.6 us (2.1 TB/s); 1 x 4096 x 7168 7.9 us; 7 x 7168 x 2048, group 64, zero points, bias 7.6 us; 1 x 512 x 256, group 32
// 4.4 us (launch and latency).
//
// Also the one-time preparation of such weights: moe_quantize_weight_w4 and moe_pack_w4.
#include <algorithm>

#include "few.cuh"

namespace moe {
namespace few {

constexpr int LIN_COLS = 32;
// Warps of a CTA: 16 as far as 128 registers a thread do; 12 otherwise (24 columns: 42.0 us with 12, 45 to
// 47 with 13 to 15, whose rings leave less room for x).
template <int NT>
__host__ __device__ constexpr int lin_warps() { return NT == 1 ? 16 : 12; }
constexpr int LIN_SMEM = 225 * 1024;

struct LinearArgs {
  const uint16_t* x;
  long long x_stride, out_stride;
  int T, N, K;
  const uint8_t* w;
  int zeros;
  const float* bias;
  void* out;
  int out_f32;
  int32_t* dev_status;
  unsigned long long limit_ns; // of each wait
  int nsl;                     // items per tile row
  int splits, split_len;       // shares of K, items per share
  Cut cut;                     // of a share
  int rows, blocks;            // row tiles, blocks of LIN_COLS rows of x
  int pitch;                   // elements from one row of x to the next in shared memory
  int slots;                   // of the joins
  int32_t* count;              // [rows x blocks] shares done, zero between launches
  float* part;                 // [rows x blocks][splits][NT * 256]
};

// CTA c has share c % splits of K and, of the tiles (row tile, block of x), c / splits and every
// (CTAs / splits)-th on; its warps take the units of that sequence in turn.
template <int GROUP, int NT>
struct LinearSource {
  const LinearArgs& a;
  int share, items, parts, first, step, total;   // items of a tile here, its units; units in all
  int next;
  __device__ __forceinline__ int claim(int) {
    const int u = next;
    next += lin_warps<NT>();
    return u;
  }
  __device__ __forceinline__ int state(int u, int) const { return u < total ? 1 : 2; }
  __device__ __forceinline__ void at(int, int) const {}
  __device__ __forceinline__ Unit unit(int u) const {
    const int len = a.cut.len;
    const int q = u / parts, tile = first + q * step, row = tile / a.blocks;
    const int block = w4_block(GROUP, a.zeros);
    Unit k;
    k.part = (short)(u - q * parts);
    k.parts = (short)parts;
    const int s0 = k.part * len;                         // within the share
    k.s0 = (short)s0;
    k.n = (short)min(len, items - s0);
    k.entry = tile - row * a.blocks;
    k.row = row;
    k.p0 = a.w + ((long long)row * 2 * a.nsl + share * a.split_len + s0) * block;
    k.p1 = k.p0 + (long long)a.nsl * block;
    return k;
  }
};
template <int GROUP, int NT>
using LinearStream = Stream<F_W4, GROUP, true, true, LinearSource<GROUP, NT>>;

// The CTA's rows of x, its share of K, as FP16, by all warps: several to a row, or several rows to a
// warp, each lane with BATCH loads in flight (8 with many rows: 42.7 us against 52.5 for 24 x 40960 x 4096
// with one row after the other; 2 with few: less code, and 1 x 512 x 256 is fetching code).  Zeros up to a whole item.
template <int WARPS, int BATCH>
__device__ __forceinline__ void stage_rows(const LinearArgs& a, uint16_t* xs, uint32_t* most, float* unit, int t0,
                                           int k0, int k, int warp, int lane) {
  const int n = min(LIN_COLS, a.T - t0), chunks = (a.pitch - 32) / 8, real = k / 8;
  const int lg = WARPS == 16 ? max(0, 4 - (32 - __clz(n - 1))) : 0;
  const int share = 1 << lg, at_once = WARPS >> lg;      // warps to a row (a power of two), rows at a time
  const int row = warp >> lg, first = (warp & (share - 1)) * 32 + lane, step = share * 32;
  if (share > 1) {
    if (warp == 0) most[lane] = 0;
    __syncthreads();
  }
  for (int r0 = 0; r0 < n; r0 += at_once) {       // once if share > 1
    const int r = r0 + row;
    const bool mine = r < n;
    const uint4* src = reinterpret_cast<const uint4*>(a.x + (t0 + (mine ? r : 0)) * a.x_stride + k0);
    uint4* dst = reinterpret_cast<uint4*>(xs + (mine ? r : 0) * a.pitch);
    uint4 v[BATCH];
    auto load = [&](int c0) {
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int c = c0 + first + i * step;
        v[i] = c < real ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
      }
    };
    uint32_t m = 0;
    for (int c0 = (chunks - 1) & -(BATCH * step); c0 >= 0; c0 -= BATCH * step) {   // the first chunks last: they stay
      load(c0);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) m = max(m, bf16_max(v[i]));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (share > 1) {
      if (lane == 0 && mine) atomicMax(&most[r], m);
      __syncthreads();
      if (mine) m = most[r];
    }
    const float sc = to_half_scale(m);
    if (first == 0 && mine) unit[r] = 1.0f / sc;   // a power of two
    for (int c0 = 0; c0 < chunks; c0 += BATCH * step) {
      if (c0) load(c0);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int c = c0 + first + i * step;
        if (c < chunks && mine) dst[c] = bf16_to_half8(v[i], sc);
      }
    }
  }
  __syncthreads();
}

template <int GROUP, int NT>
__device__ __forceinline__ void linear_unit(const LinearArgs& a, LinearStream<GROUP, NT>& in, JoinShared& j, float4* parts,
                                            uint32_t xs, const float* unit, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const Unit un = in.src.unit(in.cur);
  const int t0 = un.entry * LIN_COLS;
  int off[1][NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) off[0][n] = (t0 + n * 8 + g < a.T ? n * 8 + g : 0) * a.pitch;
  Sums<NT> sums;
  if (!in.template run<NT, 1>(sums, Acts<true>{nullptr, xs}, off)) return;
  if (!join<NT>(sums, j, parts, a.slots, NT * 64, in.cur, in.cur - un.part, un.parts, lane, in.patience)) return;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float f = unit[n * 8 + 2 * t + i];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sums.v[n][h][i] *= f;
        sums.v[n][h][i + 2] *= f;
      }
    }
  if (a.splits > 1) {
    const int tile = un.row * a.blocks + un.entry;
    float4* p = reinterpret_cast<float4*>(a.part) + (size_t)tile * a.splits * (NT * 64);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        __stcg(&p[in.src.share * (NT * 64) + (n * 2 + h) * 32 + lane],
               make_float4(sums.v[n][h][0], sums.v[n][h][1], sums.v[n][h][2], sums.v[n][h][3]));
    __syncwarp();
    int old = 0;
    if (lane == 0) old = atom_add_release(&a.count[tile], 1);
    if (__shfl_sync(0xffffffffu, old, 0) != a.splits - 1) return;
    __threadfence();
    if (lane == 0) a.count[tile] = 0;
    sums.clear();
#pragma unroll 1
    for (int s = 0; s < a.splits; ++s)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 v = __ldcg(&p[s * (NT * 64) + (n * 2 + h) * 32 + lane]);
          sums.v[n][h][0] += v.x;
          sums.v[n][h][1] += v.y;
          sums.v[n][h][2] += v.z;
          sums.v[n][h][3] += v.w;
        }
  }
  const int r0 = un.row * 32 + g;               // rows r0 + 8 q, q = 2 h + i / 2
  if (a.bias) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float b = r0 + 8 * q < a.N ? __ldg(a.bias + r0 + 8 * q) : 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) sums.v[n][q >> 1][(q & 1) * 2 + j] += b;
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = t0 + n * 8 + 2 * t + j;
      if (c >= a.T) continue;
      const long long o = c * a.out_stride + r0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v = sums.v[n][q >> 1][(q & 1) * 2 + j];
        if (r0 + 8 * q >= a.N) break;
        if (a.out_f32)
          static_cast<float*>(a.out)[o + 8 * q] = v;
        else
          static_cast<uint16_t*>(a.out)[o + 8 * q] = f32_to_bf16(v);
      }
    }
}

template <int GROUP, int NT>
__global__ void __launch_bounds__(lin_warps<NT>() * 32, 1) linear_w4_kernel(const __grid_constant__ LinearArgs a) {
  extern __shared__ __align__(1024) uint8_t rings[];
  __shared__ JoinShared j;
  __shared__ int gave_up;                          // a wait of this CTA ran out
  constexpr int LIN_WARPS = lin_warps<NT>();
  __shared__ uint32_t most[LIN_COLS];              // largest finite |x| of a row, as bits
  __shared__ float unit[LIN_COLS];                 // what 1 in the FP16 row stands for
  __shared__ __align__(8) unsigned long long full[LIN_WARPS][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int RING = 2 * Format<F_W4, GROUP>::STAGE;
  float4* parts = reinterpret_cast<float4*>(rings + LIN_WARPS * RING);
  uint16_t* xs = reinterpret_cast<uint16_t*>(rings + LIN_WARPS * RING + a.slots * NT * 1024);
  const int share = blockIdx.x % a.splits, first = blockIdx.x / a.splits, step = gridDim.x / a.splits;
  const int tiles = a.rows * a.blocks;
  const int mine = first < tiles ? (tiles - first + step - 1) / step : 0;
  const int items = min(a.split_len, a.nsl - share * a.split_len), n_parts = (items + a.cut.len - 1) / a.cut.len;
  LinearStream<GROUP, NT> in{{a, share, items, n_parts, first, step, mine * n_parts, warp}, rings + warp * RING};
  in.ring_addr = gg::smem_u32(in.ring);
  in.bars = gg::smem_u32(&full[warp][0]);
  in.lane = lane;
  in.patience = {&gave_up, a.dev_status, a.limit_ns};
  if (threadIdx.x == 0) gave_up = 0;
  in.block = w4_block(GROUP, a.zeros);
  in.zeros = a.zeros;
  if (lane == 0) {
    gg::mbar_init(in.bars, 1);
    gg::mbar_init(in.bars + 8, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  in.start();                  // the weights are on their way while x is converted
  join_init(j);
  const int k0 = share * a.split_len * 256, k = min(a.K - k0, a.split_len * 256);
  // one block of x at a time stays in shared memory: with more blocks every CTA has one (launch_linear)
  stage_rows<LIN_WARPS, NT == 1 ? 2 : 8>(a, xs, most, unit, (first % a.blocks) * LIN_COLS, k0, k, warp, lane);
  while (in.take()) linear_unit<GROUP, NT>(a, in, j, parts, gg::smem_u32(xs), unit, lane);
  in.finish();
}

// ------------------------------------------------------------------- weight preparation
// One thread per group of one row: scale (and zero point), then the codes, two per byte.
//   symmetric   s = bf16(amax / 7), code = clamp(rn(w / s), -8, 7) + 8
//   zero points lo = min(0, min w), hi = max(0, max w), s = bf16((hi - lo) / 15),
//               z = clamp(rn(-lo / s), 0, 15), code = clamp(rn(w / s) + z, 0, 15)
// s = 1 where that is not positive; IEEE float32 divisions, halves to even.
__global__ void __launch_bounds__(256) quant_w4_kernel(const uint16_t* __restrict__ w, long long groups, int rows,
                                                       int cols, int group, uint8_t* __restrict__ q,
                                                       uint16_t* __restrict__ scales, uint8_t* __restrict__ zeros) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= groups) return;
  const int per_row = cols / group;
  const long long mr = i / per_row;            // matrix * rows + row
  const int gi = (int)(i - mr * per_row);
  const long long m = mr / rows;
  const int r = (int)(mr - m * rows);
  const uint16_t* src = w + mr * cols + (long long)gi * group;
  float lo = 0.0f, hi = 0.0f;
  for (int c = 0; c < group; ++c) {
    const float v = bf16_to_f32(src[c]);
    lo = fminf(lo, v);
    hi = fmaxf(hi, v);
  }
  const float raw = zeros ? __fdiv_rn(__fsub_rn(hi, lo), 15.0f) : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
  uint16_t sb = f32_to_bf16(raw);
  if (!(bf16_to_f32(sb) > 0.0f)) sb = 0x3f80;
  const float s = bf16_to_f32(sb);
  const float z = zeros ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f) : 8.0f;
  uint8_t* dst = q + (mr * cols + (long long)gi * group) / 2;
  for (int c = 0; c < group; c += 2) {
    uint32_t b = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float v = rintf(__fdiv_rn(bf16_to_f32(src[c + j]), s)) + z;
      b |= (uint32_t)fminf(fmaxf(v, 0.0f), 15.0f) << (4 * j);
    }
    dst[c / 2] = (uint8_t)b;
  }
  const long long o = (m * per_row + gi) * rows + r;
  scales[o] = sb;
  if (zeros) zeros[o] = (uint8_t)z;
}

// One warp per block (16 rows x 256 columns).  Codes: for row g (then g + 8) and J = 0, 1, lane (g, t)'s
// 16 bytes: word i holds columns (4 J + i) * 32 + t * 8 .. + 8, even ones in nibbles 0-3, odd ones in
// nibbles 4-7.  Then the scales, [g][group][row g, row g + 8], and the zero points likewise.  Rows
// past N and columns past K are code 0 with scale 0.
__global__ void __launch_bounds__(256) pack_w4_kernel(const uint8_t* __restrict__ q, const uint16_t* __restrict__ sc,
                                                      const uint8_t* __restrict__ zp, long long blocks, int N, int K,
                                                      int group, uint8_t* __restrict__ out) {
  const long long blk = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (blk >= blocks) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int nsl = w4_slices(K), nrb = (int)ceil_div(N, 32) * 2;
  const int s = (int)(blk % nsl);
  const long long mrb = blk / nsl;
  const int rb = (int)(mrb % nrb);
  const long long m = mrb / nrb;
  uint8_t* dst = out + blk * w4_block(group, zp != nullptr);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = rb * 16 + h * 8 + g;
#pragma unroll
    for (int J = 0; J < 2; ++J) {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = s * 256 + (4 * J + i) * 32 + t * 8;
        uint32_t v = 0;
        if (row < N && k < K) {
          const uint32_t u = *reinterpret_cast<const uint32_t*>(q + ((m * N + row) * K + k) / 2);
#pragma unroll
          for (int b = 0; b < 4; ++b)
            v |= ((u >> (8 * b)) & 15u) << (4 * b) | ((u >> (8 * b + 4)) & 15u) << (4 * b + 16);
        }
        o[i] = v;
      }
      *reinterpret_cast<uint4*>(dst + h * 1024 + J * 512 + lane * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  const int ng = 256 / group, kg = K / group;
  uint32_t* osc = reinterpret_cast<uint32_t*>(dst + 2048);
  uint16_t* ozp = reinterpret_cast<uint16_t*>(dst + 2048 + 8 * ng * 4);
  for (int i = lane; i < 8 * ng; i += 32) {
    const int gg = i / ng, gi = i % ng, kgi = s * ng + gi;
    uint32_t sv = 0, zv = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = rb * 16 + h * 8 + gg;
      if (row < N && kgi < kg) {
        const long long o = (m * kg + kgi) * N + row;
        sv |= (uint32_t)sc[o] << (16 * h);
        if (zp) zv |= (uint32_t)zp[o] << (8 * h);
      }
    }
    osc[gg * ng + gi] = sv;
    if (zp) ozp[gg * ng + gi] = (uint16_t)zv;
  }
}

// How a product is laid out on the GPU: shares of K so that a block of x fits in shared memory
// beside the rings and the joins' slots; a whole number of blocks of x per step of tiles, so that
// a CTA always has the same block.
struct LinearPlan {
  int nt, slots, splits, split_len, pitch, ctas, smem;
  Cut cut;
  long long tiles, cost;
  size_t sum_bytes() const { return splits > 1 ? (size_t)tiles * splits * nt * 1024 : 0; }
};
inline int linear_cols(int T) { return T < LIN_COLS ? T : LIN_COLS; }
// With room for this many slots of the joins, which are as many as a tile may have units.
inline LinearPlan plan_linear(int T, int N, int K, int group, int sms, int slots) {
  LinearPlan p;
  const int cols = linear_cols(T);
  p.nt = (cols + 7) / 8;
  p.slots = slots;
  const int warps = p.nt == 1 ? lin_warps<1>() : lin_warps<4>();
  const int stage = 2 * (2048 + 8 * (256 / group) * 6);
  const int fixed = warps * 2 * stage + slots * p.nt * 1024;
  const int room = (LIN_SMEM - fixed) / 2 / cols - 32;      // elements of a row
  const int nsl = w4_slices(K), fit = room / 256 < 1 ? 1 : room / 256;
  p.splits = (nsl + fit - 1) / fit;
  p.split_len = (nsl + p.splits - 1) / p.splits;
  p.splits = (nsl + p.split_len - 1) / p.split_len;
  const int blocks = (T + LIN_COLS - 1) / LIN_COLS;
  p.tiles = ceil_div(N, 32) * blocks;
  p.pitch = p.split_len * 256 + 32;          // rows 64 bytes past a multiple of 128: two rows' chunks in different banks
  p.smem = fixed + cols * p.pitch * 2;
  const int unit = p.splits * blocks;
  p.ctas = sms / unit * unit;
  if (p.ctas == 0) p.ctas = unit;
  const long long most = p.tiles * p.splits;
  if (most < p.ctas) p.ctas = (int)most;
  // Warps take units in turn, so a CTA works in rounds of a unit per warp; a unit costs its items and
  // UNIT_COST.  Against units of four items, eight with many tiles: 12 x 16384 x 4096 18.2
  // and 22.9 us, 7 x 7168 x 2048 7.5 and 8.1, others the same; with a cost of two instead of four 24 x 40960 x
  // 4096 takes 44.5 instead of 42.3.
  const long long mine = (p.tiles + p.ctas / p.splits - 1) / (p.ctas / p.splits);      // tiles of a CTA
  for (int parts = 1; parts <= p.slots && parts <= p.split_len; ++parts) {
    const int len = (p.split_len + parts - 1) / parts;
    const long long cost = (mine * parts + warps - 1) / warps * (len + UNIT_COST);
    if (parts > 1 && cost >= p.cost) continue;
    p.cost = cost;
    p.cut.set(p.split_len, parts);
  }
  return p;
}
// 32 KB of slots, and one for each warp; with three or four column groups three for each four warps instead where the
// shares of K that this saves make the rounds cheaper: 32 x 40960 x 4096, groups of 32, 58.7 us instead of 75.9 (four
// shares, six); 32 x 7168 x 7168 25.0 instead of 33.2.  Where they do not, more slots are better: 25 x 2048 x 4096,
// groups of 128, 12.3 us with 12, 14.3 with 9 and a share less.
inline int linear_slots(int T) { return std::max(lin_warps<4>(), 32 / ((linear_cols(T) + 7) / 8)); }
inline LinearPlan plan_linear(int T, int N, int K, int group, int sms) {
  const LinearPlan p = plan_linear(T, N, K, group, sms, linear_slots(T));
  if (p.nt < 3 || p.splits == 1) return p;
  const LinearPlan q = plan_linear(T, N, K, group, sms, lin_warps<4>() * 3 / 4);
  return q.cost < p.cost ? q : p;
}

template <int GROUP, int NT>
moe_status_t launch_linear(const LinearArgs& a, const LinearPlan& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  if (!once_per_device(done, [] {
        return cudaFuncSetAttribute(linear_w4_kernel<GROUP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    LIN_SMEM) == cudaSuccess;
      }))
    return MOE_ERR_CUDA;
  linear_w4_kernel<GROUP, NT><<<p.ctas, lin_warps<NT>() * 32, p.smem, stream>>>(a);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
template <int GROUP>
moe_status_t launch_linear(const LinearArgs& a, const LinearPlan& p, cudaStream_t stream) {
  return p.nt == 1 ? launch_linear<GROUP, 1>(a, p, stream)
         : p.nt == 2 ? launch_linear<GROUP, 2>(a, p, stream)
         : p.nt == 3 ? launch_linear<GROUP, 3>(a, p, stream)
                     : launch_linear<GROUP, 4>(a, p, stream);
}

inline bool w4_shape_ok(int mats, int N, int K, int group) {
  return mats >= 0 && N > 0 && K > 0 && (group == 32 || group == 64 || group == 128) && K % 128 == 0 &&
         N <= (1 << 24) && K <= (1 << 22);
}
inline uintptr_t bits_of(const void* p) { return reinterpret_cast<uintptr_t>(p); }

}  // namespace few
}  // namespace moe

extern "C" moe_status_t moe_quantize_weight_w4(const uint16_t* w, int mats, int rows, int cols, int group, uint8_t* q,
                                               uint16_t* scales, uint8_t* zeros, void* stream) {
  using namespace moe;
  using namespace moe::few;
  if (!w4_shape_ok(mats, rows, cols, group)) return MOE_ERR_ARG;
  if (mats == 0) return MOE_OK;
  if (!w || !q || !scales) return MOE_ERR_ARG;
  const long long groups = (long long)mats * rows * (cols / group);
  if (ceil_div(groups, 256) > 0x7fffffffll) return MOE_ERR_ARG;
  quant_w4_kernel<<<(unsigned)ceil_div(groups, 256), 256, 0, as_stream(stream)>>>(w, groups, rows, cols, group, q,
                                                                                  scales, zeros);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" size_t moe_w4_packed_bytes(int N, int K, int group, int zeros) {
  using namespace moe::few;
  if (!w4_shape_ok(0, N, K, group) || (zeros != 0 && zeros != 1)) return 0;
  // whole 32-row tiles, so that the last tile's second half is there to be read
  return (size_t)(ceil_div(N, 32) * 2 * w4_slices(K) * w4_block(group, zeros));
}

extern "C" moe_status_t moe_pack_w4(const uint8_t* q, const uint16_t* scales, const uint8_t* zeros, int mats, int N,
                                    int K, int group, uint8_t* packed, void* stream) {
  using namespace moe;
  using namespace moe::few;
  if (!w4_shape_ok(mats, N, K, group)) return MOE_ERR_ARG;
  if (mats == 0) return MOE_OK;
  if (!q || !scales || !packed) return MOE_ERR_ARG;
  if ((bits_of(q) & 3) || (bits_of(scales) & 1) || (bits_of(packed) & 15)) return MOE_ERR_ARG;
  const size_t in = (size_t)mats * N * K / 2, outb = (size_t)mats * moe_w4_packed_bytes(N, K, group, zeros != nullptr);
  if (bits_of(q) < bits_of(packed) + outb && bits_of(packed) < bits_of(q) + in) return MOE_ERR_ARG;   // overlap
  if (mats > 1 && N % 32) return MOE_ERR_ARG;     // a stack of matrices is addressed by whole tiles
  const long long blocks = (long long)(outb / w4_block(group, zeros != nullptr));
  if (ceil_div(blocks, 8) > 0x7fffffffll) return MOE_ERR_ARG;
  pack_w4_kernel<<<(unsigned)ceil_div(blocks, 8), 256, 0, as_stream(stream)>>>(q, scales, zeros, blocks, N, K, group,
                                                                               packed);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

// The counters of the tiles at the start, the shares' sums at the end of what the caller has: a workspace
// made for T serves fewer rows too, whose sums must not lie where more rows have counters.  So the sums get
// what any T up to this one needs, with the group whose items leave least room for x and the most slots.
extern "C" size_t moe_linear_w4_workspace_bytes(int T, int N, int K) {
  using namespace moe;
  using namespace moe::few;
  if (T < 0 || !w4_shape_ok(0, N, K, 32)) return 0;
  if (T == 0) return 256;
  auto plan = [&](int t) { return plan_linear(t, N, K, 32, num_sms(), linear_slots(t)); };
  size_t sums = 0;
  for (int t = 8; t < T && t < LIN_COLS; t += 8) sums = std::max(sums, plan(t).sum_bytes());
  const LinearPlan p = plan(T);
  return align256(4 * (size_t)p.tiles) + std::max(sums, p.sum_bytes());
}

static moe_status_t linear_impl(const uint16_t* x, int T, int K, long long x_stride, const uint8_t* packed, int N,
                                int group, int zeros, const float* bias, void* out, int out_f32, long long out_stride,
                                void* ws, size_t ws_bytes, int32_t* dev_status, unsigned long long limit_ns,
                                void* stream) {
  using namespace moe;
  using namespace moe::few;
  if (T < 0 || !w4_shape_ok(0, N, K, group) || (zeros != 0 && zeros != 1) || x_stride < K || x_stride % 8 ||
      out_stride < N || (out_f32 != 0 && out_f32 != 1))
    return MOE_ERR_ARG;
  if (!ws || ws_bytes < moe_linear_w4_workspace_bytes(T, N, K)) return MOE_ERR_WORKSPACE;
  if (bits_of(ws) & 255) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !packed || !out) return MOE_ERR_ARG;
  if ((bits_of(x) & 15) || (bits_of(packed) & 15) || (bits_of(out) & (out_f32 ? 3 : 1)) || (bits_of(bias) & 3))
    return MOE_ERR_ARG;
  LinearArgs a;
  a.x = x;
  a.x_stride = x_stride;
  a.out_stride = out_stride;
  a.T = T;
  a.N = N;
  a.K = K;
  a.w = packed;
  a.zeros = zeros;
  a.bias = bias;
  a.out = out;
  a.out_f32 = out_f32;
  const LinearPlan p = plan_linear(T, N, K, group, num_sms());
  if (p.tiles > 0x3fffffff / p.cut.parts) return MOE_ERR_ARG;
  a.nsl = w4_slices(K);
  a.splits = p.splits;
  a.split_len = p.split_len;
  a.cut = p.cut;
  a.rows = (int)ceil_div(N, 32);
  a.blocks = (int)ceil_div(T, LIN_COLS);
  a.pitch = p.pitch;
  a.slots = p.slots;
  a.count = static_cast<int32_t*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + (ws_bytes - p.sum_bytes()) / 256 * 256);
  a.dev_status = dev_status;
  a.limit_ns = limit_ns;
  cudaStream_t st = as_stream(stream);
  return group == 32   ? launch_linear<32>(a, p, st)
         : group == 64 ? launch_linear<64>(a, p, st)
                       : launch_linear<128>(a, p, st);
}

extern "C" moe_status_t moe_linear_w4(const uint16_t* x, int T, int K, long long x_stride, const uint8_t* packed, int N,
                                      int group, int zeros, const float* bias, void* out, int out_f32,
                                      long long out_stride, void* ws, size_t ws_bytes, int32_t* dev_status,
                                      void* stream) {
  return linear_impl(x, T, K, x_stride, packed, N, group, zeros, bias, out, out_f32, out_stride, ws, ws_bytes, dev_status,
                     moe::few::TIMEOUT_NS, stream);
}

// Test hook, deliberately absent from the public header: moe_linear_w4 with the limit of each wait in
// nanoseconds instead of the built-in 2 s, so that a test can make a wait run out.
extern "C" moe_status_t moe_testing_linear_w4_wait_limit(const uint16_t* x, int T, int K, long long x_stride,
                                                         const uint8_t* packed, int N, int group, int zeros,
                                                         const float* bias, void* out, int out_f32,
                                                         long long out_stride, void* ws, size_t ws_bytes,
                                                         int32_t* dev_status, unsigned long long limit_ns,
                                                         void* stream) {
  return linear_impl(x, T, K, x_stride, packed, N, group, zeros, bias, out, out_f32, out_stride, ws, ws_bytes, dev_status,
                     limit_ns, stream);
}
