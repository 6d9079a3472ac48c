// moe_linear_w4: y = x W^T (+ bias) for a few rows of BF16 x and 4-bit weights with a BF16
// scale (and optionally a zero point) per group of 32, 64 or 128 columns.  The weight
// stream, the work division and the arithmetic are those of few.cuh, with one matrix and the
// rows of x as columns, 32 at a time (each pass over the weights serves 32 rows of x).
//
// Also the one-time preparation of such weights: moe_quantize_weight_w4 and moe_pack_w4.
#include "few.cuh"

namespace moe {
namespace few {

constexpr int LIN_COLS = 32;
constexpr int LIN_WARPS = 16;
constexpr int LIN_WORKERS = LIN_WARPS - 1;   // the last warp schedules
constexpr int LIN_PARTS = 64 * 1024;

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
  Cut cut;
  int tiles;                   // row tiles x blocks of x
  int blocks;                  // blocks of LIN_COLS rows of x
};

// CTA c takes tiles c, c + CTAs, ...; tile = (row tile, block of x rows), blocks inner, so that the
// second block of a row tile finds its weights in L2.
template <int GROUP>
struct LinearSched {
  const LinearArgs& a;
  int q;
  __device__ __forceinline__ bool next(int, int& t, int& n) {
    const long long i = blockIdx.x + (long long)q++ * gridDim.x;
    t = (int)i;
    n = 1;
    return i < a.tiles;
  }
  __device__ __forceinline__ int same(int) const { return 1; }
  __device__ __forceinline__ Cut cut(int) const { return a.cut; }
  __device__ __forceinline__ bool done() const { return true; }
  __device__ __forceinline__ bool idle(int) { return false; }
  __device__ __forceinline__ void give_up(int) {}
  __device__ __forceinline__ void describe(int t, int part, const Cut& c, Unit& u) const {
    const int row = t / a.blocks, s0 = part * c.len, block = w4_block(GROUP, a.zeros);
    u.entry = t - row * a.blocks;
    u.row = row;
    u.s0 = (short)s0;
    u.n = (short)min(c.len, c.nsl - s0);
    u.part = (short)part;
    u.parts = (short)c.parts;
    u.p0 = a.w + ((long long)row * 2 * c.nsl + s0) * block;
    u.p1 = u.p0 + (long long)c.nsl * block;
  }
};
template <int GROUP>
using LinearStream = Stream<F_W4, GROUP, false, LIN_WORKERS>;

template <int GROUP, int NT>
__device__ __forceinline__ void linear_unit(const LinearArgs& a, LinearStream<GROUP>& in, JoinShared& j, float4* parts,
                                            int slots, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const Unit& un = in.unit();
  const int row = un.row, t0 = un.entry * LIN_COLS, part = un.part;
  const uint16_t* x[1][NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) x[0][n] = t0 + n * 8 + g < a.T ? a.x + (t0 + n * 8 + g) * a.x_stride : nullptr;
  Sums<NT> sums;
  in.template run<NT, 1>(sums, a.K, x);
  if (!join<NT>(sums, j, parts, slots, NT * 64, in.cur, in.cur - part, a.cut.parts, lane, a.dev_status)) return;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row * 32 + h * 16 + (i >> 1) * 8 + g;
      if (r >= a.N) continue;
      const float b = a.bias ? __ldg(a.bias + r) : 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int c = t0 + n * 8 + 2 * t + (i & 1);
        if (c >= a.T) continue;
        const float v = a.bias ? sums.v[n][h][i] + b : sums.v[n][h][i];
        const long long o = c * a.out_stride + r;
        if (a.out_f32)
          static_cast<float*>(a.out)[o] = v;
        else
          static_cast<uint16_t*>(a.out)[o] = f32_to_bf16(v);
      }
    }
}

template <int GROUP, int NT>
__global__ void __launch_bounds__(LIN_WARPS * 32, 1) linear_w4_kernel(const LinearArgs a) {
  extern __shared__ __align__(1024) uint8_t rings[];
  __shared__ JoinShared j;
  __shared__ Feed<LIN_WORKERS> feed;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int RING = 2 * Format<F_W4, GROUP>::STAGE;
  constexpr int SLOTS = LIN_PARTS / 1024 / NT < MAX_SLOTS ? LIN_PARTS / 1024 / NT : MAX_SLOTS;
  join_init(j);
  feed_init(feed);
  __syncthreads();
  if (warp == LIN_WORKERS) {
    LinearSched<GROUP> src{a, 0};
    schedule<LIN_WORKERS>(feed, src, lane, a.dev_status);
    return;
  }
  float4* parts = reinterpret_cast<float4*>(rings + LIN_WORKERS * RING);
  LinearStream<GROUP> in{feed, rings + warp * RING};
  in.ring_addr = gg::smem_u32(in.ring);
  in.bars = gg::smem_u32(&feed.full[warp][0]);
  in.lane = lane;
  in.worker = warp;
  in.dev_status = a.dev_status;
  in.block = w4_block(GROUP, a.zeros);
  in.zeros = a.zeros;
  in.start();
  while (in.take()) linear_unit<GROUP, NT>(a, in, j, parts, SLOTS, lane);
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
        if (zp) zv |= (uint32_t)(zp[o] & 15) << (8 * h);
      }
    }
    osc[gg * ng + gi] = sv;
    if (zp) ozp[gg * ng + gi] = (uint16_t)zv;
  }
}

template <int GROUP, int NT>
moe_status_t launch_linear(const LinearArgs& a, cudaStream_t stream) {
  constexpr int smem = LIN_WORKERS * 2 * Format<F_W4, GROUP>::STAGE + LIN_PARTS;
  static std::atomic<unsigned long long> done{0};
  if (!once_per_device(done, [] {
        return cudaFuncSetAttribute(linear_w4_kernel<GROUP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) ==
               cudaSuccess;
      }))
    return MOE_ERR_CUDA;
  const int ctas = a.tiles < num_sms() ? a.tiles : num_sms();
  linear_w4_kernel<GROUP, NT><<<ctas, LIN_WARPS * 32, smem, stream>>>(a);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
template <int GROUP>
moe_status_t launch_linear(const LinearArgs& a, cudaStream_t stream) {
  const int cols = a.T < LIN_COLS ? a.T : LIN_COLS;
  return cols <= 8    ? launch_linear<GROUP, 1>(a, stream)
         : cols <= 16 ? launch_linear<GROUP, 2>(a, stream)
                      : launch_linear<GROUP, 4>(a, stream);
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

extern "C" size_t moe_linear_w4_workspace_bytes(int T, int N, int K) {
  using namespace moe::few;
  if (T < 0 || !w4_shape_ok(0, N, K, 32)) return 0;
  return 256;
}

extern "C" moe_status_t moe_linear_w4(const uint16_t* x, int T, int K, long long x_stride, const uint8_t* packed, int N,
                                      int group, int zeros, const float* bias, void* out, int out_f32,
                                      long long out_stride, void* ws, size_t ws_bytes, int32_t* dev_status,
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
  a.blocks = (int)ceil_div(T, LIN_COLS);
  const long long tiles = ceil_div(N, 32) * a.blocks;
  if (tiles > 0x7fffffffll) return MOE_ERR_ARG;
  a.tiles = (int)tiles;
  a.cut.set(w4_slices(K), LIN_WORKERS, a.tiles <= num_sms());
  a.dev_status = dev_status;
  cudaStream_t st = as_stream(stream);
  return group == 32 ? launch_linear<32>(a, st) : group == 64 ? launch_linear<64>(a, st) : launch_linear<128>(a, st);
}
