// Root-mean-square norm of a residual stream ahead of a layer, with the residual's addition and
// E4M3 rows out.  For a row of H columns, all in float32:
//     h = x (+ residual)                      residual_out = h, rounded once to its type
//     r = 1 / sqrt(sum(h^2) / H + eps)
//     y = (h * r) * weight                    out = bf16(y)
//     per 128 columns: s = amax|y| / 448 (1 if that is not positive), q = e4m3(y / s)
// y is never rounded to BF16 on its way to the codes, and h is normalised as it was summed, not as
// the residual keeps it: each output has one rounding.
//
// Bound by memory: x and the residual are read once and held in registers between the sum and the
// outputs.  A row belongs to a block; a thread holds VPT vectors of 8 columns, vector j of thread t being
// columns 8 (t + j * threads).. so that 16 lanes next to each other hold one 128-column block.
//   Rows up to the SMs: one vector a thread, the most loads in flight (1 x 7168: 3.0 us, launch and latency).
//   More: two vectors and 1024 threads an SM, the next row loaded ahead: 12000 x 7168, BF16 residual, all outputs: 121 us,
//   0.96 of the measured copy bandwidth (without loading ahead 141, four vectors 129, 1536 threads 147); 16384 x 2048 48.6 us.
//   Rows longer than 8192 columns, whose registers leave no room for the next: four or eight vectors.  Four: 4096 x 12288 with a
//   BF16 residual and all outputs 85 us, 4096 x 16384 103 (0.80 and 0.88 of the copy bandwidth).  Eight, beyond 32768 columns,
//   are more than 64 registers hold: 120, 168 and 240 bytes of a thread (no, BF16, float32 residual) stand in local memory;
//   1024 x 65536 147 us (0.62), 2048 x 32768, still four, 114 (0.80).
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

struct NormArgs {
  const uint16_t* x;
  long long x_stride;
  int T, H;
  const void* weight;
  int weight_f32;
  float eps;
  const void* residual;
  int residual_f32;
  void* residual_out;
  uint16_t* out;
  uint8_t* q;
  float* q_scales;
  const int32_t* num_tokens;
};

__device__ __forceinline__ void unpack8(const uint4 u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (uint32_t)f32_to_bf16(f[2 * i]) | ((uint32_t)f32_to_bf16(f[2 * i + 1]) << 16);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Codes of 8 values with scale s: e4m3(v / s) with the quotients correctly rounded.  The division is Markstein's ("Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990): with inv the correctly rounded reciprocal,
// t = v inv is within an ulp, and t - (t s - v) inv rounds to the quotient.  It asks that nothing on the way under- or
// overflows: outside [2^-80, 2^80] s is divided by as usual (inside, a v so small that the remainder underflows is below
// half of the smallest code either way).  A quotient of zero keeps the sign of v: of -0 the remainder t s - v is
// +0, as a sum of zeros of both signs is, and t less +0 stays -0; the other way round, t + (v - t s) inv, it would be +0.
// Every block by the usual division instead: 12000 x 7168 133 us, this 121.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float s) {
  uint32_t c[2] = {0, 0};
  if (s > 8e-25f && s < 1e24f) {
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = __fmul_rn(v[i], inv);
      c[i >> 2] |= (uint32_t)f32_to_e4m3(fmaf(-fmaf(t, s, -v[i]), inv, t)) << (8 * (i & 3));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i >> 2] |= (uint32_t)f32_to_e4m3(__fdiv_rn(v[i], s)) << (8 * (i & 3));
  }
  return make_uint2(c[0], c[1]);
}

// What a thread holds of a row as it was loaded.  RES: 0 no residual, 1 BF16, 2 float32.
template <int VPT, int RES>
struct Raw {
  uint4 x[VPT], r[RES == 2 ? 2 * VPT : VPT];
  __device__ __forceinline__ void load(const NormArgs& a, int row, int nvec) {
    const uint4* xr = reinterpret_cast<const uint4*>(a.x + (size_t)row * a.x_stride);
    const uint4* rr = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.residual) + (size_t)row * a.H * (2 * RES));
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      const bool ok = v < nvec;
      x[j] = ok ? xr[v] : make_uint4(0, 0, 0, 0);
      if (RES == 1) r[j] = ok ? rr[v] : make_uint4(0, 0, 0, 0);
      if (RES == 2) {
        r[2 * j] = ok ? rr[2 * v] : make_uint4(0, 0, 0, 0);
        r[2 * j + 1] = ok ? rr[2 * v + 1] : make_uint4(0, 0, 0, 0);
      }
    }
  }
  __device__ __forceinline__ void sum(float (&h)[VPT][8]) const {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      unpack8(x[j], h[j]);
      if (RES == 1) {
        float f[8];
        unpack8(r[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = __fadd_rn(h[j][i], f[i]);
      }
      if (RES == 2) {
        const uint32_t f[8] = {r[2 * j].x, r[2 * j].y, r[2 * j].z, r[2 * j].w,
                               r[2 * j + 1].x, r[2 * j + 1].y, r[2 * j + 1].z, r[2 * j + 1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = __fadd_rn(h[j][i], __uint_as_float(f[i]));
      }
    }
  }
};

// A block's rows one after the other.  AHEAD: the next row is loaded while this one is summed, scaled and stored (where a
// block has several rows).
template <int VPT, int RES, bool AHEAD>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormArgs a) {
  __shared__ float part[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int nvec = a.H / 8;
  const int rows = a.num_tokens ? min(max(*a.num_tokens, 0), a.T) : a.T;
  int side = 0;
  Raw<VPT, RES> raw;
  if (AHEAD && (int)blockIdx.x < rows) raw.load(a, blockIdx.x, nvec);
  for (int row = blockIdx.x; row < rows; row += gridDim.x, side ^= 1) {
    float h[VPT][8];
    float ss = 0.0f;
    if (!AHEAD) raw.load(a, row, nvec);
    raw.sum(h);
    if (AHEAD && row + (int)gridDim.x < rows) raw.load(a, row + gridDim.x, nvec);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[j][i], h[j][i], ss);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if (lane == 0) part[side][warp] = ss;
    __syncthreads();   // the other side was read before the barrier of the row before
    ss = lane < nw ? part[side][lane] : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)a.H), a.eps)));
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      const bool ok = v < nvec;
      if (RES == 1 && ok)
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.residual_out) + (size_t)row * a.H)[v] = pack8(h[j]);
      if (RES == 2 && ok) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.residual_out) + (size_t)row * a.H) + 2 * v;
        d[0] = make_float4(h[j][0], h[j][1], h[j][2], h[j][3]);
        d[1] = make_float4(h[j][4], h[j][5], h[j][6], h[j][7]);
      }
      float w[8];
      if (!ok) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0.0f;
      } else if (a.weight_f32) {
        const float4* wp = static_cast<const float4*>(a.weight) + 2 * v;
        const float4 w0 = __ldg(wp), w1 = __ldg(wp + 1);
        w[0] = w0.x, w[1] = w0.y, w[2] = w0.z, w[3] = w0.w, w[4] = w1.x, w[5] = w1.y, w[6] = w1.z, w[7] = w1.w;
      } else {
        unpack8(__ldg(static_cast<const uint4*>(a.weight) + v), w);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = __fmul_rn(__fmul_rn(h[j][i], r), w[i]);
      if (a.out && ok) reinterpret_cast<uint4*>(a.out + (size_t)row * a.H)[v] = pack8(h[j]);
      if (a.q) {
        float amax = 0.0f;
        if (ok) {
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(h[j][i]));
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        const float s = block_scale(amax);
        const uint2 c = codes8(h[j], s);
        if (ok) {
          reinterpret_cast<uint2*>(a.q + (size_t)row * a.H)[v] = c;
          if ((lane & 15) == 0) a.q_scales[(size_t)row * (a.H / 128) + v / 16] = s;
        }
      }
    }
  }
}

constexpr int kNormMaxH = 65536;   // 1024 threads of 8 vectors
constexpr int kNormMaxT = 1 << 30;  // a row and the grid's step to the next one in 32 bits

template <int VPT, bool AHEAD>
void launch_norm(const NormArgs& a, int threads, int blocks, cudaStream_t s) {
  if (!a.residual)
    rmsnorm_kernel<VPT, 0, AHEAD><<<blocks, threads, 0, s>>>(a);
  else if (!a.residual_f32)
    rmsnorm_kernel<VPT, 1, AHEAD><<<blocks, threads, 0, s>>>(a);
  else
    rmsnorm_kernel<VPT, 2, AHEAD><<<blocks, threads, 0, s>>>(a);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_rmsnorm(const uint16_t* x, int T, int H, long long x_stride, const void* weight,
                                    int weight_f32, float eps, const void* residual, int residual_f32,
                                    void* residual_out, uint16_t* out, uint8_t* q, float* q_scales,
                                    const int32_t* num_tokens, void* stream) {
  using namespace moe;
  if (T < 0 || T > kNormMaxT || H <= 0 || H % 8 != 0 || H > kNormMaxH || !(eps >= 0.0f)) return MOE_ERR_ARG;
  if ((weight_f32 != 0 && weight_f32 != 1) || (residual_f32 != 0 && residual_f32 != 1)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;   // tensors without rows have no addresses
  if (!out && !q) return MOE_ERR_ARG;
  if (q && H % 128 != 0) return MOE_ERR_ARG;
  if ((q != nullptr) != (q_scales != nullptr) || (residual != nullptr) != (residual_out != nullptr)) return MOE_ERR_ARG;
  if (!x || !weight || x_stride % 8 != 0 || (T > 1 && x_stride < H)) return MOE_ERR_ARG;
  if (!aligned16(x) || !aligned16(weight) || !aligned16(residual) || !aligned16(residual_out) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(q) & 7) || (reinterpret_cast<uintptr_t>(q_scales) & 3) ||
      (reinterpret_cast<uintptr_t>(num_tokens) & 3))
    return MOE_ERR_ARG;
  NormArgs a{x, x_stride, T, H, weight, weight_f32, eps, residual, residual_f32, residual_out, out, q, q_scales, num_tokens};
  cudaStream_t s = as_stream(stream);
  const int nvec = H / 8;
  auto threads = [&](int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; };
  if (threads(1) <= 1024 && T <= num_sms())
    launch_norm<1, false>(a, threads(1), T, s);
  else if (threads(2) <= 512)
    launch_norm<2, true>(a, threads(2), std::min(T, num_sms() * (1024 / threads(2))), s);
  else if (threads(4) <= 1024)
    launch_norm<4, false>(a, threads(4), std::min(T, num_sms() * std::max(1, 1024 / threads(4))), s);
  else
    launch_norm<8, false>(a, threads(8), std::min(T, num_sms()), s);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
