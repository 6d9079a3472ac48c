// moe_linear_e4m3: out[t, n] = sum_b xs[t, b] * ws[n / 128, b] * (sum over the 128 columns k of block b of
// x[t, k] * w[n, k]) (+ bias[n]), x and w E4M3, every sum in float32, one rounding at the end.
//
// The weights are the 16-row operand of mma.sync and the rows of x its 8 columns.  A 128-column block is four
// instructions of 32 columns; which column sits where inside a block does not matter as long as both operands agree, so a
// lane loads 16 consecutive bytes of a row and uses them as the operands of two instructions.
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace lin8 {

struct Args {
  const uint8_t* x;
  const float* x_scales;
  const uint8_t* w;
  const float* w_scales;
  const float* bias;
  void* out;
  long long out_stride;
  int T, N, K, out_f32;
};

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int ROWS = 16, COLS = 32, NT = COLS / 8, WARPS = 8;

__global__ void __launch_bounds__(WARPS * 32) linear_kernel(const Args a) {
  __shared__ float part[WARPS][NT][4][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int n0 = blockIdx.x * ROWS, t0 = blockIdx.y * COLS, kblocks = a.K / 128;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const bool r0 = n0 + g < a.N, r1 = n0 + g + 8 < a.N;
  float acc[NT][4] = {};
  for (int kb = warp; kb < kblocks; kb += WARPS) {
    const uint8_t* w0 = a.w + (size_t)(n0 + g) * a.K + kb * 128 + 16 * c;
    const uint8_t* w1 = w0 + (size_t)8 * a.K;
    uint4 p[2], q[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      p[j] = r0 ? __ldg(reinterpret_cast<const uint4*>(w0 + 64 * j)) : zero;
      q[j] = r1 ? __ldg(reinterpret_cast<const uint4*>(w1 + 64 * j)) : zero;
    }
    const float ws = a.w_scales[(size_t)(n0 / 128) * kblocks + kb];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = t0 + 8 * i + g;
      float d[4] = {};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 b = t < a.T ? __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)t * a.K + kb * 128 + 16 * c + 64 * j)) : zero;
        mma_e4m3(d, p[j].x, q[j].x, p[j].y, q[j].y, b.x, b.y);
        mma_e4m3(d, p[j].z, q[j].z, p[j].w, q[j].w, b.z, b.w);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int col = t0 + 8 * i + 2 * c + h;
        const float s = col < a.T ? __fmul_rn(a.x_scales[(size_t)col * kblocks + kb], ws) : 0.0f;
        acc[i][h] = fmaf(d[h], s, acc[i][h]);
        acc[i][2 + h] = fmaf(d[2 + h], s, acc[i][2 + h]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) part[warp][i][v][lane] = acc[i][v];
  __syncthreads();
  for (int e = threadIdx.x; e < NT * 128; e += WARPS * 32) {
    // element e: row r of the tile, column t of the block
    const int r = e & 15, t = e >> 4;
    const int l = (r & 7) * 4 + ((t & 7) >> 1), v = (r >> 3) * 2 + (t & 1);
    float s = 0.0f;
    for (int w = 0; w < WARPS; ++w) s += part[w][t >> 3][v][l];
    if (n0 + r >= a.N || t0 + t >= a.T) continue;
    if (a.bias) s += a.bias[n0 + r];
    const long long o = (long long)(t0 + t) * a.out_stride + n0 + r;
    if (a.out_f32)
      static_cast<float*>(a.out)[o] = s;
    else
      static_cast<uint16_t*>(a.out)[o] = f32_to_bf16(s);
  }
}

inline bool shape_ok(int T, int N, int K) { return T >= 0 && N > 0 && K > 0 && K % 128 == 0 && N <= (1 << 24) && K <= (1 << 22); }

}  // namespace lin8
}  // namespace moe

extern "C" size_t moe_linear_e4m3_workspace_bytes(int T, int N, int K) {
  return moe::lin8::shape_ok(T, N, K) ? 256 : 0;
}

extern "C" moe_status_t moe_linear_e4m3(const uint8_t* x, const float* x_scales, int T, int K, const uint8_t* w,
                                        const float* w_scales, int N, const float* bias, void* out, int out_f32,
                                        long long out_stride, void* ws, size_t ws_bytes, int32_t* dev_status,
                                        void* stream) {
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
  if ((T + COLS - 1) / COLS > 65535) return MOE_ERR_UNSUPPORTED;
  const Args a{x, x_scales, w, w_scales, bias, out, out_stride, T, N, K, out_f32};
  linear_kernel<<<dim3((N + ROWS - 1) / ROWS, (T + COLS - 1) / COLS), WARPS * 32, 0, as_stream(stream)>>>(a);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
