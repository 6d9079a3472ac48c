// moe_linear_e4m3 on the 5th-generation tensor cores for up to 32 rows of x: the weights are the MMA's M operand (128 rows),
// the rows of x its N (32 columns), so that a K block of 16 KB of weights needs 4 KB of x beside it, where a 128-row tile
// of x would be mostly padding.  Such a call is a stream of weights, each read once: 32 x 40960 x 4096 32.1 us (5.2 TB/s; 38
// with 128 x 64 tiles), 32 x 4096 x 7168 10.7 us with each tile's K in four parts (12.0 in two).  The same with 64 or 128 columns
// was not kept: 64 x 4096 x 7168 13.1 against 12.5, 64 x 40960 x 4096 37.0 against 39.4, 128 x 40960 x 4096 59 against 42 (the
// scales of each column have to be fetched for each block).
//
// As in linear_e4m3_tc.cu every K block is an accumulation of its own, scaled and added to float32 registers.  Here a lane
// holds a weight row and the columns are rows of x, so the scales differ from column to column: warp 3 multiplies a block's
// row scales with its weight scale (one for 128 rows) and leaves them in shared memory, a buffer for each accumulator,
// from where the epilogue warps read them four at a time.  Results leave straight from registers: the lanes of a warp are
// neighbours in a row of out.
//
// Warps: 0 TMA, 1 and 2 MMA issuers (1 allocates the tensor memory), 3 scales, 4..11 epilogue: warp w reads TMEM lanes
// 32 (w % 4).. of every second K block (warps 4..7 the even ones, 8..11 the odd ones); the sums of the two meet in shared
// memory at the end of a tile.  Shared K and bounded waits as in linear_e4m3_tc.cu.
#include "linear_e4m3_tc.cuh"

namespace moe {
namespace lin8 {

namespace {

constexpr int EPI = 8;

struct C {
  static constexpr int TB = SWAP_ROWS;
  static constexpr int stage = A_BYTES + TB * KB_BYTES;
  static constexpr int stages = 192 * 1024 / stage < 8 ? 192 * 1024 / stage : 8;
  static constexpr int bufs = 4;
  static constexpr int tmem = bufs * TB;
  static constexpr int meet_bytes = 16 * 32 * 4;               // of an epilogue warp
  static constexpr int meets = stages * stage;
  static constexpr int scales = meets + EPI * meet_bytes;      // float [bufs][TB]
  static constexpr int bars = scales + bufs * TB * 4;
  static constexpr int n_bars = 2 * stages + 2 * bufs + 2;
  static constexpr int smem = bars + n_bars * 8 + 16 + 1024;   // + align slack
  static_assert(smem <= SMEM_MAX, "shared memory");
  static_assert(stage % 1024 == 0, "swizzle atoms");
  static_assert(TB == 32, "a lane of the scale warp to a row of x, one load of an accumulator");
};

__global__ void __launch_bounds__(TC_THREADS, 1)
    linear_swap_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Args a,
                       const Split split) {
  constexpr int TB = C::TB;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  float* scales = reinterpret_cast<float*>(smem + C::scales);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::bars);
  auto bar_full = [&](int s) { return smem_u32(bars + s); };
  auto bar_done = [&](int s) { return smem_u32(bars + C::stages + s); };
  auto bar_tempty = [&](int b) { return smem_u32(bars + 2 * C::stages + b); };             // accumulator and scales read
  auto bar_sfull = [&](int b) { return smem_u32(bars + 2 * C::stages + C::bufs + b); };    // scales written
  const uint32_t bar_drain = smem_u32(bars + 2 * C::stages + 2 * C::bufs);                 // two
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::n_bars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int kblocks = a.K / 128, tiles = (a.N + 127) / 128;

  if (tid == 96) {
    for (int s = 0; s < C::stages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_done(s), 1);
    }
    for (int b = 0; b < C::bufs; ++b) {
      mbar_init(bar_tempty(b), EPI / 2);
      mbar_init(bar_sfull(b), 1);
    }
    mbar_init(bar_drain, 1);
    mbar_init(bar_drain + 8, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(C::tmem));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag, a.dev_status, a.limit_ns); };
  Walk walk((int)blockIdx.x, tiles, kblocks, split);
  Piece p;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      if (elect_one())
        load_tiles<C::stages, C::stage>(walk, &tmW, &tmX, sbase, bar_full(0), bar_done(0), wait, [&](int tile, int& ra, int& rb) {
          ra = tile * 128;
          rb = 0;
        });
    } else if (warp < 3) {
      if (!a.mute && elect_one())
        issue_mmas<C::stages, C::stage, C::bufs, TB>(walk, (uint32_t)warp - 1, sbase, tmem_base, bar_full(0), bar_done(0),
                                                     bar_tempty(0), bar_drain, wait);
    } else {
      // -------------------------------------------------------------- scales: lane l that of row l
      int buf = 0;
      uint32_t tphase = 0;
      bool ok = true;
      while (ok && walk.get(p)) {
        const float* ws = a.w_scales + (long long)p.tile * kblocks;
        const float* xs = a.x_scales + (long long)min(lane, a.T - 1) * kblocks;
        float x = __ldg(xs + p.k0), w = __ldg(ws + p.k0);
        for (int kb = p.k0; kb < p.k1; ++kb) {
          const float s = __fmul_rn(x, w);
          if (kb + 1 < p.k1) {
            w = __ldg(ws + kb + 1);
            x = __ldg(xs + kb + 1);
          }
          if (!__all_sync(0xffffffffu, wait(bar_tempty(buf), tphase ^ 1))) {
            ok = false;
            break;
          }
          scales[buf * TB + lane] = s;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_sfull(buf));
          if (++buf == C::bufs) {
            buf = 0;
            tphase ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // ---------------------------------------------------------------- epilogue: the warpgroups take K blocks in turns
    const int ew = warp - 4, q = warp & 3, half = ew >> 2;
    const uint32_t lane_addr = (uint32_t)(32 * q) << 16;
    float* mine = reinterpret_cast<float*>(smem + C::meets + ew * C::meet_bytes);
    const float* other = reinterpret_cast<const float*>(smem + C::meets + (ew ^ 4) * C::meet_bytes);
    int buf = 0, stage = 0;
    uint32_t phase = 0, bphase = 0, g = (uint32_t)half;
    bool ok = true;
    while (ok && walk.get(p)) {
      float acc[TB];
#pragma unroll
      for (int i = 0; i < TB; ++i) acc[i] = 0.0f;
      for (int kb = p.k0; kb < p.k1; ++kb, ++g) {
        if ((g & 1u) == 0) {
          // the warp leaves together: what follows is executed by all of its lanes
          if (!__all_sync(0xffffffffu, wait(bar_sfull(buf), bphase) && wait(bar_done(stage), phase))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tb = tmem_base + lane_addr + buf * TB;
          const float4* sc = reinterpret_cast<const float4*>(scales + buf * TB);
          uint32_t r[32];
          float4 f[8];
          tmem_ld32(tb, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = sc[i];
          wait_ld(r);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[4 * i] = fmaf(__uint_as_float(r[4 * i]), f[i].x, acc[4 * i]);
            acc[4 * i + 1] = fmaf(__uint_as_float(r[4 * i + 1]), f[i].y, acc[4 * i + 1]);
            acc[4 * i + 2] = fmaf(__uint_as_float(r[4 * i + 2]), f[i].z, acc[4 * i + 2]);
            acc[4 * i + 3] = fmaf(__uint_as_float(r[4 * i + 3]), f[i].w, acc[4 * i + 3]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_tempty(buf));
        }
        if (++buf == C::bufs) {
          buf = 0;
          bphase ^= 1;
        }
        if (++stage == C::stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      constexpr int KEEP = TB / 2;
      float v[KEEP];
      if (!meet<16>(acc, v, mine, other, half, lane, 1 + q, ok)) break;
      const int n = p.tile * 128 + 32 * q + lane, t0 = half * KEEP;
      if (p.tile * 128 + 32 * q >= a.N || t0 >= a.T) continue;
      if (p.tile >= split.whole && !join_parts(a, split, p.tile, (int)blockIdx.x, ew, lane, v)) continue;
      if (n < a.N) {
        const float b = a.bias ? __ldg(a.bias + n) : 0.0f;
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
          if (t0 + i < a.T) {
            const float o = a.bias ? __fadd_rn(v[i], b) : v[i];
            const long long at = (long long)(t0 + i) * a.out_stride + n;
            if (a.out_f32)
              static_cast<float*>(a.out)[at] = o;
            else
              static_cast<uint16_t*>(a.out)[at] = f32_to_bf16(o);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(C::tmem));
}

}  // namespace

moe_status_t launch_swap(const Args& a, const Split& split, cudaStream_t s) {
  static std::atomic<unsigned long long> attr_done{0};
  if (!once_per_device(attr_done, [&] {
        return cudaFuncSetAttribute(linear_swap_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem) == cudaSuccess;
      }))
    return MOE_ERR_CUDA;
  CUtensorMap mw, mx;
  if (!make_map(&mw, a.w, true, a.K, a.N) || !make_map(&mx, a.x, true, a.K, a.T, C::TB)) return MOE_ERR_CUDA;
  linear_swap_kernel<<<split.workers, TC_THREADS, C::smem, s>>>(mw, mx, a, split);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

}  // namespace lin8
}  // namespace moe
