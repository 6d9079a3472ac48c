// moe_linear_e4m3 on the 5th-generation tensor cores, for calls of many rows.
//
// out[t, n] = sum_b xs[t, b] ws[n / 128, b] (sum over block b's 128 columns of x w).  The scales are float32 values of
// blocks of 128, not a format that the MMA applies itself, so every block is an accumulation of its own: the MMAs of a K
// block write a fresh accumulator in tensor memory, and the epilogue warps add it, times the product of its two
// scales, to float32 sums in registers ("promotion") while the MMAs of the next blocks run.  A tile's 128 x BN float32
// sums therefore have to fit into the registers of eight warps (BN <= 256: 128 of a thread's 224).
//
// What bounds it (8192 x 4096 x 7168, 200 us, 2400 TFLOP/s; a K block of a 128 x 256 tile takes 900 cycles where its MMAs need
// 512): the hand-over of an accumulator.  Two of them fill tensor memory, and from a block's first MMA to the one that
// overwrites it pass the MMAs, 280 cycles until the epilogue warps see them done, 400 until its 128 columns are
// read (64 at a time: the sums leave no registers for more), and 300 until the issuing thread sees them free.  The same loop
// without the reading takes 715, and without the MMAs 600 (operand tiles from L2, 48 KB a block, 19 TB/s).
//   Tried and not kept: pairs of SMs (cta_group::2, M = 256, 32 KB a block): 222 us where this took 207, each hand-over crosses
//   an SM more; 192 columns, read at once: 265; 128 columns, four accumulators: 236 here and behind 64 or 256 at every other
//   size; two MMAs of 128 columns with barriers of their own: 236; packed fma.f32x2: 228 against 217 (its operands have to be
//   moved into pairs); sixteen epilogue warps of 64 columns: 208.
//   Kept: one lane issues, named by elect.sync instead of a condition on its number (128 columns: 326 -> 228 us);
//   one commit per block, on whose barrier both the producer and the epilogue wait; the accumulator is given back before
//   its last 64 columns are added (217 -> 207); two issuing threads, even and odd blocks (64 columns: 345 -> 308); 56 registers
//   for the first warpgroup, whose threads kept some in local memory with 40 (207 -> 200).
//
// Warps (384 threads, one CTA per SM): 0 loads the operands by TMA; 1 and 2 issue the MMAs (1 allocates the tensor
// memory); 3 is idle; 4..11 epilogue: warp w reads TMEM lanes 32 (w % 4).. and half (w - 4) / 4 of the columns.  The first
// warpgroup gives its registers to the other two.
//
// Shared K (64 and 128 columns, the tiles of a last, partly filled round): the K of each tile is cut into equal parts, a CTA each; an epilogue warp leaves its sums
// in the workspace and counts itself in, and the last of a tile's parts to arrive adds all of them up in their order.  No
// one waits.
//
// Every wait is bounded; on expiry the CTA sets MOE_DEV_PIPELINE_TIMEOUT and every role leaves its loop, as in the
// grouped GEMM kernels.
#include "linear_e4m3_tc.cuh"

namespace moe {
namespace lin8 {

namespace {

constexpr int EPI = 8;
constexpr int STAGE_RING = 192 * 1024;
constexpr int OUT_BYTES = 32 * 128;      // an epilogue warp's transpose: 32 rows of 128 bytes

template <int BN_>
struct Cfg {
  static constexpr int stage = A_BYTES + BN_ * KB_BYTES;
  static constexpr int stages = STAGE_RING / stage < 8 ? STAGE_RING / stage : 8;
  static constexpr int bufs = 512 / BN_ < 4 ? 512 / BN_ : 4;
  static constexpr int tmem = bufs * BN_;
  // TURNS: the epilogue's two warpgroups take even and odd K blocks in turns, all columns each; else every block, half of
  // the columns each
  static constexpr bool TURNS = BN_ == 128;
  static constexpr int cols = TURNS ? BN_ : BN_ / 2;           // of an epilogue warp
  static constexpr int out = stages * stage;
  static constexpr int bars = out + EPI * OUT_BYTES;
  static constexpr int n_bars = 2 * stages + bufs + 2;
  static constexpr int smem = bars + n_bars * 8 + 16 + 1024;   // + align slack
  static_assert(smem <= SMEM_MAX, "shared memory");
  static_assert(stage % 1024 == 0, "swizzle atoms");
};

// Tile -> row tile and column tile: groups of 8 row tiles, column tile after column tile inside a group, so that
// the workers of a round share both operands' tiles in L2.
constexpr int GROUP_M = 8;
__device__ __forceinline__ void tile_at(int tile, int mt, int nt, int& m, int& n) {
  const int per = GROUP_M * nt, g = tile / per, r = tile - g * per;
  const int gm = min(GROUP_M, mt - g * GROUP_M);
  n = r / gm;
  m = g * GROUP_M + r - n * gm;
}

// 32 rows (lane = row) x 32 columns of sums, from column col on, into out: through the warp's transpose in shared
// memory, so that a store covers whole sectors.  Rows [0, rows) and columns below N are stored.
__device__ __forceinline__ void store_chunk(const Args& a, const float (&v)[32], uint8_t* buf, int lane, long long row0,
                                            int rows, int col, bool vec) {
  const bool full = vec && col + 32 <= a.N;
  if (full && !a.out_f32) {
    uint16_t* out = static_cast<uint16_t*>(a.out);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = (uint32_t)f32_to_bf16(v[8 * p + 2 * j]) | ((uint32_t)f32_to_bf16(v[8 * p + 2 * j + 1]) << 16);
      *reinterpret_cast<uint4*>(buf + stage_out_off(lane, p)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (lane >> 2) + 8 * i, p = lane & 3;
      const uint4 o = *reinterpret_cast<const uint4*>(buf + stage_out_off(r, p));
      if (r < rows) *reinterpret_cast<uint4*>(out + (row0 + r) * a.out_stride + col + 8 * p) = o;
    }
  } else {
#pragma unroll
    for (int p = 0; p < 8; ++p)
      *reinterpret_cast<float4*>(buf + lane * 128 + ((p ^ (lane & 7)) << 4)) =
          make_float4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
    __syncwarp();
    if (full) {
      float* out = static_cast<float*>(a.out);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = (lane >> 3) + 4 * i, p = lane & 7;
        const float4 o = *reinterpret_cast<const float4*>(buf + r * 128 + ((p ^ (r & 7)) << 4));
        if (r < rows) *reinterpret_cast<float4*>(out + (row0 + r) * a.out_stride + col + 4 * p) = o;
      }
    } else if (col < a.N) {
      // the edge of N, and rows that do not start on 16 bytes: a value per lane
      const bool ok = col + lane < a.N;
      for (int r = 0; r < min(rows, 32); ++r) {
        const float o = *reinterpret_cast<const float*>(buf + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + 4 * (lane & 3));
        const long long at = (row0 + r) * a.out_stride + col + lane;
        if (ok) {
          if (a.out_f32)
            static_cast<float*>(a.out)[at] = o;
          else
            static_cast<uint16_t*>(a.out)[at] = f32_to_bf16(o);
        }
      }
    }
  }
  __syncwarp();
}
__device__ __forceinline__ void add_bias(const Args& a, float (&v)[32], int col) {
  if (!a.bias) return;
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (col + i < a.N) v[i] = __fadd_rn(v[i], __ldg(a.bias + col + i));
}

template <int BN_>
__global__ void __launch_bounds__(TC_THREADS, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Args a,
                     const Split split) {
  using C = Cfg<BN_>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::bars);
  auto bar_full = [&](int s) { return smem_u32(bars + s); };
  // a stage's MMAs are complete: its operands may be overwritten, its accumulator read
  auto bar_done = [&](int s) { return smem_u32(bars + C::stages + s); };
  auto bar_tempty = [&](int b) { return smem_u32(bars + 2 * C::stages + b); };
  const uint32_t bar_drain = smem_u32(bars + 2 * C::stages + C::bufs);   // two
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::n_bars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int worker = (int)blockIdx.x;
  const int kblocks = a.K / 128;
  const int mt = (a.T + 127) / 128, nt = (a.N + BN_ - 1) / BN_;

  if (tid == 96) {
    for (int s = 0; s < C::stages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_done(s), 1);
    }
    for (int b = 0; b < C::bufs; ++b) mbar_init(bar_tempty(b), C::TURNS ? EPI / 2 : EPI);
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
  Walk walk(worker, mt * nt, kblocks, split);
  Piece p;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && elect_one()) {
      load_tiles<C::stages, C::stage>(walk, &tmA, &tmB, sbase, bar_full(0), bar_done(0), wait, [&](int tile, int& ra, int& rb) {
        tile_at(tile, mt, nt, ra, rb);
        ra *= 128;
        rb *= BN_;
      });
    } else if ((warp == 1 || warp == 2) && !a.mute && elect_one()) {
      issue_mmas<C::stages, C::stage, C::bufs, BN_>(walk, (uint32_t)warp - 1, sbase, tmem_base, bar_full(0), bar_done(0),
                                                    bar_tempty(0), bar_drain, wait);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // ---------------------------------------------------------------- epilogue
    const int ew = warp - 4, q = warp & 3, half = ew >> 2;
    const uint32_t lane_addr = (uint32_t)(32 * q) << 16;
    uint8_t* buf_w = smem + C::out + ew * OUT_BYTES;
    const bool vec = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && a.out_stride % (a.out_f32 ? 4 : 8) == 0;
    int buf = 0, stage = 0;
    uint32_t phase = 0, g = (uint32_t)half;     // g: K blocks until this warp's next one (TURNS)
    bool ok = true;
    while (ok && walk.get(p)) {
      int m, n;
      tile_at(p.tile, mt, nt, m, n);
      const long long row0 = (long long)m * 128 + 32 * q;
      const int rows = (int)min((long long)32, a.T - row0);     // of this warp that exist (may be negative)
      const int col0 = n * BN_ + (C::TURNS ? 0 : half * C::cols);
      const bool live = rows > 0 && col0 < a.N;
      float acc[C::cols];
#pragma unroll
      for (int i = 0; i < C::cols; ++i) acc[i] = 0.0f;
      const float* xs = a.x_scales + (row0 + min(lane, max(rows - 1, 0))) * kblocks;
      const float* ws = a.w_scales + (long long)(col0 >> 7) * kblocks;
      constexpr int STEP = C::TURNS ? 2 : 1;
      const int kb0 = p.k0 + (C::TURNS ? (int)(g & 1u) : 0);     // the first that is this warp's
      float sx = live && kb0 < p.k1 ? __ldg(xs + kb0) : 0.0f, sw = live && kb0 < p.k1 ? __ldg(ws + kb0) : 0.0f;
      for (int kb = p.k0; kb < p.k1; ++kb, ++g) {
        if (!C::TURNS || (g & 1u) == 0) {
          const float s = __fmul_rn(sx, sw);
          if (live && kb + STEP < p.k1) {
            sx = __ldg(xs + kb + STEP);
            sw = __ldg(ws + kb + STEP);
          }
          // the warp leaves together: what follows is executed by all of its lanes
          if (!__all_sync(0xffffffffu, wait(bar_done(stage), phase))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tb = tmem_base + lane_addr + buf * BN_ + (C::TURNS ? 0 : half * C::cols);
          auto release = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_tempty(buf));
          };
          constexpr int CH = C::cols / 32;
          uint32_t r[2][32];
          auto add = [&](int c) {
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[32 * c + i] = fmaf(__uint_as_float(r[c & 1][i]), s, acc[32 * c + i]);
          };
          if (live) {
            tmem_ld32(tb, r[0]);
            if (CH > 1) tmem_ld32(tb + 32, r[1]);
            wait_ld(r[0]);
            if (CH > 1) wait_ld(r[1]);
            if (CH == 4) {
              add(0);
              tmem_ld32(tb + 64, r[0]);
              add(1);
              tmem_ld32(tb + 96, r[1]);
              wait_ld(r[0]);
              wait_ld(r[1]);
              release();
              add(2);
              add(3);
            } else {
              release();
              add(0);
              if (CH > 1) add(1);
            }
          } else {
            release();
          }
        }
        if (++buf == C::bufs) buf = 0;
        if (++stage == C::stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      auto store = [&](const float* sums, int c, int col) {
        float u[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i] = sums[c + i];
        add_bias(a, u, col + c);
        store_chunk(a, u, buf_w, lane, row0, rows, col + c, vec);
      };
      if constexpr (C::TURNS) {
        constexpr int KEEP = C::cols / 2;
        float v[KEEP];
        if (!meet<32>(acc, v, reinterpret_cast<float*>(buf_w), reinterpret_cast<const float*>(smem + C::out + (ew ^ 4) * OUT_BYTES),
                      half, lane, 1 + q, ok))
          break;
        const int col = col0 + KEEP * half;
        if (!live || col >= a.N) continue;
        if (p.tile >= split.whole && !join_parts(a, split, p.tile, worker, ew, lane, v)) continue;
#pragma unroll
        for (int c = 0; c < KEEP; c += 32) store(v, c, col);
      } else {
        if (!ok) break;
        if (!live) continue;
        if constexpr (BN_ == 64)
          if (p.tile >= split.whole && !join_parts(a, split, p.tile, worker, ew, lane, acc)) continue;
#pragma unroll
        for (int c = 0; c < C::cols; c += 32) store(acc, c, col0);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(C::tmem));
}

template <int BN_>
moe_status_t launch(const Args& a, const Split& split, cudaStream_t s) {
  using C = Cfg<BN_>;
  auto kern = linear_tc_kernel<BN_>;
  static std::atomic<unsigned long long> attr_done{0};
  if (!once_per_device(attr_done, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem) == cudaSuccess;
      }))
    return MOE_ERR_CUDA;
  CUtensorMap ma, mb;
  if (!make_map(&ma, a.x, true, a.K, a.T) || !make_map(&mb, a.w, true, a.K, a.N, BN_)) return MOE_ERR_CUDA;
  kern<<<split.workers, TC_THREADS, C::smem, s>>>(ma, mb, a, split);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

}  // namespace

moe_status_t launch_tc(Variant v, const Args& a, const Split& split, cudaStream_t s) {
  switch (v) {
    case TC_64: return launch<64>(a, split, s);
    case TC_128: return launch<128>(a, split, s);
    default: return launch<256>(a, split, s);
  }
}

}  // namespace lin8
}  // namespace moe
