// Pieces shared by moe_linear_e4m3's tensor-core kernels (linear_e4m3_tc.cu: rows of x as the MMA's M; linear_e4m3_swap.cu:
// weight rows): how a worker walks its tiles, the TMA and MMA roles.  Internal header.
#pragma once

#include "gemm_common.cuh"
#include "linear_e4m3.cuh"

namespace moe {
namespace lin8 {

using namespace gg;

constexpr int TC_THREADS = 384;

// tcgen05.wait::ld, with the loaded registers as operands: nothing that uses them is moved ahead of it.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
// One lane of a converged warp: elect.sync names a single thread where a condition on the lane's number only happens to.
// Measured on the product of 128-column tiles (8192 x 4096 x 7168): 228 us behind elect.sync, 326 behind lane == 0.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.b32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// A stretch of one tile's K.
struct Piece {
  int tile, k0, k1;
};
// The pieces of worker `w`, in order (the same for every role of its CTA): whole tiles, one for each round of the workers,
// then its part of the one tile that it shares.
struct Walk {
  int next, step, whole, shared, k0, k1, kblocks;
  __device__ __forceinline__ Walk(int w, int tiles, int kblocks_, const Split& s)
      : next(w), step(s.workers), whole(s.whole), shared(w < (tiles - s.whole) * s.parts ? s.whole + w / s.parts : -1),
        k0((int)((long long)kblocks_ * (w % s.parts) / s.parts)), k1((int)((long long)kblocks_ * (w % s.parts + 1) / s.parts)),
        kblocks(kblocks_) {}
  __device__ __forceinline__ bool get(Piece& p) {
    if (next < whole) {
      p = Piece{next, 0, kblocks};
      next += step;
      return true;
    }
    if (shared < 0) return false;
    p = Piece{shared, k0, k1};
    shared = -1;
    return true;
  }
};

// Join of a shared tile's parts: a warp's N sums of each lane go to this worker's slot, and the last of the tile's parts to be
// counted gets all of them, added up in their order; false for the others.  (Loading several parts at once cost the K
// loop more, by what the registers were given to: 12.9 -> 20.3 us at 24 x 576 x 7168.)
template <int N>
__device__ __forceinline__ bool join_parts(const Args& a, const Split& split, int tile, int worker, int ew, int lane, float (&v)[N]) {
  auto slot = [&](int w) { return reinterpret_cast<float4*>(a.part) + ((size_t)w * 8 + ew) * (N * 8) + lane; };
  float4* own = slot(worker);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) __stcg(own + 32 * i, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
  __syncwarp();
  int before = 0;
  int32_t* count = a.count + (tile - split.whole) * 8 + ew;
  if (lane == 0) asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(count) : "memory");
  before = __shfl_sync(0xffffffffu, before, 0);
  if (before != split.parts - 1) return false;
  if (lane == 0) *count = 0;
  __syncwarp();
  const int first = worker - worker % split.parts;
  for (int w = 0; w < split.parts; ++w) {
    float4 f[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) f[i] = __ldcg(slot(first + w) + 32 * i);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float u[4] = {f[i].x, f[i].y, f[i].z, f[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = w ? __fadd_rn(v[4 * i + j], u[j]) : u[j];
    }
  }
  return true;
}

// The epilogue's two warpgroups took even and odd K blocks in turns, all N columns each; the warps of a pair (the same
// TMEM lanes) now give each other half of their columns' sums, through their buffers of CHUNK x 32 floats, and keep the
// sums of the other half in v.  False (for both) where a wait of one of them ran out.
template <int CHUNK, int N>
__device__ __forceinline__ bool meet(const float (&acc)[N], float (&v)[N / 2], float* mine, const float* other, int half, int lane,
                                     uint32_t barrier, bool ok) {
#pragma unroll
  for (int c = 0; c < N / 2; c += CHUNK) {
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) mine[i * 32 + lane] = half ? acc[c + i] : acc[N / 2 + c + i];
    if (bar_red_or(barrier, 64, !ok)) return false;
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) v[c + i] = __fadd_rn(half ? acc[N / 2 + c + i] : acc[c + i], other[i * 32 + lane]);
    asm volatile("bar.sync %0, 64;" ::"r"(barrier) : "memory");     // both have read; the buffers are free again
  }
  return true;
}

// TMA producer (one thread): the operands of the worker's K blocks, 128 rows of the M operand and STAGE - 16 KB of the N
// operand a stage, at the rows that rows_of(tile, ra, rb) gives.
template <int STAGES, int STAGE, class Wait, class Rows>
__device__ __forceinline__ void load_tiles(Walk walk, const CUtensorMap* tmA, const CUtensorMap* tmB, uint32_t ring, uint32_t full,
                                           uint32_t done, Wait&& wait, Rows&& rows_of) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tmA)) : "memory");
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tmB)) : "memory");
  int stage = 0;
  uint32_t phase = 0, armed = 0, last_parity = 0;
  bool ok = true;
  Piece p;
  while (ok && walk.get(p)) {
    int ra, rb;
    rows_of(p.tile, ra, rb);
    for (int kb = p.k0; kb < p.k1; ++kb) {
      if (!wait(done + 8 * stage, phase ^ 1)) {
        ok = false;
        break;
      }
      armed |= 1u << stage;
      last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
      const uint32_t sa = ring + stage * STAGE;
      mbar_expect_tx(full + 8 * stage, STAGE);
      tma_load_2d(sa, tmA, kb * 128, ra, full + 8 * stage);
      tma_load_2d(sa + A_BYTES, tmB, kb * 128, rb, full + 8 * stage);
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
  // a stage's copies, and the MMAs that read them, are over before this CTA's shared memory goes away; where a wait ran out
  // its MMAs may never be issued, and the copies are waited for
  for (int s = 0; s < STAGES; ++s) {
    if (!(armed & (1u << s))) continue;
    const uint32_t parity = (last_parity >> s) & 1u;
    ok = ok && wait(done + 8 * s, parity);
    if (!ok) mbar_drain(full + 8 * s, parity);
  }
}

// MMA issuer `lane01` of two (one thread each): even and odd K blocks of the CTA's sequence.  The stages and accumulators are
// even in number, so each issuer has its own of them.  Every K block is an accumulation of its own, into buffer
// (block % BUFS) of N columns.
template <int STAGES, int STAGE, int BUFS, int N, class Wait>
__device__ __forceinline__ void issue_mmas(Walk walk, uint32_t lane01, uint32_t ring, uint32_t tmem, uint32_t full, uint32_t done,
                                           uint32_t tempty, uint32_t drain, Wait&& wait) {
  static_assert(STAGES % 2 == 0 && BUFS % 2 == 0, "each issuer's own stages and buffers");
  constexpr uint32_t idesc = (1u << 4) | (uint32_t)(N >> 3) << 17 | (uint32_t)(128 >> 4) << 24;   // E4M3 x E4M3 -> float32
  int stage = 0, buf = 0;
  uint32_t phase = 0, tphase = 0, g = lane01;
  bool ok = true;
  Piece p;
  while (ok && walk.get(p)) {
    for (int kb = p.k0; kb < p.k1; ++kb, ++g) {
      if ((g & 1u) == 0) {
        if (!wait(full + 8 * stage, phase) || !wait(tempty + 8 * buf, tphase ^ 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sa = ring + stage * STAGE, dt = tmem + buf * N;
#pragma unroll
        for (int k = 0; k < 4; ++k) tc_mma<true>(dt, smem_desc(sa + 32 * k), smem_desc(sa + A_BYTES + 32 * k), idesc, k != 0);
        tc_commit(done + 8 * stage);
      }
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
      if (++buf == BUFS) {
        buf = 0;
        tphase ^= 1;
      }
    }
  }
  if (!ok) {
    tc_commit(drain + 8 * lane01);   // arrives once every MMA that this thread issued has completed
    mbar_drain(drain + 8 * lane01, 0);
  }
}

}  // namespace lin8
}  // namespace moe
