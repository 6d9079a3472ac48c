// moe_linear_e4m3's three kernels (few rows, tiles of rows of x, weight rows as M) and how a call is cut.  Internal header.
#pragma once

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
  int32_t* count;          // arrivals at the tiles whose K is shared, zero between launches
  float* part;             // their sums
  int32_t* dev_status;
  unsigned long long limit_ns;   // of each wait
  int mute;                // tests only: what the waits are for is never issued, so that they run out
};

constexpr unsigned long long LIMIT_NS = 2000000000ull;

// A workspace: the counters (eight for each shared tile, of which there are fewer than SMs), then the sums of the parts (of at
// most 128 x 128 values, no more of them than SMs).
inline size_t count_bytes() { return ((size_t)num_sms() * 32 + 255) / 256 * 256; }
inline size_t sum_bytes() { return (size_t)num_sms() * 128 * 128 * 4; }

// Variants of the tensor-core kernels: tiles of 128 rows of x by 64, 128 or 256 weight rows (linear_e4m3_tc.cu), or of 128
// weight rows by all of up to 32 rows of x (linear_e4m3_swap.cu).
enum Variant { TC_64 = 0, TC_128 = 1, TC_256 = 2, SWAP = 3, VARIANTS = 4 };
constexpr int SWAP_ROWS = 32;

// Tiles [0, whole): worker w computes the tiles w, w + workers, ..  The others are shared: worker w computes part w % parts
// of tile whole + w / parts, if there is one.
struct Split {
  int workers, whole, parts;
};

moe_status_t launch_tc(Variant v, const Args& a, const Split& split, cudaStream_t s);
moe_status_t launch_swap(const Args& a, const Split& split, cudaStream_t s);

}  // namespace lin8
}  // namespace moe
