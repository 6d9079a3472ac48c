// Host side of moe_layer_few: workspace, argument checks, choice of the weight format's kernel.
#include "few_layer.cuh"

namespace moe {
namespace few {

struct FewPlan {
  size_t off_tile, off_entry, off_htop, off_logits, off_x16, off_xunit, off_hexp, off_hhi, off_hlo, off_y, total;
};

inline bool plan_few(const moe_few_desc_t* d, FewPlan* p) {
  if (!d) return false;
  if (d->T < 0 || d->T > kMaxTokens || d->H <= 0 || d->I <= 0 || d->H % 128 || d->I % 128 || d->H > kMaxWidth ||
      d->I > kMaxWidth || d->E < 1 || d->E > kMaxExperts || d->K < 1 || d->K > d->E || d->K > kMaxTopK ||
      (d->has_shared != 0 && d->has_shared != 1) || (d->weight_tiles != 0 && d->weight_tiles != 1))
    return false;
  if (d->dtype != MOE_BF16 && d->dtype != MOE_E4M3 && d->dtype != MOE_W4) return false;
  if (d->zeros != 0 && d->zeros != 1) return false;
  if (d->dtype == MOE_W4 ? (d->group != 32 && d->group != 64 && d->group != 128) || d->weight_tiles
                         : d->group != 0 || d->zeros != 0)
    return false;
  const size_t slots = (size_t)d->T * d->K + d->T;
  const bool half = d->dtype != MOE_BF16;
  size_t o = 256;                                                       // barrier, queue
  // zero between calls; at the same places for every T
  p->off_tile = o;   o = align256(o + 4 * (size_t)(d->H / 32));
  p->off_entry = o;  o = align256(o + 4 * (size_t)kMaxEntries);
  p->off_htop = o;   o = align256(o + 4 * (size_t)kMaxTokens * (d->K + 1));
  // not kept
  p->off_logits = o; o = align256(o + 4 * (size_t)d->T * d->E);
  p->off_x16 = o;    o = align256(o + (half ? 2 * (size_t)d->T * half_pitch(d->H) : 0));
  p->off_xunit = o;  o = align256(o + 4 * (size_t)d->T);
  p->off_hexp = o;   o = align256(o + (half ? slots * exp_pitch(d->I) : 0));
  p->off_hhi = o;    o = align256(o + 2 * slots * (half ? half_pitch(d->I) : d->I));
  p->off_hlo = o;    o = align256(o + 2 * slots * (half ? half_pitch(d->I) : d->I));
  p->off_y = o;      o = align256(o + 4 * slots * d->H);
  p->total = o;
  return true;
}

}  // namespace few
}  // namespace moe

extern "C" size_t moe_layer_few_workspace_bytes(const moe_few_desc_t* d) {
  moe::few::FewPlan p;
  return moe::few::plan_few(d, &p) ? p.total : 0;
}

static moe_status_t layer_few_impl(const moe_few_desc_t* d, const moe_few_weights_t* w, const uint16_t* x,
                                   const float* logits, const int32_t* num_tokens, int32_t* topk_idx, float* topk_w,
                                   uint16_t* out, void* ws, size_t ws_bytes, int32_t* dev_status,
                                   unsigned long long limit_ns, void* stream) {
  using namespace moe;
  using namespace moe::few;
  FewPlan p;
  if (!plan_few(d, &p) || !w) return MOE_ERR_ARG;
  if (!ws || ws_bytes < p.total) return MOE_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) & 255) return MOE_ERR_ARG;
  if (d->T == 0) return MOE_OK;
  if (!x || !topk_idx || !topk_w || !out || !w->w13 || !w->w2) return MOE_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(out) & 7) return MOE_ERR_ARG;
  if (w->w_router && logits) return MOE_ERR_ARG;          // one source of the routing
  if (d->dtype == MOE_E4M3 && (!w->w13_scales || !w->w2_scales)) return MOE_ERR_ARG;
  if (d->has_shared) {
    if (!w->shared_w13 || !w->shared_w2) return MOE_ERR_ARG;
    if (d->dtype == MOE_E4M3 && (!w->shared_w13_scales || !w->shared_w2_scales)) return MOE_ERR_ARG;
  }
  const void* al[] = {x, w->w_router, w->w13, w->w2, d->has_shared ? w->shared_w13 : nullptr,
                      d->has_shared ? w->shared_w2 : nullptr};
  for (const void* q : al)
    if (reinterpret_cast<uintptr_t>(q) & 15) return MOE_ERR_ARG;
  // weight coordinates are int32: rows, or lines of 128 bytes for tiled weights
  const long long wide = d->H > 2 * d->I ? d->H : 2 * d->I;
  const long long bytes_per = d->dtype == MOE_BF16 ? 2 : 1;
  if ((d->weight_tiles ? 2ll * d->I * d->H * bytes_per / 128 : wide) * d->E > 0x7fffffffll) return MOE_ERR_ARG;
  uint8_t* b = static_cast<uint8_t*>(ws);
  LayerArgs a;
  a.T = d->T; a.H = d->H; a.I = d->I; a.E = d->E; a.K = d->K;
  a.shared = d->has_shared;
  a.tiled = d->weight_tiles;
  a.zeros = d->zeros;
  const void* wp[4] = {w->w13, w->w2, w->shared_w13, w->shared_w2};
  const float* sp[4] = {w->w13_scales, w->w2_scales, w->shared_w13_scales, w->shared_w2_scales};
  for (int i = 0; i < 4; ++i) {
    const bool used = i < 2 || d->has_shared;
    a.w[i] = used ? static_cast<const uint8_t*>(wp[i]) : nullptr;
    a.scales[i] = used ? sp[i] : nullptr;
    if (used && d->dtype != MOE_W4) {
      const uint64_t rows = (uint64_t)(i % 2 ? d->H : 2 * d->I) * (i < 2 ? d->E : 1);
      const uint64_t bytes = (uint64_t)(i % 2 ? d->I : d->H) * bytes_per;
      const bool ok = d->weight_tiles ? gg::make_map(&a.map[i], wp[i], true, 128, rows * bytes / 128, 16)
                                      : gg::make_map(&a.map[i], wp[i], true, bytes, rows, 16);
      if (!ok) return MOE_ERR_CUDA;
    }
  }
  a.w_router = w->w_router;
  a.router_bias = w->router_bias;
  a.logits_in = logits;
  a.num_tokens = num_tokens;
  a.logits = reinterpret_cast<float*>(b + p.off_logits);
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.x = x;
  a.out = out;
  a.dev_status = dev_status;
  a.limit_ns = limit_ns;
  a.ctl = reinterpret_cast<uint32_t*>(b);
  a.tile_count = reinterpret_cast<int32_t*>(b + p.off_tile);
  a.entry_done = reinterpret_cast<int32_t*>(b + p.off_entry);
  a.h_top = reinterpret_cast<int32_t*>(b + p.off_htop);
  a.x16 = reinterpret_cast<uint16_t*>(b + p.off_x16);
  a.x_unit = reinterpret_cast<float*>(b + p.off_xunit);
  a.h_exp = b + p.off_hexp;
  a.h_hi = reinterpret_cast<uint16_t*>(b + p.off_hhi);
  a.h_lo = (int)((p.off_hlo - p.off_hhi) / 2);
  a.y = reinterpret_cast<float*>(b + p.off_y);
  cudaStream_t st = as_stream(stream);
  const cudaError_t e = d->dtype == MOE_BF16   ? launch_layer_bf16(a, st)
                        : d->dtype == MOE_E4M3 ? launch_layer_e4m3(a, st)
                                               : launch_layer_w4(a, d->group, st);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

extern "C" moe_status_t moe_layer_few(const moe_few_desc_t* d, const moe_few_weights_t* w, const uint16_t* x,
                                      const float* logits, const int32_t* num_tokens, int32_t* topk_idx,
                                      float* topk_w, uint16_t* out, void* ws, size_t ws_bytes, int32_t* dev_status,
                                      void* stream) {
  return layer_few_impl(d, w, x, logits, num_tokens, topk_idx, topk_w, out, ws, ws_bytes, dev_status,
                        moe::few::TIMEOUT_NS, stream);
}

// Test hook, deliberately absent from the public header: moe_layer_few with the limit of each wait in
// nanoseconds instead of the built-in 2 s, so that a test can make a wait run out.
extern "C" moe_status_t moe_testing_layer_few_wait_limit(const moe_few_desc_t* d, const moe_few_weights_t* w,
                                                         const uint16_t* x, const float* logits,
                                                         const int32_t* num_tokens, int32_t* topk_idx, float* topk_w,
                                                         uint16_t* out, void* ws, size_t ws_bytes, int32_t* dev_status,
                                                         unsigned long long limit_ns, void* stream) {
  return layer_few_impl(d, w, x, logits, num_tokens, topk_idx, topk_w, out, ws, ws_bytes, dev_status, limit_ns, stream);
}
