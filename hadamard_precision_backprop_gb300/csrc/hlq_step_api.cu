// hlq_step_api.cu -- the C ABI of the operators around the layer in a
// training step (declared in include/hlq.h): argument validation and the
// launch sequence of each.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "hlq.h"
#include "hlq_host.h"
#include "hlq_kernels.h"

namespace hlq {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 31;  // rows, and columns, of one call
constexpr int64_t kMaxStride = (int64_t)1 << 40;

bool dtype_ok(int dt) { return dt == HLQ_F32 || dt == HLQ_BF16; }
size_t elem_bytes(int dt) { return dt == HLQ_BF16 ? 2 : 4; }
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Rows of `cols` elements, `ld` apart.  An input may repeat one row (ld 0).
bool stride_ok(int64_t ld, int64_t rows, int64_t cols, bool input) {
  if (rows <= 1) return true;
  return (ld >= cols && ld <= kMaxStride) || (input && ld == 0);
}

hlq_status check_rows(int64_t T, int64_t C) {
  if (T < 0 || C < 1) return HLQ_ERR_SHAPE;
  if (T >= kMaxRows || C >= kMaxRows) return HLQ_ERR_UNSUPPORTED;
  return HLQ_OK;
}

size_t norm_bwd_ws(int64_t T, int64_t C) {
  return align_up((size_t)norm_bwd_most_slabs(T) * 2 * (size_t)C * 4);
}

size_t policy_ws(int64_t T) { return align_up((size_t)(T > 0 ? T : 1) * 3 * 4); }

// Partial sums of a clipping call: every CTA that scales adds them all, so
// they are few, and each launch over up to kClipTensors tensors gets its share.
constexpr int64_t kClipParts = 4096;
int64_t clip_launches(int64_t n) { return n > 0 ? (n + kClipTensors - 1) / kClipTensors : 1; }
size_t clip_ws(int64_t n) {
  const int64_t parts = 1024 * clip_launches(n);
  return (size_t)(parts < kClipParts ? parts : kClipParts) * sizeof(float);
}

}  // namespace
}  // namespace hlq

using namespace hlq;

extern "C" {

hlq_status hlq_layer_norm(const void* d_x, int64_t ldx, const void* d_residual, int64_t ldr,
                          int x_dt, const void* d_weight, const void* d_bias, int w_dt,
                          int64_t T, int64_t C, float eps, void* d_y, int64_t ldy, int y_dt,
                          void* d_h, int64_t ldh, float* d_mean, float* d_rstd, void* stream) {
  if (!dtype_ok(x_dt) || !dtype_ok(w_dt) || !dtype_ok(y_dt)) return HLQ_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || std::isinf(eps)) return HLQ_ERR_INVALID_ARG;
  hlq_status st = check_rows(T, C);
  if (st != HLQ_OK) return st;
  if (!d_residual != !d_h || !d_mean != !d_rstd) return HLQ_ERR_INVALID_ARG;
  if (T > 0 && (!d_x || !d_y)) return HLQ_ERR_INVALID_ARG;
  if (!stride_ok(ldx, T, C, true) || !stride_ok(ldy, T, C, false) ||
      (d_residual && (!stride_ok(ldr, T, C, true) || !stride_ok(ldh, T, C, false))))
    return HLQ_ERR_SHAPE;
  if (!aligned_to(d_x, elem_bytes(x_dt)) || !aligned_to(d_residual, elem_bytes(x_dt)) ||
      !aligned_to(d_h, elem_bytes(x_dt)) || !aligned_to(d_y, elem_bytes(y_dt)) ||
      !aligned_to(d_weight, elem_bytes(w_dt)) || !aligned_to(d_bias, elem_bytes(w_dt)) ||
      !aligned_to(d_mean, 4) || !aligned_to(d_rstd, 4))
    return HLQ_ERR_ALIGN;
  if (T == 0) return HLQ_OK;
  NormFwd p{};
  p.x = d_x; p.residual = d_residual; p.weight = d_weight; p.bias = d_bias;
  p.y = d_y; p.h = d_h; p.mean = d_mean; p.rstd = d_rstd;
  p.ldx = ldx; p.ldr = ldr; p.ldy = ldy; p.ldh = ldh; p.T = T; p.C = C;
  p.eps = eps;
  p.x_bf16 = x_dt == HLQ_BF16; p.w_bf16 = w_dt == HLQ_BF16; p.y_bf16 = y_dt == HLQ_BF16;
  p.status = device_status_ptr();
  if (!p.status) return HLQ_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  HLQ_LAUNCH("norm_fwd", s, launch_norm_fwd(p, s));
  return HLQ_OK;
}

size_t hlq_layer_norm_backward_workspace_bytes(int64_t T, int64_t C) {
  return check_rows(T, C) == HLQ_OK ? norm_bwd_ws(T, C) : 0;
}

hlq_status hlq_layer_norm_backward(const void* d_gy, int64_t ldgy, int gy_dt, const void* d_x,
                                   int64_t ldx, int x_dt, const float* d_mean,
                                   const float* d_rstd, const void* d_weight, int w_dt,
                                   const void* d_gres, int64_t ldgr, int64_t T, int64_t C,
                                   void* d_gx, int64_t ldgx, int gx_dt, float* d_gweight,
                                   float* d_gbias, void* d_ws, size_t ws_bytes, void* stream) {
  if (!dtype_ok(gy_dt) || !dtype_ok(x_dt) || !dtype_ok(w_dt) || !dtype_ok(gx_dt))
    return HLQ_ERR_INVALID_ARG;
  hlq_status st = check_rows(T, C);
  if (st != HLQ_OK) return st;
  if (T > 0 && (!d_gy || !d_x || !d_mean || !d_rstd || !d_gx)) return HLQ_ERR_INVALID_ARG;
  if (!stride_ok(ldgy, T, C, true) || !stride_ok(ldx, T, C, true) ||
      !stride_ok(ldgx, T, C, false) || (d_gres && !stride_ok(ldgr, T, C, true)))
    return HLQ_ERR_SHAPE;
  if (!aligned_to(d_gy, elem_bytes(gy_dt)) || !aligned_to(d_x, elem_bytes(x_dt)) ||
      !aligned_to(d_gx, elem_bytes(gx_dt)) || !aligned_to(d_gres, elem_bytes(gx_dt)) ||
      !aligned_to(d_weight, elem_bytes(w_dt)) || !aligned_to(d_mean, 4) ||
      !aligned_to(d_rstd, 4) || !aligned_to(d_gweight, 4) || !aligned_to(d_gbias, 4))
    return HLQ_ERR_ALIGN;
  const bool cols = d_gweight || d_gbias;
  if (cols && T > 0) {
    if (!d_ws || ws_bytes < norm_bwd_ws(T, C)) return HLQ_ERR_WORKSPACE;
    if (!aligned256(d_ws)) return HLQ_ERR_ALIGN;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // empty sums
    if (d_gweight) HLQ_TRY(cudaMemsetAsync(d_gweight, 0, (size_t)C * 4, s));
    if (d_gbias) HLQ_TRY(cudaMemsetAsync(d_gbias, 0, (size_t)C * 4, s));
    return HLQ_OK;
  }
  NormBwd p{};
  p.gy = d_gy; p.x = d_x; p.weight = d_weight; p.gres = d_gres;
  p.mean = d_mean; p.rstd = d_rstd; p.gx = d_gx; p.gweight = d_gweight; p.gbias = d_gbias;
  p.part = cols ? static_cast<float*>(d_ws) : nullptr;
  p.ldgy = ldgy; p.ldx = ldx; p.ldgr = ldgr; p.ldgx = ldgx; p.T = T; p.C = C;
  p.gy_bf16 = gy_dt == HLQ_BF16; p.x_bf16 = x_dt == HLQ_BF16; p.w_bf16 = w_dt == HLQ_BF16;
  p.gx_bf16 = gx_dt == HLQ_BF16;
  p.status = device_status_ptr();
  if (!p.status) return HLQ_ERR_CUDA;
  int slabs = 0;
  HLQ_LAUNCH("norm_bwd", s, launch_norm_bwd(p, &slabs, s));
  if (slabs > 0 && cols) HLQ_LAUNCH("norm_bwd_join", s, launch_norm_bwd_join(p, slabs, s));
  return HLQ_OK;
}

hlq_status hlq_token_logprobs(const void* d_logits, int64_t ld, int dt, const int64_t* d_targets,
                              int64_t T, int64_t V, float scale, float* d_logp, float* d_lse,
                              void* stream) {
  if (!dtype_ok(dt) || !(scale > 0.f) || std::isinf(scale)) return HLQ_ERR_INVALID_ARG;
  hlq_status st = check_rows(T, V);
  if (st != HLQ_OK) return st;
  if (T > loss_most_rows(V)) return HLQ_ERR_UNSUPPORTED;
  if (T > 0 && (!d_logits || !d_targets || !d_logp)) return HLQ_ERR_INVALID_ARG;
  if (!stride_ok(ld, T, V, true)) return HLQ_ERR_SHAPE;
  if (!aligned_to(d_logits, elem_bytes(dt)) || !aligned_to(d_targets, 8) ||
      !aligned_to(d_logp, 4) || !aligned_to(d_lse, 4))
    return HLQ_ERR_ALIGN;
  if (T == 0) return HLQ_OK;
  TokenLogprobs p{};
  p.logits = d_logits; p.targets = d_targets; p.logp = d_logp; p.lse = d_lse;
  p.ld = ld; p.T = T; p.V = V; p.scale = scale; p.bf16 = dt == HLQ_BF16;
  p.status = device_status_ptr();
  if (!p.status) return HLQ_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  HLQ_LAUNCH("token_logprobs", s, launch_token_logprobs(p, s));
  return HLQ_OK;
}

size_t hlq_policy_loss_workspace_bytes(int64_t T, int64_t V) {
  return check_rows(T, V) == HLQ_OK ? policy_ws(T) : 0;
}

hlq_status hlq_policy_loss(const void* d_logits, int64_t ld, int dt, const int64_t* d_actions,
                           const float* d_old_logp, const float* d_ref_logp,
                           const float* d_advantage, const float* d_weight, int64_t T, int64_t V,
                           float scale, float clip_low, float clip_high, float kl_coef,
                           float grad_scale, float* d_stats, float* d_logp, void* d_g,
                           int64_t ldg, void* d_ws, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dt) || !(scale > 0.f) || std::isinf(scale)) return HLQ_ERR_INVALID_ARG;
  if (!(clip_low >= 0.f) || !(clip_high >= 0.f) || !std::isfinite(kl_coef) ||
      !std::isfinite(grad_scale))
    return HLQ_ERR_INVALID_ARG;
  hlq_status st = check_rows(T, V);
  if (st != HLQ_OK) return st;
  if (T > loss_most_rows(V)) return HLQ_ERR_UNSUPPORTED;
  if (!d_stats) return HLQ_ERR_INVALID_ARG;
  if (T > 0 && (!d_logits || !d_actions || !d_old_logp || !d_advantage || !d_weight))
    return HLQ_ERR_INVALID_ARG;
  if (!stride_ok(ld, T, V, true) || (d_g && !stride_ok(ldg, T, V, false))) return HLQ_ERR_SHAPE;
  if (!aligned_to(d_logits, elem_bytes(dt)) || !aligned_to(d_g, elem_bytes(dt)) ||
      !aligned_to(d_actions, 8) || !aligned_to(d_old_logp, 4) || !aligned_to(d_ref_logp, 4) ||
      !aligned_to(d_advantage, 4) || !aligned_to(d_weight, 4) || !aligned_to(d_stats, 4) ||
      !aligned_to(d_logp, 4))
    return HLQ_ERR_ALIGN;
  if (T > 0) {
    if (!d_ws || ws_bytes < policy_ws(T)) return HLQ_ERR_WORKSPACE;
    if (!aligned256(d_ws)) return HLQ_ERR_ALIGN;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // empty sums
    HLQ_TRY(cudaMemsetAsync(d_stats, 0, 16, s));
    return HLQ_OK;
  }
  PolicyLoss p{};
  p.logits = d_logits; p.actions = d_actions; p.old_logp = d_old_logp; p.ref_logp = d_ref_logp;
  p.advantage = d_advantage; p.weight = d_weight; p.stats = d_stats; p.logp = d_logp; p.g = d_g;
  p.part = static_cast<float*>(d_ws);
  p.ld = ld; p.ldg = ldg; p.T = T; p.V = V;
  p.scale = scale; p.clip_low = clip_low; p.clip_high = clip_high; p.kl_coef = kl_coef;
  p.grad_scale = grad_scale;
  p.bf16 = dt == HLQ_BF16;
  p.status = device_status_ptr();
  if (!p.status) return HLQ_ERR_CUDA;
  HLQ_LAUNCH("policy_rows", s, launch_policy_rows(p, s));
  HLQ_LAUNCH("policy_stats", s, launch_policy_stats(p, s));
  return HLQ_OK;
}

size_t hlq_clip_grad_norm_workspace_bytes(int64_t n) { return n >= 0 ? clip_ws(n) : 0; }

hlq_status hlq_clip_grad_norm(int64_t n, const void* const* h_grads, const int32_t* h_grad_dts,
                              void* const* h_outs, const int32_t* h_out_dts,
                              const int64_t* h_numels, float max_norm, float* d_norm_coef,
                              void* d_ws, size_t ws_bytes, void* stream) {
  if (n < 0 || !(max_norm >= 0.f) || !d_norm_coef) return HLQ_ERR_INVALID_ARG;
  if (clip_launches(n) > kClipParts) return HLQ_ERR_UNSUPPORTED;
  if (n > 0 && (!h_grads || !h_grad_dts || !h_numels)) return HLQ_ERR_INVALID_ARG;
  if (n > 0 && h_outs && !h_out_dts) return HLQ_ERR_INVALID_ARG;
  if (!aligned_to(d_norm_coef, 4)) return HLQ_ERR_ALIGN;
  for (int64_t i = 0; i < n; ++i) {
    if (h_numels[i] < 0) return HLQ_ERR_SHAPE;
    if (h_numels[i] > kMaxStride) return HLQ_ERR_UNSUPPORTED;
    if (!dtype_ok(h_grad_dts[i]) || (h_outs && !dtype_ok(h_out_dts[i])))
      return HLQ_ERR_INVALID_ARG;
    if (h_numels[i] > 0 && (!h_grads[i] || (h_outs && !h_outs[i]))) return HLQ_ERR_INVALID_ARG;
    if (!aligned_to(h_grads[i], elem_bytes(h_grad_dts[i])) ||
        (h_outs && !aligned_to(h_outs[i], elem_bytes(h_out_dts[i]))))
      return HLQ_ERR_ALIGN;
  }
  if (!d_ws || ws_bytes < clip_ws(n)) return HLQ_ERR_WORKSPACE;
  if (!aligned256(d_ws)) return HLQ_ERR_ALIGN;
  unsigned int* status = device_status_ptr();
  const int sms = device_sm_count();
  if (!status || sms <= 0) return HLQ_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* part = static_cast<float*>(d_ws);
  const int64_t parts_each = (int64_t)(clip_ws(n) / sizeof(float)) / clip_launches(n);
  int n_part = 0;
  ClipTable tab;
  // the tensors from i0 on that fill one table; returns the next i0
  auto fill = [&](int64_t i0) {
    tab.n = 0;
    tab.chunks = 0;
    int64_t i = i0;
    for (; i < n && tab.n < kClipTensors; ++i) {
      if (h_numels[i] == 0) continue;
      tab.in[tab.n] = h_grads[i];
      tab.out[tab.n] = h_outs ? h_outs[i] : nullptr;
      tab.numel[tab.n] = h_numels[i];
      tab.first[tab.n] = tab.chunks;
      tab.flags[tab.n] = (unsigned char)((h_grad_dts[i] == HLQ_BF16 ? kClipInBf16 : 0) |
                                         (h_outs && h_out_dts[i] == HLQ_BF16 ? kClipOutBf16 : 0));
      tab.chunks += (h_numels[i] + kClipChunk - 1) / kClipChunk;
      ++tab.n;
    }
    return i;
  };
  for (int64_t i = 0; i < n;) {
    i = fill(i);
    if (tab.n == 0) continue;
    int grid = clip_grid(tab.chunks, sms);
    if (grid > parts_each) grid = (int)parts_each;
    HLQ_LAUNCH("clip_norm", s, launch_clip_norm(tab, part + n_part, grid, s));
    n_part += grid;
  }
  const ClipSums q = {part, n_part, max_norm, d_norm_coef, status};
  if (!h_outs || n_part == 0) {
    HLQ_LAUNCH("clip_coef", s, launch_clip_coef(q, s));
    return HLQ_OK;
  }
  bool first = true;
  for (int64_t i = 0; i < n;) {
    i = fill(i);
    if (tab.n == 0) continue;
    const int grid = clip_grid(tab.chunks, sms);
    HLQ_LAUNCH("clip_scale", s, launch_clip_scale(tab, q, first, grid, s));
    first = false;
  }
  return HLQ_OK;
}

}  // extern "C"
