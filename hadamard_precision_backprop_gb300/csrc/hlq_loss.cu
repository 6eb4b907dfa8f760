// hlq_loss.cu -- log-probabilities of given tokens and the clipped policy loss
// with the gradient of the logits (hlq_token_logprobs, hlq_policy_loss).
//
// z = scale * logits; per row t with token a:  lp = z_a - lse(z).
// Policy loss, per row with weight w_t != 0:
//   r = exp(lp - old),  pg = -min(r A, clip(r, 1 - low, 1 + high) A),
//   d = ref - lp,  kl = exp(d) - d - 1,
//   loss = sum_t w_t (pg + beta kl),
//   dl/dlp = -r A [the unclipped branch holds] + beta (1 - exp(d)),
//   g[t, v] = grad_scale w_t dl/dlp scale ([v == a] - p_v).
#include "hlq_device.cuh"
#include "hlq_kernels.h"

namespace hlq {
namespace {

constexpr int kLossThreads = 256;

__device__ __forceinline__ float load_logit(const void* p, bool bf16, int64_t i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
              : static_cast<const float*>(p)[i];
}

// Maximum of the row's logits (NaN where one is NaN) and the sum of
// exp(scale (logit - maximum)), the same in every thread.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ MaxSum row_max_sum(const void* logits, bool bf16, int64_t row, int64_t V, float scale,
                              float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float m = -INFINITY;
  for (int64_t v = threadIdx.x; v < V; v += kLossThreads)
    m = nan_max(m, load_logit(logits, bf16, row + v));
  for (int o = 16; o > 0; o >>= 1) m = nan_max(m, __shfl_xor_sync(0xffffffffu, m, o));
  __syncthreads();
  if (lane == 0) red[warp] = m;
  __syncthreads();
  for (int i = 0; i < kLossThreads / 32; ++i) m = nan_max(m, red[i]);
  float s = 0.f;
  for (int64_t v = threadIdx.x; v < V; v += kLossThreads)
    s += expf(scale * (load_logit(logits, bf16, row + v) - m));
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if (lane == 0) red[warp] = s;
  __syncthreads();
  s = 0.f;
  for (int i = 0; i < kLossThreads / 32; ++i) s += red[i];
  return {m, s};
}

__global__ void __launch_bounds__(kLossThreads) token_logprobs_kernel(TokenLogprobs p) {
  __shared__ float red[32];
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const MaxSum ms = row_max_sum(p.logits, p.bf16, t * p.ld, p.V, p.scale, red);
    if (threadIdx.x == 0) {
      const int64_t a = p.targets[t];
      const float ls = logf(ms.s);
      float lp = NAN;
      if (a >= 0 && a < p.V)
        lp = p.scale * (load_logit(p.logits, p.bf16, t * p.ld + a) - ms.m) - ls;
      else
        raise_flag(p.status, HLQ_DEV_BADCODE);
      p.logp[t] = lp;
      if (p.lse) p.lse[t] = p.scale * ms.m + ls;
      if (isnan(ls)) raise_flag(p.status, HLQ_DEV_NONFINITE);
    }
  }
}

__global__ void __launch_bounds__(kLossThreads) policy_rows_kernel(PolicyLoss p) {
  __shared__ float red[32];
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const float w = p.weight[t];
    float coef = 0.f, lp = 0.f;
    MaxSum ms = {0.f, 1.f};
    int64_t a = -1;
    if (w != 0.f) {
      ms = row_max_sum(p.logits, p.bf16, t * p.ld, p.V, p.scale, red);
      a = p.actions[t];
      const bool known = a >= 0 && a < p.V;
      lp = known ? p.scale * (load_logit(p.logits, p.bf16, t * p.ld + a) - ms.m) - logf(ms.s)
                 : NAN;
      const float adv = p.advantage[t], r = expf(lp - p.old_logp[t]);
      const float inner = r * adv;
      const float outer = fminf(fmaxf(r, 1.f - p.clip_low), 1.f + p.clip_high) * adv;
      const bool clipped = outer < inner;
      const float pg = clipped ? -outer : -inner;
      float dlp = clipped ? 0.f : -inner, kl = 0.f;
      if (p.ref_logp) {
        const float d = p.ref_logp[t] - lp, e = expm1f(d);
        kl = e - d;
        if (p.kl_coef != 0.f) dlp -= p.kl_coef * e;
      }
      coef = w * dlp * p.grad_scale * p.scale;
      if (threadIdx.x == 0) {
        p.part[t] = w * pg;
        p.part[p.T + t] = w * kl;
        p.part[2 * p.T + t] = clipped ? w : 0.f;
        if (!known) raise_flag(p.status, HLQ_DEV_BADCODE);
        if (!isfinite(coef)) raise_flag(p.status, HLQ_DEV_NONFINITE);
      }
    } else if (threadIdx.x == 0) {
      p.part[t] = p.part[p.T + t] = p.part[2 * p.T + t] = 0.f;
    }
    if (threadIdx.x == 0 && p.logp) p.logp[t] = lp;
    if (!p.g) continue;
    const float inv = 1.f / ms.s;
    __syncthreads();  // the gradient may replace the logits: lp is read above
    for (int64_t v = threadIdx.x; v < p.V; v += kLossThreads) {
      float g = 0.f;
      if (w != 0.f) {
        const float pv = expf(p.scale * (load_logit(p.logits, p.bf16, t * p.ld + v) - ms.m)) * inv;
        g = v == a ? -coef * expm1f(lp) : -coef * pv;
      }
      if (p.bf16)
        static_cast<__nv_bfloat16*>(p.g)[t * p.ldg + v] = __float2bfloat16_rn(g);
      else
        static_cast<float*>(p.g)[t * p.ldg + v] = g;
    }
  }
}

// stats = sums over the rows in a fixed order, in fp64.
__global__ void __launch_bounds__(kLossThreads) policy_stats_kernel(PolicyLoss p) {
  __shared__ double red[3][kLossThreads];
  for (int k = 0; k < 3; ++k) {
    double s = 0.0;
    for (int64_t t = threadIdx.x; t < p.T; t += kLossThreads) s += p.part[k * p.T + t];
    red[k][threadIdx.x] = s;
  }
  for (int o = kLossThreads / 2; o > 0; o >>= 1) {
    __syncthreads();
    if ((int)threadIdx.x < o)
      for (int k = 0; k < 3; ++k) red[k][threadIdx.x] += red[k][threadIdx.x + o];
  }
  if (threadIdx.x == 0) {
    const double pg = red[0][0], kl = red[1][0];
    p.stats[0] = (float)(p.ref_logp && p.kl_coef != 0.f ? pg + (double)p.kl_coef * kl : pg);
    p.stats[1] = (float)pg;
    p.stats[2] = (float)kl;
    p.stats[3] = (float)red[2][0];
  }
}

}  // namespace

cudaError_t launch_token_logprobs(const TokenLogprobs& p, cudaStream_t st) {
  token_logprobs_kernel<<<(unsigned)(p.T < 65535 ? p.T : 65535), kLossThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_policy_rows(const PolicyLoss& p, cudaStream_t st) {
  policy_rows_kernel<<<(unsigned)(p.T < 65535 ? p.T : 65535), kLossThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_policy_stats(const PolicyLoss& p, cudaStream_t st) {
  policy_stats_kernel<<<1, kLossThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace hlq
