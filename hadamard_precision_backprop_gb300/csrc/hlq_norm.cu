// hlq_norm.cu -- layer norm, forward and backward (hlq_layer_norm,
// hlq_layer_norm_backward).
//
// Forward, per row t of h = x (+ residual), sums in fp32:
//   mean = sum_c h / C,  var = sum_c (h - mean)^2 / C,
//   rstd = 1 / sqrt(var + eps),  y = (h - mean) rstd w + b.
// Backward, with a = g_y w and xhat = (x - mean) rstd:
//   g_x = rstd (a - mean_c(a) - xhat mean_c(a xhat)) (+ g_residual),
//   g_w = sum_t g_y xhat,  g_b = sum_t g_y.
#include "hlq_device.cuh"
#include "hlq_kernels.h"

namespace hlq {
namespace {

__device__ __forceinline__ float load_elem(const void* p, bool bf16, int64_t i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
              : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_elem(void* p, bool bf16, int64_t i, float v) {
  if (bf16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p)[i] = v;
}

constexpr int kRowThreads = 256;

// Sum over the CTA, the same value in every thread; `red` holds one float a warp.
__device__ __forceinline__ float cta_sum(float v, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // `red` may still be read by the sum before
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < warps ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(kRowThreads) norm_fwd_kernel(NormFwd p) {
  __shared__ float red[32];
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    auto h_at = [&](int64_t c) {
      float v = load_elem(p.x, p.x_bf16, t * p.ldx + c);
      if (p.residual) v += load_elem(p.residual, p.x_bf16, t * p.ldr + c);
      return v;
    };
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < p.C; c += kRowThreads) s += h_at(c);
    const float mean = cta_sum(s, red) / (float)p.C;
    s = 0.f;
    for (int64_t c = threadIdx.x; c < p.C; c += kRowThreads) {
      const float d = h_at(c) - mean;
      s += d * d;
    }
    const float rstd = 1.f / sqrtf(cta_sum(s, red) / (float)p.C + p.eps);
    for (int64_t c = threadIdx.x; c < p.C; c += kRowThreads) {
      const float h = h_at(c);
      const float w = p.weight ? load_elem(p.weight, p.w_bf16, c) : 1.f;
      const float b = p.bias ? load_elem(p.bias, p.w_bf16, c) : 0.f;
      if (p.h) store_elem(p.h, p.x_bf16, t * p.ldh + c, h);
      store_elem(p.y, p.y_bf16, t * p.ldy + c, (h - mean) * rstd * w + b);
    }
    if (threadIdx.x == 0) {
      if (p.mean) {
        p.mean[t] = mean;
        p.rstd[t] = rstd;
      }
      if (!isfinite(mean) || !isfinite(rstd)) raise_flag(p.status, HLQ_DEV_NONFINITE);
    }
  }
}

__global__ void __launch_bounds__(kRowThreads) norm_bwd_x_kernel(NormBwd p) {
  __shared__ float red[32];
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const float mean = p.mean[t], rstd = p.rstd[t];
    float sa = 0.f, sx = 0.f;
    for (int64_t c = threadIdx.x; c < p.C; c += kRowThreads) {
      const float w = p.weight ? load_elem(p.weight, p.w_bf16, c) : 1.f;
      const float a = load_elem(p.gy, p.gy_bf16, t * p.ldgy + c) * w;
      sa += a;
      sx += a * ((load_elem(p.x, p.x_bf16, t * p.ldx + c) - mean) * rstd);
    }
    sa = cta_sum(sa, red) / (float)p.C;
    sx = cta_sum(sx, red) / (float)p.C;
    for (int64_t c = threadIdx.x; c < p.C; c += kRowThreads) {
      const float w = p.weight ? load_elem(p.weight, p.w_bf16, c) : 1.f;
      const float a = load_elem(p.gy, p.gy_bf16, t * p.ldgy + c) * w;
      const float xhat = (load_elem(p.x, p.x_bf16, t * p.ldx + c) - mean) * rstd;
      float g = rstd * (a - sa - xhat * sx);
      if (p.gres) g += load_elem(p.gres, p.gx_bf16, t * p.ldgr + c);
      store_elem(p.gx, p.gx_bf16, t * p.ldgx + c, g);
    }
    if (threadIdx.x == 0 && (!isfinite(sa) || !isfinite(sx)))
      raise_flag(p.status, HLQ_DEV_NONFINITE);
  }
}

// Per-column sums over the rows of one slab: part[slab][0 / 1][c].
__global__ void __launch_bounds__(kRowThreads) norm_bwd_cols_kernel(NormBwd p) {
  const int64_t c = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (c >= p.C) return;
  const int64_t t0 = p.T * blockIdx.y / gridDim.y, t1 = p.T * (blockIdx.y + 1) / gridDim.y;
  float gw = 0.f, gb = 0.f;
  for (int64_t t = t0; t < t1; ++t) {
    const float g = load_elem(p.gy, p.gy_bf16, t * p.ldgy + c);
    gw += g * ((load_elem(p.x, p.x_bf16, t * p.ldx + c) - p.mean[t]) * p.rstd[t]);
    gb += g;
  }
  p.part[(blockIdx.y * 2 + 0) * p.C + c] = gw;
  p.part[(blockIdx.y * 2 + 1) * p.C + c] = gb;
}

__global__ void __launch_bounds__(kRowThreads) norm_bwd_join_kernel(NormBwd p, int slabs) {
  const int64_t c = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (c >= p.C) return;
  float gw = 0.f, gb = 0.f;
  for (int s = 0; s < slabs; ++s) {
    gw += p.part[(s * 2 + 0) * p.C + c];
    gb += p.part[(s * 2 + 1) * p.C + c];
  }
  if (p.gweight) p.gweight[c] = gw;
  if (p.gbias) p.gbias[c] = gb;
}

}  // namespace

int norm_bwd_slabs(int64_t T) { return (int)(T < 128 ? (T < 1 ? 1 : T) : 128); }

cudaError_t launch_norm_fwd(const NormFwd& p, cudaStream_t st) {
  norm_fwd_kernel<<<(unsigned)(p.T < 65535 ? p.T : 65535), kRowThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_norm_bwd_x(const NormBwd& p, cudaStream_t st) {
  norm_bwd_x_kernel<<<(unsigned)(p.T < 65535 ? p.T : 65535), kRowThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_norm_bwd_cols(const NormBwd& p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.C + kRowThreads - 1) / kRowThreads), norm_bwd_slabs(p.T));
  norm_bwd_cols_kernel<<<grid, kRowThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_norm_bwd_join(const NormBwd& p, cudaStream_t st) {
  norm_bwd_join_kernel<<<(unsigned)((p.C + kRowThreads - 1) / kRowThreads), kRowThreads, 0, st>>>(
      p, norm_bwd_slabs(p.T));
  return cudaGetLastError();
}

}  // namespace hlq
