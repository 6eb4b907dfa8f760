// hlq_clip.cu -- the global norm of many gradients and their clipping
// (hlq_clip_grad_norm): norm = sqrt(sum over all elements of g^2),
// coef = min(1, max_norm / (norm + 1e-6)), out = coef g.
//
// The tensors' table travels as a kernel parameter: nothing is copied to the
// device beforehand, and a captured call replays with the addresses it was
// captured with.
#include "hlq_device.cuh"
#include "hlq_kernels.h"

namespace hlq {
namespace {

constexpr int kClipThreads = 256;

__device__ __forceinline__ double cta_sum_f64(double v, double* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  double s = 0.0;
  for (int i = 0; i < kClipThreads / 32; ++i) s += red[i];
  return s;
}

// The tensor that holds chunk `k` of the concatenation: the last one whose
// first chunk is <= k (tensors without elements have no chunk).
__device__ __forceinline__ int tensor_of(const ClipTable& tab, int64_t k) {
  int lo = 0, hi = tab.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= k)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kClipThreads)
    clip_norm_kernel(const __grid_constant__ ClipTable tab, double* part) {
  __shared__ double red[32];
  double acc = 0.0;
  for (int64_t k = blockIdx.x; k < tab.chunks; k += gridDim.x) {
    const int i = tensor_of(tab, k);
    const int64_t e0 = (k - tab.first[i]) * kClipChunk;
    const int64_t n = min((int64_t)kClipChunk, tab.numel[i] - e0);
    for (int64_t e = threadIdx.x; e < n; e += kClipThreads) {
      const double g = (tab.flags[i] & kClipInBf16)
                           ? __bfloat162float(static_cast<const __nv_bfloat16*>(tab.in[i])[e0 + e])
                           : static_cast<const float*>(tab.in[i])[e0 + e];
      acc += g * g;
    }
  }
  acc = cta_sum_f64(acc, red);
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

__global__ void __launch_bounds__(kClipThreads)
    clip_coef_kernel(const double* part, int n_part, float max_norm, float* norm_coef,
                     unsigned int* status) {
  __shared__ double red[32];
  double s = 0.0;
  for (int i = threadIdx.x; i < n_part; i += kClipThreads) s += part[i];
  s = cta_sum_f64(s, red);
  if (threadIdx.x == 0) {
    const float norm = (float)sqrt(s);
    const float c = max_norm / (norm + 1e-6f);
    norm_coef[0] = norm;
    norm_coef[1] = c > 1.f ? 1.f : c;  // a NaN stays
    if (!isfinite(norm)) raise_flag(status, HLQ_DEV_NONFINITE);
  }
}

__global__ void __launch_bounds__(kClipThreads)
    clip_scale_kernel(const __grid_constant__ ClipTable tab, const float* norm_coef) {
  const float coef = norm_coef[1];
  for (int64_t k = blockIdx.x; k < tab.chunks; k += gridDim.x) {
    const int i = tensor_of(tab, k);
    const int64_t e0 = (k - tab.first[i]) * kClipChunk;
    const int64_t n = min((int64_t)kClipChunk, tab.numel[i] - e0);
    for (int64_t e = threadIdx.x; e < n; e += kClipThreads) {
      const float g = (tab.flags[i] & kClipInBf16)
                          ? __bfloat162float(static_cast<const __nv_bfloat16*>(tab.in[i])[e0 + e])
                          : static_cast<const float*>(tab.in[i])[e0 + e];
      if (tab.flags[i] & kClipOutBf16)
        static_cast<__nv_bfloat16*>(tab.out[i])[e0 + e] = __float2bfloat16_rn(coef * g);
      else
        static_cast<float*>(tab.out[i])[e0 + e] = coef * g;
    }
  }
}

}  // namespace

int clip_norm_grid(int64_t chunks, int sms) {
  const int64_t most = (int64_t)sms * 4;
  return (int)(chunks < 1 ? 1 : chunks < most ? chunks : most);
}

cudaError_t launch_clip_norm(const ClipTable& tab, double* part, int grid, cudaStream_t st) {
  clip_norm_kernel<<<grid, kClipThreads, 0, st>>>(tab, part);
  return cudaGetLastError();
}

cudaError_t launch_clip_coef(const double* part, int n_part, float max_norm, float* norm_coef,
                             unsigned int* status, cudaStream_t st) {
  clip_coef_kernel<<<1, kClipThreads, 0, st>>>(part, n_part, max_norm, norm_coef, status);
  return cudaGetLastError();
}

cudaError_t launch_clip_scale(const ClipTable& tab, const float* norm_coef, int grid,
                              cudaStream_t st) {
  clip_scale_kernel<<<grid, kClipThreads, 0, st>>>(tab, norm_coef);
  return cudaGetLastError();
}

}  // namespace hlq
