// hlq_norm_range.cuh -- layer norm rows whose squares leave fp32's range: the
// forward kernels test the sum of squared differences they have, and hand such
// a row to norm_row_again.
#pragma once

#include "hlq_device.cuh"
#include "hlq_kernels.h"
#include "hlq_rows.cuh"

namespace hlq {
namespace {

// Differences above 2^64 have squares that overflow, and elements above 2^97
// may do so in their sum (the differences to that mean are infinite too).
// Differences below 2^-45 have squares that lose bits, which shows where eps is
// not far above them; `least` is 0 for any usual eps.
__device__ __forceinline__ float norm_least(float eps) { return eps < 0x1p-90f ? 0x1p-90f : 0.f; }
__device__ __forceinline__ bool norm_in_range(float squares, float least) {
  return squares >= least && squares < INFINITY;
}

// Such a row is multiplied by a power of two.  With 2^-96 no square overflows in
// sums of up to 2^31 terms, and what vanishes is beneath the last bit of a sum
// that had overflowed; with 2^96 a sum that was below 2^-90 stays below 2^102.
// Rows of infinity or NaN stay what they are.
__device__ __forceinline__ float norm_scale(float mean, float squares) {
  return !(squares < INFINITY) ? 0x1p-96f : fabsf(mean) < 1.f ? 0x1p96f : 1.f;
}
// 1 / standard deviation of the row that was multiplied so (its own is `scale`
// times this).  A row of equal elements goes back to its own mean: it has eps
// alone, which 2^-192 would make vanish.
__device__ __forceinline__ float norm_rstd(float var, float eps, float& mean, float& scale) {
  if (var == 0.f && scale < 1.f) {
    mean *= 0x1p96f;
    scale = 1.f;
  }
  return 1.f / sqrtf(var + eps * scale * scale);
}
__device__ __forceinline__ void write_stats(const NormFwd& p, int64_t t, float mean, float rstd) {
  if (p.mean) {
    p.mean[t] = mean;
    p.rstd[t] = rstd;
  }
  if (!isfinite(mean) || !isfinite(rstd)) raise_flag(p.status, HLQ_DEV_NONFINITE);
}

// Sum over the kTeam consecutive threads of a team, in every one of them; of a
// warp's teams those may call it that need to.
template <int kTeam>
__device__ __forceinline__ float team_total(float v) {
  const uint32_t lanes =
      kTeam < 32 ? ((1u << (kTeam & 31)) - 1) << (threadIdx.x & (32 - kTeam)) : 0xffffffffu;
#pragma unroll
  for (int o = (kTeam < 32 ? kTeam : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(lanes, v, o);
  if constexpr (kTeam > 32) {
    __shared__ float red[kTeam / 32];
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < kTeam / 32; ++i) v += red[i];
    __syncthreads();
  }
  return v;
}

// Row t once more, from memory, by a team of kTeam threads: y, h and the
// statistics.  `mean` and `squares` are the first try's.
template <int kTeam>
__device__ __forceinline__ void norm_row_again(const NormFwd& p, int64_t t, float mean, float squares) {
  const int tid = threadIdx.x % kTeam;
  auto h_at = [&](int64_t c) {
    float v = load_elem(p.x, p.x_bf16, t * p.ldx + c);
    if (p.residual) v += load_elem(p.residual, p.x_bf16, t * p.ldr + c);
    return v;
  };
  float scale = norm_scale(mean, squares), s = 0.f;
#pragma unroll 1
  for (int64_t c = tid; c < p.C; c += kTeam) s = fmaf(h_at(c), scale, s);
  mean = team_total<kTeam>(s) / (float)p.C;
  s = 0.f;
#pragma unroll 1
  for (int64_t c = tid; c < p.C; c += kTeam) {
    const float d = fmaf(h_at(c), scale, -mean);
    s = fmaf(d, d, s);
  }
  s = team_total<kTeam>(s);
  const float rstd = norm_rstd(s / (float)p.C, p.eps, mean, scale);
#pragma unroll 1
  for (int64_t c = tid; c < p.C; c += kTeam) {
    const float h = h_at(c);
    const float w = p.weight ? load_elem(p.weight, p.w_bf16, c) : 1.f;
    const float b = p.bias ? load_elem(p.bias, p.w_bf16, c) : 0.f;
    if (p.h) store_elem(p.h, p.x_bf16, t * p.ldh + c, h);
    store_elem(p.y, p.y_bf16, t * p.ldy + c, fmaf(fmaf(h, scale, -mean) * rstd, w, b));
  }
  if (tid == 0) write_stats(p, t, mean / scale, rstd * scale);
}

}  // namespace
}  // namespace hlq
