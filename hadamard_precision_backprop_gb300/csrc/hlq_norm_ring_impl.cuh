// hlq_norm_ring_impl.cuh -- the kernel of hlq_norm_ring.cuh.
//
// A team of kTeam threads takes every (number of teams)-th row: a warp, with
// several in a CTA and one CTA per SM, or for longer rows the whole CTA, one
// to four per SM.  The rows of x, g_y and the residual's gradient come into a
// ring of shared-memory stages by bulk copies, several rows ahead; each thread
// owns up to kUnits groups of four columns and keeps their weights, and their
// sums for g_w and g_b over all its rows, in registers.  The CTA's teams add
// their sums in shared memory and write one slab of partial sums, which
// norm_bwd_join_kernel adds; few rows go to one cluster, whose CTAs add their
// sums through distributed shared memory.
//
// Bound by HBM for long rows: 16384 x 14336 bf16 (1.41 GB) in 213 us, 0.99 of
// the measured copy rate, 16384 x 4096 with fp32 g_y and a residual (671 MB) in
// 105 us, 0.95.  16384 x 1024 with fp32 g_y (134 MB) takes 34 us, 0.60.  At 12608
// x 768 (97 MB, 25 us) each further row costs what its
// bytes do (1.15 us for 1000), and the rest is about 10 us of launch, first
// copies, the sums' joining and its launch.
//
// Groups of four: fp32 and bf16 columns both lie next to each other over a
// warp, without bank conflicts; pairs of fp32 go through one instruction (26
// instructions an element before that and before the output type was decided
// outside the column loop: 264 us at 16384 x 14336).  Rows go to CTAs in turn,
// not in runs: with a run of consecutive rows for each CTA that case took 246.
#pragma once

#include <type_traits>

#include "hlq_device.cuh"
#include "hlq_norm_ring.cuh"
#include "hlq_rows.cuh"
#include "hlq_tma.cuh"

namespace hlq {
namespace {

template <int kTeam>
__device__ __forceinline__ void team_sync() {
  if constexpr (kTeam == 32)
    __syncwarp();
  else
    __syncthreads();
}

// The sums of a and b over a warp: the halves of the warp take one each, which
// halves the shuffles.  Lane 0 ends with the sum of a, lane 16 with that of b.
__device__ __forceinline__ float warp_sum_pair(float a, float b) {
  const bool high = threadIdx.x & 16;
  float v = (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <bool kXBf16, bool kGyBf16, int kTeam, int kUnits>
__global__ void __launch_bounds__(ring_threads(kTeam, kUnits), kTeam == 32 ? 1 : 512 / kTeam)
    norm_bwd_ring_kernel(const __grid_constant__ NormBwd p, const __grid_constant__ RingPlan plan) {
  constexpr int kWarps = kTeam / 32, kPairs = kUnits * 2;
  constexpr int kSx = kXBf16 ? 2 : 4, kSg = kGyBf16 ? 2 : 4;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int abort_flag;
  const int team = threadIdx.x / kTeam, tid = threadIdx.x % kTeam;
  const int lane = threadIdx.x & 31, warp = tid >> 5;
  const int C = (int)p.C, sr = p.gx_bf16 ? 2 : 4;
  unsigned char* ring = smem + (size_t)team * plan.stages * plan.stage_bytes;
  unsigned char* tail = smem + plan.smem - (8 * 8 + 8 * kWarps) * plan.teams;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail) + team * 8;
  float* red = reinterpret_cast<float*>(tail + 8 * 8 * plan.teams) + team * 2 * kWarps;

  if (threadIdx.x == 0) abort_flag = 0;
  if (tid == 0) {
    for (int s = 0; s < plan.stages; ++s) mbar_init(&full[s], 1);
    // the copies complete on the barriers through the async proxy
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  const int64_t step = (int64_t)gridDim.x * plan.teams;
  const int64_t t0 = blockIdx.x + (int64_t)gridDim.x * team;
  int64_t issued = 0;
  auto issue = [&](int64_t t, int s) {
    if (t >= p.T || *(volatile int*)&abort_flag) return;
    ++issued;
    const uint32_t dst = saddr(ring + (size_t)s * plan.stage_bytes);
    mbar_expect_tx(&full[s], (uint32_t)plan.stage_bytes);
    bulk_load(dst, static_cast<const char*>(p.x) + t * p.ldx * kSx, C * kSx, &full[s]);
    bulk_load(dst + C * kSx, static_cast<const char*>(p.gy) + t * p.ldgy * kSg, C * kSg, &full[s]);
    if (p.gres)
      bulk_load(dst + C * (kSx + kSg), static_cast<const char*>(p.gres) + t * p.ldgr * sr, C * sr,
                &full[s]);
  };
  // The warp goes on together: lanes that spun on a stage ahead of the lane
  // that fills it could keep that lane from running.
  if (tid == 0)
    for (int s = 0; s < plan.stages; ++s) issue(t0 + s * step, s);
  __syncwarp();

  F2 gw[kPairs], gb[kPairs], w[kPairs];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int c = (i * kTeam + tid) * 4;
    Quad q = {{f2(1.f), f2(1.f)}};
    if (p.weight && c < C) q = p.w_bf16 ? load4<true>(p.weight, c) : load4<false>(p.weight, c);
    w[i * 2] = q.v[0], w[i * 2 + 1] = q.v[1];
    gw[i * 2] = gw[i * 2 + 1] = gb[i * 2] = gb[i * 2 + 1] = f2(0.f);
  }
  const float inv = 1.f / (float)C;
  int stage = 0;
  uint32_t parity = 0;
  float mean_next = 0.f, rstd_next = 0.f;
  if (t0 < p.T) mean_next = p.mean[t0], rstd_next = p.rstd[t0];
  for (int64_t t = t0; t < p.T; t += step) {
    const float mean = mean_next, rstd = rstd_next;
    if (t + step < p.T) mean_next = p.mean[t + step], rstd_next = p.rstd[t + step];
    // after a wait that gave up, the others return at once and the loop runs
    // to its end: every barrier is still met
    mbar_wait(&full[stage], parity, &abort_flag, p.status);
    const unsigned char* row = ring + (size_t)stage * plan.stage_bytes;
    const unsigned char *xs = row + tid * 4 * kSx, *gs = row + C * kSx + tid * 4 * kSg;
    const F2 neg_mean = f2(-mean), rstd2 = f2(rstd);
    F2 sa2 = f2(0.f), sx2 = f2(0.f);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if ((i * kTeam + tid) * 4 < C) {
        const Quad x = load4<kXBf16>(xs, i * kTeam * 4), g = load4<kGyBf16>(gs, i * kTeam * 4);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const F2 xhat = (x.v[k] + neg_mean) * rstd2, a = g.v[k] * w[i * 2 + k];
          sa2 = sa2 + a;
          sx2 = fma2(a, xhat, sx2);
          gw[i * 2 + k] = fma2(g.v[k], xhat, gw[i * 2 + k]);
          gb[i * 2 + k] = gb[i * 2 + k] + g.v[k];
        }
      }
    }
    const float2 pa = split(sa2), px = split(sx2);
    float sum = warp_sum_pair(pa.x + pa.y, px.x + px.y), sa, sx;
    if constexpr (kWarps > 1) {
      if ((lane & 15) == 0) red[(lane >> 4) * kWarps + warp] = sum;
      team_sync<kTeam>();  // written again only after the sync at the row's end
      sum = (lane & 15) < kWarps ? red[(lane >> 4) * kWarps + (lane & 15)] : 0.f;
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    sa = __shfl_sync(0xffffffffu, sum, 0) * inv;
    sx = __shfl_sync(0xffffffffu, sum, 16) * inv;
    // g_x = rstd (a - sa - (x - mean) (rstd sx)) (+ g_residual): no rstd^2, which
    // leaves fp32's range long before these do
    const F2 shift = f2(-sa), slope = f2(-rstd * sx);
    auto write = [&](auto out_bf16, auto with_residual) {
      constexpr bool kOut = decltype(out_bf16)::value;
      constexpr int kSr = kOut ? 2 : 4;
      char* to = static_cast<char*>(p.gx) + (t * p.ldgx + tid * 4) * kSr;
      const unsigned char* rs = row + C * (kSx + kSg) + tid * 4 * kSr;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        if ((i * kTeam + tid) * 4 < C) {
          const Quad x = load4<kXBf16>(xs, i * kTeam * 4), g = load4<kGyBf16>(gs, i * kTeam * 4);
          Quad o;
          if constexpr (decltype(with_residual)::value) o = load4<kOut>(rs, i * kTeam * 4);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const F2 d = fma2(x.v[k] + neg_mean, slope, fma2(g.v[k], w[i * 2 + k], shift));
            if constexpr (decltype(with_residual)::value)
              o.v[k] = fma2(d, rstd2, o.v[k]);
            else
              o.v[k] = d * rstd2;
          }
          store4<kOut>(to, i * kTeam * 4, o);
        }
      }
    };
    if (p.gx_bf16)
      p.gres ? write(std::true_type{}, std::true_type{}) : write(std::true_type{}, std::false_type{});
    else
      p.gres ? write(std::false_type{}, std::true_type{})
             : write(std::false_type{}, std::false_type{});
    if (tid == 0 && !(fabsf(sa) < INFINITY && fabsf(sx) < INFINITY))
      raise_flag(p.status, HLQ_DEV_NONFINITE);
    team_sync<kTeam>();  // the stage has been read by the whole team
    if (tid == 0) issue(t + plan.stages * step, stage);
    __syncwarp();
    if (++stage == plan.stages) stage = 0, parity ^= 1;
  }
  if (tid == 0 && *(volatile int*)&abort_flag) ring_drain(full, plan.stages, issued);
  if (!p.part) return;
  float* slab = p.part + (size_t)blockIdx.x * 2 * p.C;
  if (plan.teams == 1 && !plan.cluster) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = (i * kTeam + tid) * 4;
      if (c < C) {
        store4<false>(slab, c, {{gw[i * 2], gw[i * 2 + 1]}});
        store4<false>(slab, C + c, {{gb[i * 2], gb[i * 2 + 1]}});
      }
    }
    return;
  }
  // Every copy has been waited for by its team: the ring is free for the
  // teams' sums, which are added in the teams' order.
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int c = (i * kTeam + tid) * 4;
    if (c < C) {
      store4<false>(sums + team * 2 * C, c, {{gw[i * 2], gw[i * 2 + 1]}});
      store4<false>(sums + team * 2 * C, C + c, {{gb[i * 2], gb[i * 2 + 1]}});
    }
  }
  __syncthreads();
  float* cta_sums = plan.cluster ? sums : slab;
  for (int c = threadIdx.x * 4; c < 2 * C; c += blockDim.x * 4) {
    Quad q = load4<false>(sums, c);
    for (int k = 1; k < plan.teams; ++k) {
      const Quad r = load4<false>(sums + k * 2 * C, c);
      q.v[0] = q.v[0] + r.v[0], q.v[1] = q.v[1] + r.v[1];
    }
    store4<false>(cta_sums, c, q);
  }
  if (!plan.cluster) return;
  // Few rows: the CTAs are one cluster, and each adds a part of the columns
  // over all of them, from their shared memory.
  __syncthreads();
  cluster_sync();
  for (int c = (blockIdx.x * blockDim.x + threadIdx.x) * 4; c < 2 * C;
       c += plan.cluster * blockDim.x * 4) {
    float4 v = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < plan.cluster; ++k) {
      const float4 a = load_cluster(cluster_map(saddr(sums + c), k));
      v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
    }
    // C is a multiple of four: the group lies in one of the two
    const bool first = c < C;
    float* to = first ? p.gweight : p.gbias;
    if (to) {
      to += first ? c : c - C;
      to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;  // any alignment
    }
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while its sums may be read
}

template <bool kXBf16, bool kGyBf16, int kTeam, int kUnits>
cudaError_t launch_ring(const NormBwd& p, const RingPlan& r, cudaStream_t st) {
  const cudaError_t e = allow_smem<norm_bwd_ring_kernel<kXBf16, kGyBf16, kTeam, kUnits>>(r.smem_most);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(r.grid);
  cfg.blockDim = dim3(kTeam * r.teams);
  cfg.dynamicSmemBytes = r.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = r.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = r.cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, norm_bwd_ring_kernel<kXBf16, kGyBf16, kTeam, kUnits>, p, r);
}

template <bool kXBf16, bool kGyBf16>
cudaError_t pick_ring(const NormBwd& p, const RingPlan& r, cudaStream_t st) {
// Few steps of kUnits for the compiler's sake.  Those of the longest rows pay for
// themselves: with 8 in place of 6 and 7, 8192 x 12288 takes 143 us instead of 99
// and 8192 x 14336 156 instead of 110.
#define HLQ_RING(TEAM, UNITS) \
  if (r.team == TEAM && r.units <= UNITS) return launch_ring<kXBf16, kGyBf16, TEAM, UNITS>(p, r, st)
  HLQ_RING(32, 2);
  HLQ_RING(32, 4);
  HLQ_RING(32, 6);
  HLQ_RING(32, 8);
  HLQ_RING(128, 4);
  HLQ_RING(256, 4);
  HLQ_RING(512, 4);
  HLQ_RING(512, 6);
  HLQ_RING(512, 7);
  HLQ_RING(512, 8);
#undef HLQ_RING
  return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace hlq
