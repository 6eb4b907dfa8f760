// hlq_norm_ring_impl.cuh -- the kernel of hlq_norm_ring.cuh.
//
// One CTA per SM; a team of kTeam threads takes every (number of teams)-th
// row.  The rows of x, g_y and the residual's gradient come into a ring of
// shared-memory stages by bulk copies, several rows ahead; each thread owns up
// to kUnits groups of four columns and keeps their weights, and their sums
// for g_w and g_b over all its rows, in registers.  The CTA's teams add their
// sums in shared memory and write one slab of partial sums, which
// norm_bwd_join_kernel adds.
#pragma once

#include "hlq_device.cuh"
#include "hlq_norm_ring.cuh"
#include "hlq_rows.cuh"
#include "hlq_tma.cuh"

namespace hlq {
namespace {

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(saddr(bar))
      : "memory");
}

template <int kTeam>
__device__ __forceinline__ void team_sync(int team) {
  if constexpr (kTeam == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(kTeam) : "memory");
}

template <bool kXBf16, bool kGyBf16, int kTeam, int kUnits>
__global__ void __launch_bounds__(kTeam == 32 ? 256 : 512, 1)
    norm_bwd_ring_kernel(const __grid_constant__ NormBwd p, const __grid_constant__ RingPlan plan) {
  constexpr int kWarps = kTeam / 32, kPairs = kUnits * 2;
  // the first pass's x - mean and g_y w kept for the second, where a thread
  // has the registers (256 threads a CTA)
  constexpr bool kKeep = kTeam == 32;
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
  if (tid == 0)
    for (int s = 0; s < plan.stages; ++s) mbar_init(&full[s], 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  const int64_t step = (int64_t)gridDim.x * plan.teams;
  const int64_t t0 = (int64_t)blockIdx.x * plan.teams + team;
  auto issue = [&](int64_t t, int s) {
    if (t >= p.T || *(volatile int*)&abort_flag) return;
    const uint32_t dst = saddr(ring + (size_t)s * plan.stage_bytes);
    mbar_expect_tx(&full[s], (uint32_t)plan.stage_bytes);
    bulk_load(dst, static_cast<const char*>(p.x) + t * p.ldx * kSx, C * kSx, &full[s]);
    bulk_load(dst + C * kSx, static_cast<const char*>(p.gy) + t * p.ldgy * kSg, C * kSg, &full[s]);
    if (p.gres)
      bulk_load(dst + C * (kSx + kSg), static_cast<const char*>(p.gres) + t * p.ldgr * sr, C * sr,
                &full[s]);
  };
  if (tid == 0)
    for (int s = 0; s < plan.stages; ++s) issue(t0 + s * step, s);

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
  float mean = 0.f, rstd = 0.f;
  if (t0 < p.T) mean = p.mean[t0], rstd = p.rstd[t0];
  for (int64_t t = t0; t < p.T; t += step) {
    float mean_next = 0.f, rstd_next = 0.f;
    if (t + step < p.T) mean_next = p.mean[t + step], rstd_next = p.rstd[t + step];
    // after a wait that gave up, the others return at once and the loop runs
    // to its end: every barrier is still met
    mbar_wait(&full[stage], parity, &abort_flag, p.status);
    const unsigned char* row = ring + (size_t)stage * plan.stage_bytes;
    const F2 neg_mean = f2(-mean), rstd2 = f2(rstd);
    F2 keep_d[kKeep ? kPairs : 1], keep_a[kKeep ? kPairs : 1];
    F2 sa2 = f2(0.f), sx2 = f2(0.f);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = (i * kTeam + tid) * 4;
      if (c < C) {
        const Quad x = load4<kXBf16>(row, c), g = load4<kGyBf16>(row + C * kSx, c);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const F2 d = x.v[k] + neg_mean, xhat = d * rstd2, a = g.v[k] * w[i * 2 + k];
          sa2 = sa2 + a;
          sx2 = fma2(a, xhat, sx2);
          gw[i * 2 + k] = fma2(g.v[k], xhat, gw[i * 2 + k]);
          gb[i * 2 + k] = gb[i * 2 + k] + g.v[k];
          if constexpr (kKeep) keep_d[i * 2 + k] = d, keep_a[i * 2 + k] = a;
        }
      }
    }
    const float2 pa = split(sa2), px = split(sx2);
    float sa = pa.x + pa.y, sx = px.x + px.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sa += __shfl_xor_sync(0xffffffffu, sa, o);
      sx += __shfl_xor_sync(0xffffffffu, sx, o);
    }
    if constexpr (kWarps > 1) {
      if (lane == 0) red[warp] = sa, red[kWarps + warp] = sx;
      team_sync<kTeam>(team);  // written again only after the sync at the row's end
      sa = lane < kWarps ? red[lane] : 0.f;
      sx = lane < kWarps ? red[kWarps + lane] : 0.f;
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) {
        sa += __shfl_xor_sync(0xffffffffu, sa, o);
        sx += __shfl_xor_sync(0xffffffffu, sx, o);
      }
      sa = __shfl_sync(0xffffffffu, sa, 0);
      sx = __shfl_sync(0xffffffffu, sx, 0);
    }
    sa *= inv;
    sx *= inv;
    // g_x = rstd a - rstd sa - (x - mean) rstd^2 sx
    const F2 shift = f2(-rstd * sa), slope = f2(-rstd * rstd * sx);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = (i * kTeam + tid) * 4;
      if (c < C) {
        Quad o = {{shift, shift}};
        if (p.gres) {
          const void* r = row + C * (kSx + kSg);
          o = p.gx_bf16 ? load4<true>(r, c) : load4<false>(r, c);
          o.v[0] = o.v[0] + shift, o.v[1] = o.v[1] + shift;
        }
        if constexpr (kKeep) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            o.v[k] = fma2(keep_d[i * 2 + k], slope, fma2(keep_a[i * 2 + k], rstd2, o.v[k]));
        } else {
          const Quad x = load4<kXBf16>(row, c), g = load4<kGyBf16>(row + C * kSx, c);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            o.v[k] = fma2(x.v[k] + neg_mean, slope, fma2(g.v[k] * w[i * 2 + k], rstd2, o.v[k]));
        }
        if (p.gx_bf16)
          store4<true>(p.gx, t * p.ldgx + c, o);
        else
          store4<false>(p.gx, t * p.ldgx + c, o);
      }
    }
    if (tid == 0 && (!isfinite(sa) || !isfinite(sx))) raise_flag(p.status, HLQ_DEV_NONFINITE);
    team_sync<kTeam>(team);  // the stage has been read by the whole team
    if (tid == 0) issue(t + plan.stages * step, stage);
    mean = mean_next, rstd = rstd_next;
    if (++stage == plan.stages) stage = 0, parity ^= 1;
  }
  if (!p.part) return;
  float* slab = p.part + (size_t)blockIdx.x * 2 * p.C;
  if (plan.teams == 1) {
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
  // every copy has been waited for by its team: the ring is free
  float* sum = reinterpret_cast<float*>(smem);
  for (int k = 0; k < plan.teams; ++k) {
    __syncthreads();
    if (team != k) continue;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = (i * kTeam + tid) * 4;
      if (c < C) {
        Quad a = {{gw[i * 2], gw[i * 2 + 1]}}, b = {{gb[i * 2], gb[i * 2 + 1]}};
        if (k > 0) {
          const Quad a0 = load4<false>(sum, c), b0 = load4<false>(sum, C + c);
#pragma unroll
          for (int j = 0; j < 2; ++j) a.v[j] = a.v[j] + a0.v[j], b.v[j] = b.v[j] + b0.v[j];
        }
        store4<false>(sum, c, a);
        store4<false>(sum, C + c, b);
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x * 4; c < 2 * C; c += blockDim.x * 4)
    *reinterpret_cast<float4*>(slab + c) = *reinterpret_cast<const float4*>(sum + c);
}

template <bool kXBf16, bool kGyBf16, int kTeam, int kUnits>
cudaError_t launch_ring(const NormBwd& p, const RingPlan& r, cudaStream_t st) {
  const cudaError_t e = allow_smem<norm_bwd_ring_kernel<kXBf16, kGyBf16, kTeam, kUnits>>(kRingSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_bwd_ring_kernel<kXBf16, kGyBf16, kTeam, kUnits>, dim3(r.grid),
                    dim3(kTeam * r.teams), r.smem, st, p, r);
}

template <bool kXBf16, bool kGyBf16>
cudaError_t pick_ring(const NormBwd& p, const RingPlan& r, cudaStream_t st) {
#define HLQ_RING(TEAM, UNITS) \
  if (r.team == TEAM && r.units <= UNITS) return launch_ring<kXBf16, kGyBf16, TEAM, UNITS>(p, r, st)
  HLQ_RING(32, 2);
  HLQ_RING(32, 4);
  HLQ_RING(32, 6);
  HLQ_RING(32, 8);
  HLQ_RING(128, 4);
  HLQ_RING(128, 6);
  HLQ_RING(128, 8);
  HLQ_RING(512, 4);
  HLQ_RING(512, 6);
  HLQ_RING(512, 7);
  HLQ_RING(512, 8);
#undef HLQ_RING
  return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace hlq
