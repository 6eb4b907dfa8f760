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
#include "hlq_host.h"
#include "hlq_kernels.h"
#include "hlq_rows.cuh"
#include "hlq_tma.cuh"

namespace hlq {
namespace {

// Sum over the kTeam consecutive threads of a team, the same value in every
// one.  Teams of more than a warp are the whole CTA (`red`: a float a warp).
template <int kTeam>
__device__ __forceinline__ float team_sum(float v, float* red) {
#pragma unroll
  for (int o = (kTeam < 32 ? kTeam : 32) / 2; o > 0; o >>= 1)
    v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (kTeam > 32) {
    constexpr int kWarps = kTeam / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < kWarps ? red[lane] : 0.f;
#pragma unroll
    for (int o = (kWarps < 32 ? kWarps : 32) / 2; o > 0; o >>= 1)
      v += __shfl_xor_sync(0xffffffffu, v, o);
    v = __shfl_sync(0xffffffffu, v, 0);
  }
  return v;
}

// ---------------------------------------------------------------------------
// Forward.  A team of kTeam threads holds a row in registers, 32 elements a
// thread at most, so that the row is read once and the variance is taken from
// the differences to the mean; all of a thread's loads are in flight before
// the first is used.  kUnit = 8: 16-byte accesses.  kUnit = 1: single
// elements, for rows that are not made of aligned groups of eight.
// ---------------------------------------------------------------------------
constexpr int kHeld = 32;

template <bool kXBf16, int kTeam, int kUnit>
__global__ void __launch_bounds__(kTeam < 128 ? 128 : kTeam) norm_fwd_kernel(NormFwd p) {
  constexpr int kNum = kHeld / kUnit, kThreads = kTeam < 128 ? 128 : kTeam;
  __shared__ float red[2][32];
  const int tid = threadIdx.x % kTeam;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / kTeam) + threadIdx.x / kTeam;
  const bool live = t < p.T;
  const int C = (int)p.C;
  pdl_wait();
  float v[kHeld];
#pragma unroll
  for (int i = 0; i < kNum; ++i) {
    const int c = (i * kTeam + tid) * kUnit;
    if constexpr (kUnit == 8) {
      F8 f = {};
      if (live && c < C) f = load8(p.x, kXBf16, t * p.ldx + c);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i * 8 + k] = f.v[k];
    } else {
      v[i] = live && c < C ? load_elem(p.x, kXBf16, t * p.ldx + c) : 0.f;
    }
  }
  if (p.residual) {
#pragma unroll
    for (int i = 0; i < kNum; ++i) {
      const int c = (i * kTeam + tid) * kUnit;
      if constexpr (kUnit == 8) {
        F8 f = {};
        if (live && c < C) f = load8(p.residual, kXBf16, t * p.ldr + c);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i * 8 + k] += f.v[k];
      } else {
        v[i] += live && c < C ? load_elem(p.residual, kXBf16, t * p.ldr + c) : 0.f;
      }
    }
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) s += v[i];
  const float mean = team_sum<kTeam>(s, red[0]) / (float)C;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kNum; ++i) {
    if ((i * kTeam + tid) * kUnit < C) {
#pragma unroll
      for (int k = 0; k < kUnit; ++k) {
        const float d = v[i * kUnit + k] - mean;
        s = fmaf(d, d, s);
      }
    }
  }
  const float rstd = 1.f / sqrtf(team_sum<kTeam>(s, red[1]) / (float)C + p.eps);
  pdl_trigger();
  if (!live) return;
#pragma unroll
  for (int i = 0; i < kNum; ++i) {
    const int c = (i * kTeam + tid) * kUnit;
    if (c >= C) continue;
    if constexpr (kUnit == 8) {
      F8 h, w, b, y;
#pragma unroll
      for (int k = 0; k < 8; ++k) h.v[k] = v[i * 8 + k], w.v[k] = 1.f, b.v[k] = 0.f;
      if (p.weight) w = load8(p.weight, p.w_bf16, c);
      if (p.bias) b = load8(p.bias, p.w_bf16, c);
      if (p.h) store8(p.h, kXBf16, t * p.ldh + c, h);
#pragma unroll
      for (int k = 0; k < 8; ++k) y.v[k] = fmaf((h.v[k] - mean) * rstd, w.v[k], b.v[k]);
      store8(p.y, p.y_bf16, t * p.ldy + c, y);
    } else {
      const float w = p.weight ? load_elem(p.weight, p.w_bf16, c) : 1.f;
      const float b = p.bias ? load_elem(p.bias, p.w_bf16, c) : 0.f;
      if (p.h) store_elem(p.h, kXBf16, t * p.ldh + c, v[i]);
      store_elem(p.y, p.y_bf16, t * p.ldy + c, fmaf((v[i] - mean) * rstd, w, b));
    }
  }
  if (tid == 0) {
    if (p.mean) {
      p.mean[t] = mean;
      p.rstd[t] = rstd;
    }
    if (!isfinite(mean) || !isfinite(rstd)) raise_flag(p.status, HLQ_DEV_NONFINITE);
  }
}

// Rows too long for registers (more than 32 x 1024 elements): three passes,
// the later ones from L2.
constexpr int kLongThreads = 1024;

__global__ void __launch_bounds__(kLongThreads) norm_fwd_long_kernel(NormFwd p) {
  __shared__ float red[2][32];
  pdl_wait();
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    auto h_at = [&](int64_t c) {
      float v = load_elem(p.x, p.x_bf16, t * p.ldx + c);
      if (p.residual) v += load_elem(p.residual, p.x_bf16, t * p.ldr + c);
      return v;
    };
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < p.C; c += kLongThreads) s += h_at(c);
    const float mean = team_sum<kLongThreads>(s, red[0]) / (float)p.C;
    s = 0.f;
    for (int64_t c = threadIdx.x; c < p.C; c += kLongThreads) {
      const float d = h_at(c) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd =
        1.f / sqrtf(team_sum<kLongThreads>(s, red[1]) / (float)p.C + p.eps);
    for (int64_t c = threadIdx.x; c < p.C; c += kLongThreads) {
      const float h = h_at(c);
      const float w = p.weight ? load_elem(p.weight, p.w_bf16, c) : 1.f;
      const float b = p.bias ? load_elem(p.bias, p.w_bf16, c) : 0.f;
      if (p.h) store_elem(p.h, p.x_bf16, t * p.ldh + c, h);
      store_elem(p.y, p.y_bf16, t * p.ldy + c, fmaf((h - mean) * rstd, w, b));
    }
    if (threadIdx.x == 0) {
      if (p.mean) {
        p.mean[t] = mean;
        p.rstd[t] = rstd;
      }
      if (!isfinite(mean) || !isfinite(rstd)) raise_flag(p.status, HLQ_DEV_NONFINITE);
    }
    __syncthreads();  // red[0] is written again in the next row
  }
}

// ---------------------------------------------------------------------------
// Backward, rows of aligned groups of eight.  One CTA per SM; a team of
// kTeam threads takes every (teams)-th row.  The rows of g_y, x and the
// residual's gradient come into a ring of shared-memory stages by bulk
// copies, several rows ahead; each thread owns up to kNum groups of eight
// columns and keeps their sums for g_w and g_b in registers over all its
// rows.  The CTA's teams add their sums in shared memory and write one slab
// of partial sums.
// ---------------------------------------------------------------------------
struct RingPlan {
  int teams, stages, stage_bytes, grid;
  int w_bytes;  // the weights as fp32 in shared memory; 0: read from global
  size_t smem;
};

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

template <int kTeam, int kNum>
__global__ void __launch_bounds__(kTeam == 32 ? 256 : 512)
    norm_bwd_ring_kernel(const __grid_constant__ NormBwd p, const __grid_constant__ RingPlan plan) {
  constexpr int kWarps = kTeam / 32;
  extern __shared__ __align__(128) unsigned char smem[];
  const int team = threadIdx.x / kTeam, tid = threadIdx.x % kTeam;
  const int lane = threadIdx.x & 31, warp = tid >> 5;
  const int C = (int)p.C, sx = p.x_bf16 ? 2 : 4, sg = p.gy_bf16 ? 2 : 4, sr = p.gx_bf16 ? 2 : 4;
  float* wsm = reinterpret_cast<float*>(smem);
  unsigned char* ring0 = smem + plan.w_bytes;
  unsigned char* ring = ring0 + (size_t)team * plan.stages * plan.stage_bytes;
  unsigned char* tail = ring0 + (size_t)plan.teams * plan.stages * plan.stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail) + team * plan.stages;
  float* red = reinterpret_cast<float*>(tail + 8 * plan.teams * plan.stages) + team * 2 * kWarps;
  __shared__ int abort_flag;

  if (threadIdx.x == 0) abort_flag = 0;
  if (tid == 0)
    for (int s = 0; s < plan.stages; ++s) mbar_init(&full[s], 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  pdl_wait();
  if (plan.w_bytes)
    for (int c = threadIdx.x; c < C; c += blockDim.x)
      wsm[c] = p.weight ? load_elem(p.weight, p.w_bf16, c) : 1.f;
  __syncthreads();

  const int64_t step = (int64_t)gridDim.x * plan.teams;
  const int64_t t0 = (int64_t)blockIdx.x * plan.teams + team;
  auto issue = [&](int64_t t, int s) {
    if (t >= p.T || *(volatile int*)&abort_flag) return;
    const uint32_t dst = saddr(ring + (size_t)s * plan.stage_bytes);
    mbar_expect_tx(&full[s], (uint32_t)plan.stage_bytes);
    bulk_load(dst, static_cast<const char*>(p.x) + t * p.ldx * sx, C * sx, &full[s]);
    bulk_load(dst + C * sx, static_cast<const char*>(p.gy) + t * p.ldgy * sg, C * sg, &full[s]);
    if (p.gres)
      bulk_load(dst + C * (sx + sg), static_cast<const char*>(p.gres) + t * p.ldgr * sr, C * sr,
                &full[s]);
  };
  if (tid == 0)
    for (int s = 0; s < plan.stages; ++s) issue(t0 + s * step, s);

  float gw[kNum * 8], gb[kNum * 8];
#pragma unroll
  for (int i = 0; i < kNum * 8; ++i) gw[i] = gb[i] = 0.f;
  const float inv = 1.f / (float)C;
  int stage = 0;
  uint32_t parity = 0;
  float mean = 0.f, rstd = 0.f;
  if (t0 < p.T) mean = p.mean[t0], rstd = p.rstd[t0];
  for (int64_t t = t0; t < p.T; t += step) {
    float mean_next = 0.f, rstd_next = 0.f;
    if (t + step < p.T) mean_next = p.mean[t + step], rstd_next = p.rstd[t + step];
    mbar_wait(&full[stage], parity, &abort_flag, p.status);
    const unsigned char* row = ring + (size_t)stage * plan.stage_bytes;
    auto weights = [&](int c) {
      if (plan.w_bytes) {
        const float4* q = reinterpret_cast<const float4*>(wsm + c);
        return join8(q[0], q[1]);
      }
      return p.weight ? load8(p.weight, p.w_bf16, c)
                      : F8{{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}};
    };
    float sa = 0.f, sx_ = 0.f;
#pragma unroll
    for (int i = 0; i < kNum; ++i) {
      const int c = (i * kTeam + tid) * 8;
      if (c < C) {
        const F8 x = load8(row, p.x_bf16, c), g = load8(row + C * sx, p.gy_bf16, c);
        const F8 w = weights(c);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float xhat = (x.v[k] - mean) * rstd, a = g.v[k] * w.v[k];
          sa += a;
          sx_ = fmaf(a, xhat, sx_);
          gw[i * 8 + k] = fmaf(g.v[k], xhat, gw[i * 8 + k]);
          gb[i * 8 + k] += g.v[k];
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sa += __shfl_xor_sync(0xffffffffu, sa, o);
      sx_ += __shfl_xor_sync(0xffffffffu, sx_, o);
    }
    if constexpr (kWarps > 1) {
      if (lane == 0) red[warp] = sa, red[kWarps + warp] = sx_;
      team_sync<kTeam>(team);  // read again only after the sync at the row's end
      sa = sx_ = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) sa += red[i], sx_ += red[kWarps + i];
    }
    sa *= inv;
    sx_ *= inv;
#pragma unroll
    for (int i = 0; i < kNum; ++i) {
      const int c = (i * kTeam + tid) * 8;
      if (c < C) {
        const F8 x = load8(row, p.x_bf16, c), g = load8(row + C * sx, p.gy_bf16, c);
        const F8 w = weights(c);
        F8 o;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          o.v[k] = rstd * (fmaf(g.v[k], w.v[k], -sa) - (x.v[k] - mean) * rstd * sx_);
        if (p.gres) {
          const F8 r = load8(row + C * (sx + sg), p.gx_bf16, c);
#pragma unroll
          for (int k = 0; k < 8; ++k) o.v[k] += r.v[k];
        }
        store8(p.gx, p.gx_bf16, t * p.ldgx + c, o);
      }
    }
    if (tid == 0 && (!isfinite(sa) || !isfinite(sx_))) raise_flag(p.status, HLQ_DEV_NONFINITE);
    team_sync<kTeam>(team);  // the stage has been read by the whole team
    if (tid == 0) issue(t + plan.stages * step, stage);
    mean = mean_next, rstd = rstd_next;
    if (++stage == plan.stages) stage = 0, parity ^= 1;
  }
  pdl_trigger();
  if (!p.part) return;
  float* slab = p.part + (size_t)blockIdx.x * 2 * p.C;
  if (plan.teams == 1) {
#pragma unroll
    for (int i = 0; i < kNum; ++i) {
      const int c = (i * kTeam + tid) * 8;
      if (c < C) {
        F8 a, b;
#pragma unroll
        for (int k = 0; k < 8; ++k) a.v[k] = gw[i * 8 + k], b.v[k] = gb[i * 8 + k];
        store8(slab, false, c, a);
        store8(slab, false, C + c, b);
      }
    }
    return;
  }
  // every copy has been waited for by its team: the ring is free
  float* sum = reinterpret_cast<float*>(ring0);
  for (int k = 0; k < plan.teams; ++k) {
    __syncthreads();
    if (team != k) continue;
#pragma unroll
    for (int i = 0; i < kNum; ++i) {
      const int c = (i * kTeam + tid) * 8;
      if (c < C) {
        F8 a, b;
#pragma unroll
        for (int j = 0; j < 8; ++j) a.v[j] = gw[i * 8 + j], b.v[j] = gb[i * 8 + j];
        if (k > 0) {
          const F8 a0 = load8(sum, false, c), b0 = load8(sum, false, C + c);
#pragma unroll
          for (int j = 0; j < 8; ++j) a.v[j] += a0.v[j], b.v[j] += b0.v[j];
        }
        store8(sum, false, c, a);
        store8(sum, false, C + c, b);
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x * 4; c < 2 * C; c += blockDim.x * 4)
    *reinterpret_cast<float4*>(slab + c) = *reinterpret_cast<const float4*>(sum + c);
}

// ---------------------------------------------------------------------------
// Backward, any rows: g_x with one CTA per row, then the column sums of slabs
// of rows.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;

__global__ void __launch_bounds__(kRowThreads) norm_bwd_x_kernel(NormBwd p) {
  __shared__ float red[2][32];
  pdl_wait();
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const float mean = p.mean[t], rstd = p.rstd[t];
    float sa = 0.f, sx = 0.f;
    for (int64_t c = threadIdx.x; c < p.C; c += kRowThreads) {
      const float w = p.weight ? load_elem(p.weight, p.w_bf16, c) : 1.f;
      const float a = load_elem(p.gy, p.gy_bf16, t * p.ldgy + c) * w;
      sa += a;
      sx = fmaf(a, (load_elem(p.x, p.x_bf16, t * p.ldx + c) - mean) * rstd, sx);
    }
    sa = team_sum<kRowThreads>(sa, red[0]) / (float)p.C;
    sx = team_sum<kRowThreads>(sx, red[1]) / (float)p.C;
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
    __syncthreads();  // red is written again in the next row
  }
}

// Per-column sums over the rows of one slab: part[slab][0 / 1][c].
__global__ void __launch_bounds__(kRowThreads) norm_bwd_cols_kernel(NormBwd p) {
  pdl_wait();
  const int64_t c = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (c >= p.C) return;
  const int64_t t0 = p.T * blockIdx.y / gridDim.y, t1 = p.T * (blockIdx.y + 1) / gridDim.y;
  float gw = 0.f, gb = 0.f;
  for (int64_t t = t0; t < t1; ++t) {
    const float g = load_elem(p.gy, p.gy_bf16, t * p.ldgy + c);
    gw = fmaf(g, (load_elem(p.x, p.x_bf16, t * p.ldx + c) - p.mean[t]) * p.rstd[t], gw);
    gb += g;
  }
  p.part[(blockIdx.y * 2 + 0) * p.C + c] = gw;
  p.part[(blockIdx.y * 2 + 1) * p.C + c] = gb;
}

// The slabs' partial sums joined: a CTA takes 32 of the 2 C sums, its eight
// warps every eighth slab each.
__global__ void __launch_bounds__(256) norm_bwd_join_kernel(NormBwd p, int slabs) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane, n = 2 * p.C;
  pdl_wait();
  float s = 0.f;
  if (c < n) {
#pragma unroll 4
    for (int k = warp; k < slabs; k += 8) s += ld_dep_f32(p.part + k * n + c);
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp > 0 || c >= n) return;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) s += red[k][lane];
  if (c < p.C) {
    if (p.gweight) p.gweight[c] = s;
  } else {
    if (p.gbias) p.gbias[c - p.C] = s;
  }
}

constexpr size_t kSmemMost = 227 * 1024 - 256;  // what the static part leaves

// The ring's shape: as many stages as fit (at most 8, and no more than a team
// has rows); the weights in shared memory unless they would leave one stage.
// False: the rows do not fit.
bool ring_plan(const NormBwd& p, int team_threads, int most_teams, int sms, RingPlan* out) {
  RingPlan r{};
  const int64_t C = p.C;
  const int64_t size = (p.x_bf16 ? 2 : 4) + (p.gy_bf16 ? 2 : 4) + (p.gres ? (p.gx_bf16 ? 2 : 4) : 0);
  r.stage_bytes = (int)(C * size);
  const int64_t per_sm = (p.T + sms - 1) / sms;
  r.teams = (int)(per_sm < most_teams ? per_sm : most_teams);
  r.grid = (int)((p.T + r.teams - 1) / r.teams < sms ? (p.T + r.teams - 1) / r.teams : sms);
  const int64_t rows = (p.T + (int64_t)r.grid * r.teams - 1) / ((int64_t)r.grid * r.teams);
  const int64_t most = rows < 8 ? rows : 8;
  const size_t fixed = 8 * 8 * r.teams + 8 * r.teams * (team_threads / 32);
  for (int with_w = 1; with_w >= 0; --with_w) {
    r.w_bytes = with_w ? (int)(C * 4) : 0;
    if (fixed + r.w_bytes >= kSmemMost) continue;
    const int64_t fit = (int64_t)(kSmemMost - fixed - r.w_bytes) / ((int64_t)r.stage_bytes * r.teams);
    r.stages = (int)(fit < most ? fit : most);
    if (r.stages >= (with_w && most > 1 ? 2 : 1)) break;
  }
  if (r.stages < 1) return false;
  size_t ring = (size_t)r.stages * r.stage_bytes * r.teams;
  r.smem = fixed + r.w_bytes + ring;
  // the teams' sums are added in the ring
  if (r.teams > 1 && ring < (size_t)C * 8) r.smem += (size_t)C * 8 - ring;
  *out = r;
  return r.smem <= kSmemMost;
}

template <int kTeam, int kNum>
cudaError_t launch_ring(const NormBwd& p, const RingPlan& r, cudaStream_t st) {
  const cudaError_t e = allow_smem<norm_bwd_ring_kernel<kTeam, kNum>>(kSmemMost);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_bwd_ring_kernel<kTeam, kNum>, dim3(r.grid), dim3(kTeam * r.teams), r.smem,
                    st, p, r);
}

template <bool kXBf16>
cudaError_t launch_fwd(const NormFwd& p, bool eight, cudaStream_t st) {
  auto go = [&](auto kernel, int team) {
    const int threads = team < 128 ? 128 : team, rows = threads / team;
    return launch_pdl(kernel, dim3((unsigned)((p.T + rows - 1) / rows)), dim3(threads), 0, st, p);
  };
  if (eight) {
    if (p.C <= 8 * kHeld) return go(norm_fwd_kernel<kXBf16, 8, 8>, 8);
    if (p.C <= 32 * kHeld) return go(norm_fwd_kernel<kXBf16, 32, 8>, 32);
    if (p.C <= 128 * kHeld) return go(norm_fwd_kernel<kXBf16, 128, 8>, 128);
    if (p.C <= 512 * kHeld) return go(norm_fwd_kernel<kXBf16, 512, 8>, 512);
  } else {
    if (p.C <= 32 * kHeld) return go(norm_fwd_kernel<kXBf16, 32, 1>, 32);
    if (p.C <= 128 * kHeld) return go(norm_fwd_kernel<kXBf16, 128, 1>, 128);
  }
  if (p.C <= 1024 * kHeld) return go(norm_fwd_kernel<kXBf16, 1024, 1>, 1024);
  return launch_pdl(norm_fwd_long_kernel, dim3((unsigned)(p.T < 65535 ? p.T : 65535)),
                    dim3(kLongThreads), 0, st, p);
}

}  // namespace

int norm_bwd_most_slabs(int64_t T) { return (int)(T < 256 ? (T < 1 ? 1 : T) : 256); }

cudaError_t launch_norm_fwd(const NormFwd& p, cudaStream_t st) {
  const bool eight = rows_of_eight(p.x, p.ldx, p.x_bf16, p.T, p.C) &&
                     rows_of_eight(p.residual, p.ldr, p.x_bf16, p.T, p.C) &&
                     rows_of_eight(p.h, p.ldh, p.x_bf16, p.T, p.C) &&
                     rows_of_eight(p.y, p.ldy, p.y_bf16, p.T, p.C) &&
                     rows_of_eight(p.weight, 0, p.w_bf16, 1, p.C) &&
                     rows_of_eight(p.bias, 0, p.w_bf16, 1, p.C);
  return p.x_bf16 ? launch_fwd<true>(p, eight, st) : launch_fwd<false>(p, eight, st);
}

cudaError_t launch_norm_bwd(const NormBwd& p, int* slabs, cudaStream_t st) {
  const bool eight = rows_of_eight(p.x, p.ldx, p.x_bf16, p.T, p.C) &&
                     rows_of_eight(p.gy, p.ldgy, p.gy_bf16, p.T, p.C) &&
                     rows_of_eight(p.gres, p.ldgr, p.gx_bf16, p.T, p.C) &&
                     rows_of_eight(p.gx, p.ldgx, p.gx_bf16, p.T, p.C) &&
                     rows_of_eight(p.weight, 0, p.w_bf16, 1, p.C);
  int sms = device_sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  if (sms > 256) sms = 256;
  RingPlan r;
  const int team = p.C <= 1024 ? 32 : p.C <= 4096 ? 128 : 512;
  if (eight && p.C <= 512 * 32 && ring_plan(p, team, team == 32 ? 8 : team == 128 ? 4 : 1, sms, &r)) {
    *slabs = r.grid;
    const int num = (int)((p.C + team * 8 - 1) / (team * 8));
#define RING(TEAM, NUM) \
  if (team == TEAM && num == NUM) return launch_ring<TEAM, NUM>(p, r, st)
    RING(32, 1); RING(32, 2); RING(32, 3); RING(32, 4);
    RING(128, 2); RING(128, 3); RING(128, 4);
    RING(512, 2); RING(512, 3); RING(512, 4);
#undef RING
  }
  if (p.part) {
    *slabs = (int)(p.T < 128 ? p.T : 128);
    const dim3 grid((unsigned)((p.C + kRowThreads - 1) / kRowThreads), *slabs);
    const cudaError_t e = launch_pdl(norm_bwd_cols_kernel, grid, dim3(kRowThreads), 0, st, p);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(norm_bwd_x_kernel, dim3((unsigned)(p.T < 65535 ? p.T : 65535)),
                    dim3(kRowThreads), 0, st, p);
}

cudaError_t launch_norm_bwd_join(const NormBwd& p, int slabs, cudaStream_t st) {
  return launch_pdl(norm_bwd_join_kernel, dim3((unsigned)((2 * p.C + 31) / 32)), dim3(256), 0, st,
                    p, slabs);
}

}  // namespace hlq
