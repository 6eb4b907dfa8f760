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
#include "hlq_norm_range.cuh"
#include "hlq_norm_ring.cuh"
#include "hlq_rows.cuh"

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
// Forward.  A team of kTeam threads holds a row in registers, so that the row
// is read once and the variance is taken from the differences to the mean; all
// of a thread's loads are in flight before the first is used.  16-byte
// accesses, 32 elements a thread at most.
//
// Bound by HBM: 16384 x 4096 bf16 with a residual (537 MB) takes 83 us, 0.97 of
// the measured copy rate; 12608 x 768 fp32 without one (77 MB) 14 us, 0.83, and
// bf16 10 us, 0.58 (launch and last wave).  The team is the smallest of 8, 32,
// 128 and 512 threads that holds the row: more rows per SM are then under way,
// and short rows need no barrier.  64 registers a thread: two CTAs of 512 fit an
// SM (8192 x 14336 bf16 120 us where one took 178), and eight of 128.
// ---------------------------------------------------------------------------
constexpr int kHeld = 32;
constexpr int team_threads(int team) { return team < 128 ? 128 : team; }

template <bool kXBf16, int kTeam>
__global__ void __launch_bounds__(team_threads(kTeam), 1024 / team_threads(kTeam))
    norm_fwd_kernel(NormFwd p) {
  constexpr int kNum = kHeld / 8, kRows = team_threads(kTeam) / kTeam;
  __shared__ float red[2][32];
  const int tid = threadIdx.x % kTeam;
  const int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / kTeam;
  const bool live = t < p.T;
  const int C = (int)p.C;
  pdl_wait();
  pdl_trigger();
  float v[kHeld];
#pragma unroll
  for (int i = 0; i < kNum; ++i) {
    const int c = (i * kTeam + tid) * 8;
    F8 f = {};
    if (live && c < C) f = load8(p.x, kXBf16, t * p.ldx + c);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i * 8 + k] = f.v[k];
  }
  if (p.residual) {
#pragma unroll
    for (int i = 0; i < kNum; ++i) {
      const int c = (i * kTeam + tid) * 8;
      F8 f = {};
      if (live && c < C) f = load8(p.residual, kXBf16, t * p.ldr + c);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i * 8 + k] += f.v[k];
    }
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) s += v[i];
  const float mean = team_sum<kTeam>(s, red[0]) / (float)C;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kNum; ++i) {
    if ((i * kTeam + tid) * 8 < C) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = v[i * 8 + k] - mean;
        s = fmaf(d, d, s);
      }
    }
  }
  s = team_sum<kTeam>(s, red[1]);
  const float rstd = 1.f / sqrtf(s / (float)C + p.eps);
  if (!live) return;
  // a row beyond the squares' range writes nothing here
  const bool in_range = norm_in_range(s, norm_least(p.eps));
  const int limit = in_range ? C : 0;
#pragma unroll
  for (int i = 0; i < kNum; ++i) {
    const int c = (i * kTeam + tid) * 8;
    if (c >= limit) continue;
    F8 h, w, b, y;
#pragma unroll
    for (int k = 0; k < 8; ++k) h.v[k] = v[i * 8 + k], w.v[k] = 1.f, b.v[k] = 0.f;
    if (p.weight) w = load8(p.weight, p.w_bf16, c);
    if (p.bias) b = load8(p.bias, p.w_bf16, c);
    if (p.h) store8(p.h, kXBf16, t * p.ldh + c, h);
#pragma unroll
    for (int k = 0; k < 8; ++k) y.v[k] = fmaf((h.v[k] - mean) * rstd, w.v[k], b.v[k]);
    store8(p.y, p.y_bf16, t * p.ldy + c, y);
  }
  if (__builtin_expect(in_range, 1)) {
    if (tid == 0) write_stats(p, t, mean, rstd);
  } else {
    norm_row_again<kTeam>(p, t, mean, s);
  }
}

// Rows too long for registers (above 16384 elements), or for the shared memory
// of hlq_norm_elem.cu: three passes, the later ones from L2 or L1.  Two CTAs an
// SM; bound by latency and instructions, not by bytes: 2000 x 20001 bf16 103 us
// (24 us of bytes), 2000 x 9001 54 (11), 5000 x 2001 fp32 with a residual 80 (24).
// Holding rows of up to 16384 elements in the registers of one CTA an SM took
// 60 and 125 us for the last two.
constexpr int kLongThreads = 1024;

template <bool kXBf16>
__global__ void __launch_bounds__(kLongThreads) norm_fwd_long_kernel(NormFwd p) {
  __shared__ float red[2][32];
  pdl_wait();
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    auto h_at = [&](int64_t c) {
      float v = load_elem(p.x, kXBf16, t * p.ldx + c);
      if (p.residual) v += load_elem(p.residual, kXBf16, t * p.ldr + c);
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
    s = team_sum<kLongThreads>(s, red[1]);
    if (!norm_in_range(s, norm_least(p.eps))) {  // the same in every thread
      norm_row_again<kLongThreads>(p, t, mean, s);
      continue;
    }
    const float rstd = 1.f / sqrtf(s / (float)p.C + p.eps);
    for (int64_t c = threadIdx.x; c < p.C; c += kLongThreads) {
      const float h = h_at(c);
      const float w = p.weight ? load_elem(p.weight, p.w_bf16, c) : 1.f;
      const float b = p.bias ? load_elem(p.bias, p.w_bf16, c) : 0.f;
      if (p.h) store_elem(p.h, kXBf16, t * p.ldh + c, h);
      store_elem(p.y, p.y_bf16, t * p.ldy + c, fmaf((h - mean) * rstd, w, b));
    }
    if (threadIdx.x == 0) write_stats(p, t, mean, rstd);
    __syncthreads();  // red[0] is written again in the next row
  }
}

// ---------------------------------------------------------------------------
// Backward, rows too long for these: g_x with one CTA per row, then the column
// sums of slabs of rows.
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
// warps every eighth slab each (16 warps: 12 instead of 8 us for 152 slabs of
// 14336 columns).
__global__ void __launch_bounds__(256) norm_bwd_join_kernel(NormBwd p, int slabs) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane, n = 2 * p.C;
  pdl_wait();
  float s = 0.f;
  if (c < n) {
#pragma unroll 10
    for (int k = warp; k < slabs; k += 8) s += p.part[k * n + c];
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

template <bool kXBf16>
cudaError_t launch_fwd(const NormFwd& p, bool eight, cudaStream_t st) {
  auto go = [&](auto kernel, int team) {
    const int threads = team_threads(team), rows = threads / team;
    return launch_pdl(kernel, dim3((unsigned)((p.T + rows - 1) / rows)), dim3(threads), 0, st, p);
  };
  if (eight) {
    if (p.C <= 8 * kHeld) return go(norm_fwd_kernel<kXBf16, 8>, 8);
    if (p.C <= 32 * kHeld) return go(norm_fwd_kernel<kXBf16, 32>, 32);
    if (p.C <= 128 * kHeld) return go(norm_fwd_kernel<kXBf16, 128>, 128);
    if (p.C <= 512 * kHeld) return go(norm_fwd_kernel<kXBf16, 512>, 512);
  }
  return launch_pdl(norm_fwd_long_kernel<kXBf16>, dim3((unsigned)(p.T < 65535 ? p.T : 65535)),
                    dim3(kLongThreads), 0, st, p);
}

}  // namespace

// The ring's shape.  Teams: a warp up to 1024 columns (16 or 24 of them in the
// SM's one CTA: 8 that kept the first pass's values took 28.6 us at 12608 x 768
// where 16 take 24; above 768 columns a thread spills some 80 bytes, but teams of
// 128 threads take 36 us at 16384 x 1024 where a warp takes 34), CTAs of 128
// threads, four an SM, up to 2048 (one of 256 threads, two an SM: 64 us at 16384
// x 2048 where these take 60), of 256, two an SM, up to 4096 (four teams of 128 threads in one CTA left one stage each: 138
// us at 16384 x 4096 where these take 105), of 512 above.  As many stages as
// fit, at most 8 and no more than a team has rows.  False: the rows are not for
// the ring, or do not fit.
bool norm_bwd_ring_plan(const NormBwd& p, int sms, RingPlan* out) {
  if (sms <= 0 || p.C > 512 * kMostUnits * 4 || !rows_of_eight(p.x, p.ldx, p.x_bf16, p.T, p.C) ||
      !rows_of_eight(p.gy, p.ldgy, p.gy_bf16, p.T, p.C) ||
      !rows_of_eight(p.gres, p.ldgr, p.gx_bf16, p.T, p.C) ||
      !rows_of_eight(p.gx, p.ldgx, p.gx_bf16, p.T, p.C) ||
      !rows_of_eight(p.weight, 0, p.w_bf16, 1, p.C))
    return false;
  RingPlan r{};
  const int64_t C = p.C;
  r.team = C <= 32 * kMostUnits * 4 ? 32 : C <= 2048 ? 128 : C <= 4096 ? 256 : 512;
  const int per_sm = r.team == 32 ? 1 : 512 / r.team;
  if (sms * per_sm > kMostSlabs) sms = kMostSlabs / per_sm;
  // of the SM's 228 KB a CTA takes 1 KB more than it asks for
  r.smem_most = (size_t)(228 / per_sm - 1) * 1024 - 256;
  r.units = (int)((C + r.team * 4 - 1) / (r.team * 4));
  r.stage_bytes =
      (int)(C * ((p.x_bf16 ? 2 : 4) + (p.gy_bf16 ? 2 : 4) + (p.gres ? (p.gx_bf16 ? 2 : 4) : 0)));
  const int64_t ctas_most = (int64_t)sms * per_sm, rows_each = (p.T + ctas_most - 1) / ctas_most;
  const int teams_most = ring_threads(r.team, r.units) / r.team;
  r.teams = (int)(rows_each < teams_most ? rows_each : teams_most);
  const int64_t ctas = (p.T + r.teams - 1) / r.teams;
  r.grid = (int)(ctas < ctas_most ? ctas : ctas_most);
  // Few rows, and column sums wanted: one cluster of up to 8 CTAs, in which a
  // warp has 2 rows (a CTA team 1) at most and which joins the sums itself.
  // That costs the GPU a little and spares the host a launch: 8.4 us a call
  // instead of 9.6 for 197 x 768, 5.6 instead of 8.3 for 8 x 64.  (With 4 rows
  // a CTA it lost: 16 us instead of 10 for 32 x 14336.)
  const int64_t team_rows = r.team == 32 ? 2 : 1;
  if (p.part && p.T <= 8 * teams_most * team_rows) {
    int g = 1;
    while (g < 8 && (int64_t)g * teams_most < p.T) g *= 2;
    r.cluster = r.grid = g;
    const int64_t each = (p.T + g - 1) / g;
    r.teams = (int)(each < teams_most ? each : teams_most);
  }
  const int64_t rows = (p.T + (int64_t)r.grid * r.teams - 1) / ((int64_t)r.grid * r.teams);
  const size_t fixed = 8 * 8 * r.teams + 8 * r.teams * (r.team / 32);
  int64_t fit = (int64_t)(r.smem_most - fixed) / ((int64_t)r.stage_bytes * r.teams);
  if (fit > 8) fit = 8;
  r.stages = (int)(fit < rows ? fit : rows);
  if (r.stages < 1) return false;
  size_t ring = (size_t)r.stages * r.stage_bytes * r.teams;
  const size_t sums = r.teams > 1 || r.cluster ? (size_t)C * 8 * r.teams : 0;  // added there
  if (ring < sums) ring = sums;
  r.smem = fixed + ring;
  *out = r;
  return r.smem <= r.smem_most;
}

int norm_bwd_most_slabs(int64_t T) { return (int)(T < kMostSlabs ? (T < 1 ? 1 : T) : kMostSlabs); }

cudaError_t launch_norm_fwd(const NormFwd& p, cudaStream_t st) {
  const bool eight = rows_of_eight(p.x, p.ldx, p.x_bf16, p.T, p.C) &&
                     rows_of_eight(p.residual, p.ldr, p.x_bf16, p.T, p.C) &&
                     rows_of_eight(p.h, p.ldh, p.x_bf16, p.T, p.C) &&
                     rows_of_eight(p.y, p.ldy, p.y_bf16, p.T, p.C) &&
                     rows_of_eight(p.weight, 0, p.w_bf16, 1, p.C) &&
                     rows_of_eight(p.bias, 0, p.w_bf16, 1, p.C);
  RingPlan r;
  if (!eight && norm_fwd_elem_plan(p, device_sm_count(), &r)) return launch_norm_fwd_elem(p, r, st);
  return p.x_bf16 ? launch_fwd<true>(p, eight, st) : launch_fwd<false>(p, eight, st);
}

cudaError_t launch_norm_bwd(const NormBwd& p, int* slabs, cudaStream_t st) {
  RingPlan r;
  if (norm_bwd_ring_plan(p, device_sm_count(), &r)) {
    *slabs = r.cluster ? 0 : r.grid;
    return p.x_bf16 ? launch_norm_bwd_ring_bf16(p, r, st) : launch_norm_bwd_ring_f32(p, r, st);
  }
  if (norm_bwd_elem_plan(p, device_sm_count(), &r)) {
    *slabs = r.grid;
    return launch_norm_bwd_elem(p, r, st);
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
