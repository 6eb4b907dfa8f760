// hlq_norm_elem.cu -- layer norm, forward and backward, of rows that are not
// made of aligned groups of eight elements (odd lengths, odd strides).
//
// The rows come into a ring of shared-memory stages by bulk copies, as those
// of hlq_norm_ring_impl.cuh do.  A copy moves aligned 16-byte pieces, so it
// takes the pieces that the row touches, up to 15 bytes of its neighbours with
// it, and the row is read from where it begins in its slot.  Where that would
// leave the matrix (first and last row), the copy is the pieces inside the row
// and a thread moves the few elements around them.  From there on the work is
// by single elements: a thread owns up to 16 columns that lie kTeam apart, so
// that a warp's accesses are consecutive.
//
// Bound by instructions and by the barriers of its reductions, not by bytes
// (two- and four-byte accesses, some 20 instructions an element): forward 4689 x
// 5663 bf16 47 us (16 us of bytes), backward with fp32 g_y 77 us (32); with the
// rows loaded into registers by single elements instead, without a ring, these
// took 73 and 104 us.  A warp's lanes copy one matrix's row each: one lane for
// all of them took longer than the rest of a short row's work (20000 x 77
// backward 43 -> 22 us; its bytes take 2).
#include "hlq_device.cuh"
#include "hlq_norm_range.cuh"
#include "hlq_norm_ring.cuh"
#include "hlq_rows.cuh"
#include "hlq_tma.cuh"

namespace hlq {
namespace {

// One matrix's row as it is copied.
struct Span {
  uint64_t row, from, to;  // the row's address; the bulk copy's begin and end
};

// `pieces`: bytes of one row; [begin, end): the matrix.
__device__ __forceinline__ Span span_of(const void* base, int64_t ld_bytes, int64_t bytes,
                                        int64_t rows, int64_t t) {
  Span s;
  const uint64_t begin = reinterpret_cast<uint64_t>(base);
  const uint64_t end = begin + (rows - 1) * ld_bytes + bytes;
  s.row = begin + t * ld_bytes;
  s.from = s.row & ~15ull;
  s.to = (s.row + bytes + 15) & ~15ull;
  if (s.from < begin) s.from += 16;
  if (s.to > end) s.to -= 16;
  if (s.to < s.from) s.to = s.from;
  return s;
}
// A row's place in its slot.
__device__ __forceinline__ int row_at(const void* base, int64_t ld_bytes, int64_t t) {
  return ((uint32_t)reinterpret_cast<uint64_t>(base) + (uint32_t)t * (uint32_t)ld_bytes) & 15;
}
__host__ __device__ constexpr int slot_bytes(int64_t bytes) {
  return (int)((bytes + 15) / 16 * 16 + 16);
}

// The elements of the row outside the bulk copy, into the slot.
__device__ __forceinline__ void copy_edges(const Span& s, int64_t bytes, int size,
                                           unsigned char* slot) {
  const uint64_t row_end = s.row + bytes;
  unsigned char* at = slot + (s.row & 15) - s.row;  // address -> place
  auto copy = [&](uint64_t a, uint64_t b) {
    for (; a < b; a += size) {
      if (size == 2)
        *reinterpret_cast<uint16_t*>(at + a) = *reinterpret_cast<const uint16_t*>(a);
      else
        *reinterpret_cast<uint32_t*>(at + a) = *reinterpret_cast<const uint32_t*>(a);
    }
  };
  if (s.from == s.to) {
    copy(s.row, row_end);
  } else {
    copy(s.row, s.from);
    copy(s.to, row_end);
  }
}

// The matrix that a lane copies the rows of.
struct Source {
  const void* base;
  int64_t ld_bytes, bytes;
  int size, slot;  // element size; the slot's offset in a stage
};

// Row t of the first `n` lanes' matrices into a stage, by one warp together.
__device__ __forceinline__ void issue_rows(const Source& src, int n, int64_t rows, int64_t t,
                                           unsigned char* stage, uint64_t* bar) {
  const int lane = threadIdx.x & 31;
  Span s = {};
  if (lane < n) {
    s = span_of(src.base, src.ld_bytes, src.bytes, rows, t);
    if (s.from > s.row || s.to < s.row + src.bytes)
      copy_edges(s, src.bytes, src.size, stage + src.slot);
  }
  const uint32_t bytes = (uint32_t)(s.to - s.from);
  uint32_t total = 0;
#pragma unroll
  for (int k = 0; k < 3; ++k) total += __shfl_sync(0xffffffffu, bytes, k);  // 0 from lane n on
  __syncwarp();
  if (lane == 0) mbar_expect_tx(bar, total);  // an arrival: releases the elements just copied
  __syncwarp();
  if (bytes > 0)
    bulk_load(saddr(stage + src.slot) + (uint32_t)(s.from - (s.row & ~15ull)),
              reinterpret_cast<const void*>(s.from), bytes, bar);
  __syncwarp();
}

// The same by one thread, after another (and then its warp together again).
__device__ __forceinline__ void issue_rows_alone(const Source& a, const Source& b, int n,
                                                 int64_t rows, int64_t t, unsigned char* stage,
                                                 uint64_t* bar) {
  uint32_t total = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k < n) {
      const Source& src = k ? b : a;
      const Span s = span_of(src.base, src.ld_bytes, src.bytes, rows, t);
      total += (uint32_t)(s.to - s.from);
      if (s.from > s.row || s.to < s.row + src.bytes)
        copy_edges(s, src.bytes, src.size, stage + src.slot);
    }
  mbar_expect_tx(bar, total);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k < n) {
      const Source& src = k ? b : a;
      const Span s = span_of(src.base, src.ld_bytes, src.bytes, rows, t);
      if (s.to > s.from)
        bulk_load(saddr(stage + src.slot) + (uint32_t)(s.from - (s.row & ~15ull)),
                  reinterpret_cast<const void*>(s.from), (uint32_t)(s.to - s.from), bar);
    }
}

// A team's ring: its stages, and the barriers their copies complete on.
struct Ring {
  unsigned char* stages;
  uint64_t* full;
};
template <int kTeam>
__device__ __forceinline__ Ring ring_setup(unsigned char* smem, const RingPlan& plan, int team,
                                           int tid, int* abort_flag) {
  Ring r;
  r.stages = smem + plan.before + (size_t)team * plan.stages * plan.stage_bytes;
  r.full = reinterpret_cast<uint64_t*>(smem + plan.smem - 8 * 8 * plan.teams) + team * 8;
  if (threadIdx.x == 0) *abort_flag = 0;
  if (tid == 0) {
    for (int s = 0; s < plan.stages; ++s) mbar_init(&r.full[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  __syncthreads();
  return r;
}

template <int kTeam>
__device__ __forceinline__ void team_sync() {
  if constexpr (kTeam == 32)
    __syncwarp();
  else
    __syncthreads();
}

// Sum over the team; `red` holds a float for each of the CTA's warps and may be
// written again after the next team_sync but one.
template <int kTeam>
__device__ __forceinline__ float team_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (kTeam > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kTeam / 32; ++i) v += red[i];
  }
  return v;
}

template <bool kBf16>
__device__ __forceinline__ float shared_elem(const unsigned char* row, int c) {
  if constexpr (kBf16)
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[c]);
  else
    return reinterpret_cast<const float*>(row)[c];
}

constexpr int kCols = 16;  // columns a thread owns

// By a call: inlined, it cost the rows in range 7 us of 48 at 4689 x 5663.
template <int kTeam>
__device__ __noinline__ void row_apart(const NormFwd& p, int64_t t, float mean, float squares) {
  norm_row_again<kTeam>(p, t, mean, squares);
}

constexpr int elem_threads(int team) { return team > 32 ? team : 512; }

// Twice as many threads an SM as in the backward pass: only the row is in
// registers, weights and bias are in shared memory as fp32 (before the rings).
template <bool kXBf16, int kTeam>
__global__ void __launch_bounds__(elem_threads(kTeam), kTeam == 32 ? 2 : 1024 / kTeam)
    norm_fwd_elem_kernel(const __grid_constant__ NormFwd p, const __grid_constant__ RingPlan plan) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float red[2][kTeam / 32];
  __shared__ int abort_flag;
  constexpr int kSize = kXBf16 ? 2 : 4;
  const int team = threadIdx.x / kTeam, tid = threadIdx.x % kTeam, C = (int)p.C;
  float *w = reinterpret_cast<float*>(smem), *b = w + C;
  const Ring ring = ring_setup<kTeam>(smem, plan, team, tid, &abort_flag);
  pdl_wait();
  pdl_trigger();
  for (int c = threadIdx.x; c < C; c += blockDim.x) {
    w[c] = p.weight ? load_elem(p.weight, p.w_bf16, c) : 1.f;
    b[c] = p.bias ? load_elem(p.bias, p.w_bf16, c) : 0.f;
  }
  const int lane = threadIdx.x & 31;
  const int64_t x_ld = p.ldx * kSize, r_ld = p.ldr * kSize;
  const int r_slot = slot_bytes(p.C * kSize);
  const Source x_src = {p.x, x_ld, p.C * kSize, kSize, 0};
  const Source r_src = {p.residual, r_ld, p.C * kSize, kSize, r_slot};
  const int64_t step = (int64_t)gridDim.x * plan.teams;
  const int64_t t0 = blockIdx.x + (int64_t)gridDim.x * team;
  // a warp's short rows by its lanes together, the longer ones by one thread
  // (49 against 60 us at 4689 x 5663)
  int64_t issued = 0;
  auto issue = [&](int64_t t, int s) {
    unsigned char* to = ring.stages + (size_t)s * plan.stage_bytes;
    if constexpr (kTeam == 32) {
      if (t < p.T && !__shfl_sync(0xffffffffu, *(volatile int*)&abort_flag, 0)) {
        ++issued;
        issue_rows(lane == 0 ? x_src : r_src, p.residual ? 2 : 1, p.T, t, to, &ring.full[s]);
      }
    } else {
      if (tid == 0 && t < p.T && !*(volatile int*)&abort_flag) {
        ++issued;
        issue_rows_alone(x_src, r_src, p.residual ? 2 : 1, p.T, t, to, &ring.full[s]);
      }
    }
  };
  for (int s = 0; s < plan.stages; ++s) issue(t0 + s * step, s);
  __syncthreads();
  const float inv = 1.f / (float)C, least = norm_least(p.eps);
  int stage = 0;
  uint32_t parity = 0;
  for (int64_t t = t0; t < p.T; t += step) {
    mbar_wait(&ring.full[stage], parity, &abort_flag, p.status);
    const unsigned char* at = ring.stages + (size_t)stage * plan.stage_bytes;
    const unsigned char* xs = at + row_at(p.x, x_ld, t);
    const unsigned char* rs = at + r_slot + row_at(p.residual, r_ld, t);
    float v[kCols], s = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const int c = i * kTeam + tid;
      v[i] = 0.f;
      if (c < C) {
        v[i] = shared_elem<kXBf16>(xs, c);
        if (p.residual) v[i] += shared_elem<kXBf16>(rs, c);
      }
      s += v[i];
    }
    const float mean = team_sum<kTeam>(s, red[0]) * inv;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      v[i] -= mean;
      if (i * kTeam + tid < C) s = fmaf(v[i], v[i], s);
    }
    s = team_sum<kTeam>(s, red[1]);
    const float rstd = 1.f / sqrtf(s * inv + p.eps);
    auto write = [&](auto out_bf16) {
      constexpr bool kOut = decltype(out_bf16)::value;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int c = i * kTeam + tid;
        if (c < C) store_elem(p.y, kOut, t * p.ldy + c, fmaf(v[i] * rstd, w[c], b[c]));
      }
    };
    if (!norm_in_range(s, least)) {  // the same in the whole team
      row_apart<kTeam>(p, t, mean, s);
    } else if (p.y_bf16) {
      write(std::true_type{});
    } else {
      write(std::false_type{});
    }
    if (p.h) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int c = i * kTeam + tid;
        if (c < C)
          store_elem(p.h, kXBf16, t * p.ldh + c,
                     shared_elem<kXBf16>(xs, c) + shared_elem<kXBf16>(rs, c));
      }
    }
    if (tid == 0 && norm_in_range(s, least)) {
      if (p.mean) p.mean[t] = mean, p.rstd[t] = rstd;
      if (!(rstd < INFINITY)) raise_flag(p.status, HLQ_DEV_NONFINITE);
    }
    team_sync<kTeam>();  // the stage has been read by the whole team
    issue(t + plan.stages * step, stage);
    __syncwarp();
    if (++stage == plan.stages) stage = 0, parity ^= 1;
  }
  if (tid == 0 && *(volatile int*)&abort_flag) ring_drain(ring.full, plan.stages, issued);
}

template <bool kXBf16, bool kGyBf16, int kTeam>
__global__ void __launch_bounds__(elem_threads(kTeam), kTeam == 32 ? 1 : 512 / kTeam)
    norm_bwd_elem_kernel(const __grid_constant__ NormBwd p, const __grid_constant__ RingPlan plan) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float red[2][kTeam / 32];
  __shared__ int abort_flag;
  constexpr int kSx = kXBf16 ? 2 : 4, kSg = kGyBf16 ? 2 : 4;
  const int team = threadIdx.x / kTeam, tid = threadIdx.x % kTeam, C = (int)p.C;
  const int sr = p.gx_bf16 ? 2 : 4;
  const Ring ring = ring_setup<kTeam>(smem, plan, team, tid, &abort_flag);
  pdl_wait();
  pdl_trigger();
  const int gy_slot = slot_bytes(p.C * kSx), r_slot = gy_slot + slot_bytes(p.C * kSg);
  const int lane = threadIdx.x & 31;
  const int64_t x_ld = p.ldx * kSx, gy_ld = p.ldgy * kSg, r_ld = p.ldgr * sr;
  const int size = lane == 0 ? kSx : lane == 1 ? kSg : sr;
  const Source src = {lane == 0 ? p.x : lane == 1 ? p.gy : p.gres,
                      lane == 0 ? x_ld : lane == 1 ? gy_ld : r_ld, p.C * size, size,
                      lane == 0 ? 0 : lane == 1 ? gy_slot : r_slot};
  const int64_t step = (int64_t)gridDim.x * plan.teams;
  const int64_t t0 = blockIdx.x + (int64_t)gridDim.x * team;
  int64_t issued = 0;
  auto issue = [&](int64_t t, int s) {
    if (t >= p.T || __shfl_sync(0xffffffffu, *(volatile int*)&abort_flag, 0)) return;
    ++issued;
    issue_rows(src, p.gres ? 3 : 2, p.T, t, ring.stages + (size_t)s * plan.stage_bytes,
               &ring.full[s]);
  };
  if (tid < 32)
    for (int s = 0; s < plan.stages; ++s) issue(t0 + s * step, s);
  float w[kCols], gw[kCols], gb[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    const int c = i * kTeam + tid;
    w[i] = p.weight && c < C ? load_elem(p.weight, p.w_bf16, c) : 1.f;
    gw[i] = gb[i] = 0.f;
  }
  const float inv = 1.f / (float)C;
  int stage = 0;
  uint32_t parity = 0;
  float mean_next = 0.f, rstd_next = 0.f;
  if (t0 < p.T) mean_next = p.mean[t0], rstd_next = p.rstd[t0];
  for (int64_t t = t0; t < p.T; t += step) {
    const float mean = mean_next, rstd = rstd_next;
    if (t + step < p.T) mean_next = p.mean[t + step], rstd_next = p.rstd[t + step];
    mbar_wait(&ring.full[stage], parity, &abort_flag, p.status);
    const unsigned char* at = ring.stages + (size_t)stage * plan.stage_bytes;
    const unsigned char* xs = at + row_at(p.x, x_ld, t);
    const unsigned char* gs = at + gy_slot + row_at(p.gy, gy_ld, t);
    const unsigned char* rs = at + r_slot + row_at(p.gres, r_ld, t);
    float xhat[kCols], a[kCols], sa = 0.f, sx = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const int c = i * kTeam + tid;
      xhat[i] = a[i] = 0.f;
      if (c < C) {
        const float g = shared_elem<kGyBf16>(gs, c);
        xhat[i] = (shared_elem<kXBf16>(xs, c) - mean) * rstd;
        a[i] = g * w[i];
        gw[i] = fmaf(g, xhat[i], gw[i]);
        gb[i] += g;
      }
      sa += a[i];
      sx = fmaf(a[i], xhat[i], sx);
    }
    sa = team_sum<kTeam>(sa, red[0]) * inv;
    sx = team_sum<kTeam>(sx, red[1]) * inv;
    auto write = [&](auto out_bf16) {
      constexpr bool kOut = decltype(out_bf16)::value;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int c = i * kTeam + tid;
        if (c < C) {
          float o = rstd * (a[i] - sa - xhat[i] * sx);
          if (p.gres) o += shared_elem<kOut>(rs, c);
          store_elem(p.gx, kOut, t * p.ldgx + c, o);
        }
      }
    };
    if (p.gx_bf16)
      write(std::true_type{});
    else
      write(std::false_type{});
    if (tid == 0 && !(fabsf(sa) < INFINITY && fabsf(sx) < INFINITY))
      raise_flag(p.status, HLQ_DEV_NONFINITE);
    team_sync<kTeam>();  // the stage has been read by the whole team
    if (tid < 32) issue(t + plan.stages * step, stage);
    if (++stage == plan.stages) stage = 0, parity ^= 1;
  }
  if (tid == 0 && *(volatile int*)&abort_flag) ring_drain(ring.full, plan.stages, issued);
  if (!p.part) return;
  float* slab = p.part + (size_t)blockIdx.x * 2 * p.C;
  float* sums = plan.teams == 1 ? slab : reinterpret_cast<float*>(smem) + team * 2 * C;
  // every copy has been waited for by its team: the ring is free for the sums
  if (plan.teams > 1) __syncthreads();
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    const int c = i * kTeam + tid;
    if (c < C) sums[c] = gw[i], sums[C + c] = gb[i];
  }
  if (plan.teams == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * C; c += blockDim.x) {
    float s = 0.f;
    for (int k = 0; k < plan.teams; ++k) s += reinterpret_cast<float*>(smem)[k * 2 * C + c];
    slab[c] = s;
  }
}

// As norm_bwd_ring_plan, for rows of `stage` bytes in their slots; an SM holds
// 512 x ctas_each threads, and a CTA has `before` bytes before its rings.
bool elem_plan(int64_t T, int64_t C, int64_t stage, bool sums, int ctas_each, int64_t before,
               int sms, RingPlan* out) {
  if (sms <= 0 || C > 512 * kCols) return false;
  RingPlan r{};
  r.team = C <= 32 * kCols ? 32 : C <= 128 * kCols ? 128 : 512;
  const int per_sm = ctas_each * (r.team == 32 ? 1 : 512 / r.team);
  if (sums && sms * per_sm > kMostSlabs) sms = kMostSlabs / per_sm;
  r.smem_most = (size_t)(228 / per_sm - 1) * 1024 - 512;
  r.stage_bytes = (int)stage;
  const int64_t ctas_most = (int64_t)sms * per_sm, rows_each = (T + ctas_most - 1) / ctas_most;
  const int teams_most = elem_threads(r.team) / r.team;
  r.teams = (int)(rows_each < teams_most ? rows_each : teams_most);
  const int64_t ctas = (T + r.teams - 1) / r.teams;
  r.grid = (int)(ctas < ctas_most ? ctas : ctas_most);
  const int64_t rows = (T + (int64_t)r.grid * r.teams - 1) / ((int64_t)r.grid * r.teams);
  r.before = (int)((before + 15) / 16 * 16);
  const size_t fixed = 8 * 8 * r.teams + r.before;
  if (fixed > r.smem_most) return false;
  int64_t fit = (int64_t)(r.smem_most - fixed) / (stage * r.teams);
  if (fit > 8) fit = 8;
  r.stages = (int)(fit < rows ? fit : rows);
  if (r.stages < 1) return false;
  size_t ring = (size_t)r.stages * r.stage_bytes * r.teams;
  const size_t add = sums && r.teams > 1 ? ((size_t)C * 8 * r.teams + 15) / 16 * 16 : 0;
  if (ring < add) ring = add;
  r.smem = fixed + ring;
  *out = r;
  return r.smem <= r.smem_most;
}

template <auto kKernel, typename P>
cudaError_t go(const P& p, const RingPlan& r, cudaStream_t st) {
  const cudaError_t e = allow_smem<kKernel>(r.smem_most);
  if (e != cudaSuccess) return e;
  return launch_pdl(kKernel, dim3(r.grid), dim3(r.team * r.teams), r.smem, st, p, r);
}

template <bool kX>
cudaError_t pick_fwd(const NormFwd& p, const RingPlan& r, cudaStream_t st) {
  if (r.team == 32) return go<norm_fwd_elem_kernel<kX, 32>>(p, r, st);
  if (r.team == 128) return go<norm_fwd_elem_kernel<kX, 128>>(p, r, st);
  return go<norm_fwd_elem_kernel<kX, 512>>(p, r, st);
}
template <bool kX, bool kG>
cudaError_t pick_bwd(const NormBwd& p, const RingPlan& r, cudaStream_t st) {
  if (r.team == 32) return go<norm_bwd_elem_kernel<kX, kG, 32>>(p, r, st);
  if (r.team == 128) return go<norm_bwd_elem_kernel<kX, kG, 128>>(p, r, st);
  return go<norm_bwd_elem_kernel<kX, kG, 512>>(p, r, st);
}

}  // namespace

bool norm_fwd_elem_plan(const NormFwd& p, int sms, RingPlan* out) {
  const int64_t slot = slot_bytes(p.C * (p.x_bf16 ? 2 : 4));
  return elem_plan(p.T, p.C, slot * (p.residual ? 2 : 1), false, 2, p.C * 8, sms, out);
}
cudaError_t launch_norm_fwd_elem(const NormFwd& p, const RingPlan& r, cudaStream_t st) {
  return p.x_bf16 ? pick_fwd<true>(p, r, st) : pick_fwd<false>(p, r, st);
}

bool norm_bwd_elem_plan(const NormBwd& p, int sms, RingPlan* out) {
  const int64_t stage = slot_bytes(p.C * (p.x_bf16 ? 2 : 4)) + slot_bytes(p.C * (p.gy_bf16 ? 2 : 4)) +
                        (p.gres ? slot_bytes(p.C * (p.gx_bf16 ? 2 : 4)) : 0);
  return elem_plan(p.T, p.C, stage, p.part != nullptr, 1, 0, sms, out);
}
cudaError_t launch_norm_bwd_elem(const NormBwd& p, const RingPlan& r, cudaStream_t st) {
  return p.x_bf16 ? p.gy_bf16 ? pick_bwd<true, true>(p, r, st) : pick_bwd<true, false>(p, r, st)
                  : p.gy_bf16 ? pick_bwd<false, true>(p, r, st) : pick_bwd<false, false>(p, r, st);
}

}  // namespace hlq
