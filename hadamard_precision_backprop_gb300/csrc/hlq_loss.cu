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
//
// A row is cut into 1, 2, 4 or 8 slices; 256 threads take a slice, each up to
// 64 elements in groups of 16, which it holds in registers, and keep a running
// maximum and the sum of exp(z - maximum).  These pairs are joined over the
// warp, the slice's warps and the slices, always in the same order: a token's
// log-probability has the same bits whatever the number of rows and in both
// operators, so that the ratio of an unchanged policy is exactly 1.  (The groups
// are aligned in memory: a row at another offset from 16 bytes has others.)
//   policy loss: a cluster of CTAs, one for a slice, joins the slices through
//     distributed shared memory; the gradient is computed from the registers,
//     so that the row is read once;
//   log-probabilities: the same where there are few rows, else one CTA takes
//     all slices of its rows one after another, the loads of the next slice
//     under way while one is summed.
//
// Bound by HBM, and next to that by latency: a CTA's loads, its sums, the
// cluster's barrier, the row's few scalars (in one warp, 7 waiting) and its
// stores follow one another, and only the other CTAs of the SM fill the gaps.
// Policy loss 4096 x 128256 bf16 with a quarter of the rows masked (1.84 GB) 315
// us, 0.87 of the measured copy rate; 1000 x 50021 (175 MB) 41 us, 0.64 (ramp
// and tail, some 17 instructions an element).  Every row counted: 2048 x 128256
// fp32 (2.1 GB) 370 us, 0.85; 2048 x 151936 bf16, read twice (1.24 GB without
// that), 246 us, 0.76; 4096 x 128256 bf16 without a gradient (1.05 GB) 255 us,
// 0.62.  Log-probabilities 2048 x 32003 fp32 (262 MB) 40 us, 0.99; 4096 x 128256
// bf16 239 us, 0.66 (half as many bytes a register in flight).  With one pass
// over 64 loaded elements for the maximum and one for the sum, and clusters
// everywhere, the two masked cases took 416 and 54, these 99 and 254.
#include <cfloat>
#include <type_traits>

#include "hlq_device.cuh"
#include "hlq_host.h"
#include "hlq_kernels.h"
#include "hlq_rows.cuh"
#include "hlq_tma.cuh"

namespace hlq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kGroups = 4;                          // groups of 16 elements a thread holds
constexpr int kMostSlices = 8;
constexpr int kSliceElems = kThreads * kGroups * 16;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// sum_i exp2(c z_i) as exp2(c m) s with m the maximum (-FLT_MAX and 0 before
// the first term: then no difference below is -inf + inf).
// Eight-byte aligned: clusters store it as one pair.
struct alignas(8) MaxSum {
  float m, s;
};
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
  const float m = fmaxf(a.m, b.m);
  // no fma: join(a, b) and join(b, a) are the same bits
  return {m, __fadd_rn(__fmul_rn(a.s, ex2((a.m - m) * c)), __fmul_rn(b.s, ex2((b.m - m) * c)))};
}

// One slice of a row: `n` 16-byte vectors from element `e0` of the row, and
// for slice 0 the up to 2 x 7 single elements before the first and after the
// last vector of the row (thread j < 8: element j, j >= 8: the (j - 8)th after
// the vectors).
template <bool kBf16>
struct Slice {
  static constexpr int kSize = kBf16 ? 2 : 4, kVec = 16 / kSize;
  static constexpr int kGroup = 16 / kVec;  // vectors of a group
  const char* row;
  int e0, n;  // V is below 2^31
  int edge;   // this thread's single element, -1: none
  __device__ __forceinline__ Slice(const void* base, int64_t offset, int V, int slice,
                                   int log_slices) {
    row = static_cast<const char*>(base) + offset * kSize;
    const int phase = (int)(reinterpret_cast<uintptr_t>(row) & 15);
    const int head = min((16 - phase) % 16 / kSize, V);
    const int vecs = (V - head) / kVec, per = (vecs + (1 << log_slices) - 1) >> log_slices;
    const int v0 = min(slice * per, vecs);
    n = min(per, vecs - v0);
    e0 = head + v0 * kVec;
    edge = -1;
    if (slice == 0 && threadIdx.x < 16) {
      const int j = threadIdx.x, after = head + vecs * kVec + j - 8;
      if (j < 8 ? j < head : after < V) edge = j < 8 ? j : after;
    }
  }
  // This thread's vectors of the group that begins at vector j; -inf past the
  // slice's end.  (A branch that spares whole groups the comparison keeps the
  // groups' loads from going out together: 323 -> 352 us at 4096 x 128256.)
  static constexpr int kStep = kGroup * kThreads;  // vectors of a group of all threads
  __device__ __forceinline__ void load(int j, uint4 (&raw)[kGroup]) const {
    const uint4* at = reinterpret_cast<const uint4*>(row + (int64_t)e0 * kSize) + (j + (int)threadIdx.x);
    constexpr uint32_t none = kBf16 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      raw[i] = j + i * kThreads + (int)threadIdx.x < n ? at[i * kThreads]
                                                       : make_uint4(none, none, none, none);
  }
  __device__ __forceinline__ float elem(int64_t e) const { return load_elem(row, kBf16, e); }
};

template <bool kBf16>
__device__ __forceinline__ void widen(uint4 r, F2* v) {
  if constexpr (kBf16) {
    v[0] = widen2(r.x), v[1] = widen2(r.y), v[2] = widen2(r.z), v[3] = widen2(r.w);
  } else {
    v[0] = f2(__uint_as_float(r.x), __uint_as_float(r.y));
    v[1] = f2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The largest of a group.
template <bool kBf16>
__device__ __forceinline__ float max_of(const uint4 (&r)[Slice<kBf16>::kGroup]) {
  if constexpr (kBf16) {
    const uint32_t a = max_bf16x2(max_bf16x2(r[0].x, r[0].y), max_bf16x2(r[0].z, r[0].w));
    const uint32_t b = max_bf16x2(max_bf16x2(r[1].x, r[1].y), max_bf16x2(r[1].z, r[1].w));
    const uint32_t m = max_bf16x2(a, b);
    return fmaxf(bf16_lo(m), bf16_hi(m));
  } else {
    float m = __uint_as_float(r[0].x);
#pragma unroll
    for (int i = 0; i < Slice<kBf16>::kGroup; ++i)
      m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(r[i].x)),
                      fmaxf(__uint_as_float(r[i].y), __uint_as_float(r[i].z))),
                __uint_as_float(r[i].w));
    return m;
  }
}

// The running pair of a thread, the sum in two halves.
struct Running {
  float m = -FLT_MAX;
  F2 s = f2(0.f);
  // One group of 16.  The difference to the maximum comes first, so that the
  // maximum itself counts exactly 1.
  template <bool kBf16>
  __device__ __forceinline__ void add(const uint4 (&raw)[Slice<kBf16>::kGroup], float c) {
    using S = Slice<kBf16>;
    const float top = fmaxf(m, max_of<kBf16>(raw));
    s = s * f2(ex2((m - top) * c));
    const F2 neg = f2(-top), c2 = f2(c);
#pragma unroll
    for (int i = 0; i < S::kGroup; ++i) {
      F2 v[S::kVec / 2];
      widen<kBf16>(raw[i], v);
#pragma unroll
      for (int k = 0; k < S::kVec / 2; ++k) {
        const float2 d = split((v[k] + neg) * c2);
        s = s + f2(ex2(d.x), ex2(d.y));
      }
    }
    m = top;
  }
  __device__ __forceinline__ MaxSum pair() const {
    const float2 h = split(s);
    return {m, h.x + h.y};
  }
};

// The pairs of kLanes neighbouring lanes joined, the same in each: the maximum
// first, then the sums relative to it.
template <int kLanes>
__device__ __forceinline__ MaxSum lanes_pair(MaxSum p, float c) {
  float m = p.m;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = p.s * ex2((p.m - m) * c);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return {m, s};
}

// The CTA's pair, in its first warp; `warp_pair` may be written again after
// the next __syncthreads but one.
__device__ __forceinline__ MaxSum cta_pair(MaxSum p, bool has_edge, float edge, float c,
                                           MaxSum* warp_pair) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (has_edge) {
    const float m = fmaxf(edge, -FLT_MAX);
    p = join(p, {m, ex2((edge - m) * c)}, c);
  }
  p = lanes_pair<32>(p, c);
  if (lane == 0) warp_pair[tid >> 5] = p;
  __syncthreads();
  if (tid < 32) p = lanes_pair<kWarps>(warp_pair[lane % kWarps], c);
  return p;
}

// The row's pair, in the first warp of every CTA of the cluster (whose threads
// have all called cluster_started_arrive).
__device__ __forceinline__ MaxSum cluster_pair(MaxSum p, float c, int slice, int log_slices,
                                               MaxSum* slots) {
  if (log_slices == 0) return p;
  __syncwarp();
  cluster_started_wait();
  static_assert(sizeof(MaxSum) == 8 && alignof(MaxSum) == 8, "one aligned 8-byte store");
  if ((int)threadIdx.x < (1 << log_slices)) {
    const uint32_t at = cluster_map(saddr(slots + slice), threadIdx.x);
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(p.m), "f"(p.s)
                 : "memory");
  }
  __syncwarp();
  cluster_sync();
  p = slots[0];
  for (int i = 1; i < (1 << log_slices); ++i) p = join(p, slots[i], c);
  return p;
}

// A CTA's part of a cluster's row.  kHeld: the slice stays in `raw`;
// otherwise `raw` is filled again and again.
template <bool kBf16, bool kHeld>
__device__ __forceinline__ MaxSum slice_pair(
    const Slice<kBf16>& sl, float c, uint4 (&raw)[kGroups][Slice<kBf16>::kGroup], float& edge,
    MaxSum* warp_pair) {
  using S = Slice<kBf16>;
  edge = sl.edge >= 0 ? sl.elem(sl.edge) : 0.f;
  Running run;
  for (int b = 0; b < (kHeld ? 1 : sl.n); b += kGroups * S::kStep) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) sl.load(b + g * S::kStep, raw[g]);
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
      if (b + g * S::kStep < sl.n) run.add<kBf16>(raw[g], c);
  }
  return cta_pair(run.pair(), sl.edge >= 0, edge, c, warp_pair);
}

__device__ __forceinline__ float token_logp(float logit, MaxSum p, float scale) {
  return scale * (logit - p.m) - logf(p.s);
}

__device__ __forceinline__ void write_logprob(const TokenLogprobs& p, int64_t t, int64_t a,
                                              float logit, MaxSum pair) {
  const bool known = a >= 0 && a < p.V;
  p.logp[t] = known ? token_logp(logit, pair, p.scale) : NAN;
  const float lse = p.scale * pair.m + logf(pair.s);
  if (p.lse) p.lse[t] = lse;
  if (!known) raise_flag(p.status, HLQ_DEV_BADCODE);
  if (!isfinite(lse)) raise_flag(p.status, HLQ_DEV_NONFINITE);
}

// exp(scale d) = exp2(c d); no infinity, which a difference of 0 would make NaN.
__device__ __forceinline__ float log2_scale(float scale) {
  return fminf(scale * 1.4426950408889634f, FLT_MAX);
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) logprobs_cluster_kernel(TokenLogprobs p,
                                                                    int log_slices) {
  using S = Slice<kBf16>;
  __shared__ MaxSum warp_pair[kWarps], slots[kMostSlices];
  const int slice = blockIdx.x & ((1 << log_slices) - 1);
  const int64_t t = blockIdx.x >> log_slices;
  const float c = log2_scale(p.scale);
  pdl_wait();
  pdl_trigger();
  if (log_slices) cluster_started_arrive();
  const S sl(p.logits, t * p.ld, (int)p.V, slice, log_slices);
  int64_t a = -1;
  float logit = 0.f;
  if (slice == 0 && threadIdx.x == 0) {
    a = p.targets[t];
    if (a >= 0 && a < p.V) logit = sl.elem(a);
  }
  uint4 raw[kGroups][S::kGroup];
  float edge;
  MaxSum pair = slice_pair<kBf16, false>(sl, c, raw, edge, warp_pair);
  pair = cluster_pair(pair, c, slice, log_slices, slots);
  if (slice == 0 && threadIdx.x == 0) write_logprob(p, t, a, logit, pair);
}

// One CTA a row, slice after slice.  A group's registers are loaded with the
// next slice's (or row's) elements as soon as the group is summed.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads, kBf16 ? 3 : 2)
    logprobs_stream_kernel(TokenLogprobs p, int log_slices) {
  using S = Slice<kBf16>;
  __shared__ MaxSum warp_pair[2][kWarps];
  const float c = log2_scale(p.scale);
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  int64_t t = blockIdx.x;
  if (t >= p.T) return;
  int slice = 0, flip = 0;
  S sl(p.logits, t * p.ld, (int)p.V, 0, log_slices);
  int b = 0;
  uint4 raw[kGroups][S::kGroup];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) sl.load(g * S::kStep, raw[g]);
  float edge = sl.edge >= 0 ? sl.elem(sl.edge) : 0.f;
  int64_t a = -1;
  float logit = 0.f;
  Running run;
  MaxSum row = {-FLT_MAX, 0.f};
  while (true) {
    if (tid == 0 && slice == 0 && b == 0) {
      a = p.targets[t];
      logit = a >= 0 && a < p.V ? sl.elem(a) : 0.f;
    }
    // what comes after these groups: more of the slice, a slice, a row, nothing
    const bool slice_ends = b + kGroups * S::kStep >= sl.n;
    const bool row_ends = slice_ends && slice + 1 == 1 << log_slices;
    const int64_t t_next = row_ends ? t + gridDim.x : t;
    const int slice_next = row_ends ? 0 : slice_ends ? slice + 1 : slice;
    const int b_next = slice_ends ? 0 : b + kGroups * S::kStep;
    const bool more = t_next < p.T;
    S next = sl;
    if (slice_ends && more) next = S(p.logits, t_next * p.ld, (int)p.V, slice_next, log_slices);
    float edge_next = edge;
    if (slice_ends && more && next.edge >= 0) edge_next = next.elem(next.edge);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (b + g * S::kStep < sl.n) run.add<kBf16>(raw[g], c);
      if (more) next.load(b_next + g * S::kStep, raw[g]);
    }
    if (slice_ends) {
      const MaxSum pair = cta_pair(run.pair(), sl.edge >= 0, edge, c, warp_pair[flip]);
      flip ^= 1;
      row = slice == 0 ? pair : join(row, pair, c);
      run = Running();
      if (row_ends && tid == 0) write_logprob(p, t, a, logit, row);
    }
    if (!more) break;
    sl = next, edge = edge_next, t = t_next, slice = slice_next, b = b_next;
  }
}

// What the first warp hands to its CTA: the gradient -coef p_v is
// exp2((z - m) c) k except at the action.  The difference comes first, as in the
// sum: the product m c of a huge logit has no place for what z c adds to it.
struct RowGrad {
  float neg_m, k, at_action;
  int64_t action;
};

template <bool kBf16>
__device__ __forceinline__ uint4 narrow(const F2* v) {
  if constexpr (kBf16) {
    return make_uint4(pack_bf16(v[0]), pack_bf16(v[1]), pack_bf16(v[2]), pack_bf16(v[3]));
  } else {
    const float2 a = split(v[0]), b = split(v[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                      __float_as_uint(b.y));
  }
}

// kHeld: the slice is kept in registers between the two passes, else (rows of
// more than 8 x 16384 elements) read again.  Five CTAs an SM for bf16, in 48 registers
// with 16 to 32 bytes spilled: 320 us at 4096 x 128256 where four took 325.
// kAligned: g's rows begin at the same offset from a 16-byte boundary as the
// logits'; else g is written element by element.
template <bool kBf16, bool kHeld, bool kAligned>
__global__ void __launch_bounds__(kThreads, kBf16 ? 5 : 2)
    policy_rows_kernel(const __grid_constant__ PolicyLoss p, int log_slices) {
  using S = Slice<kBf16>;
  __shared__ MaxSum warp_pair[kWarps], slots[kMostSlices];
  __shared__ RowGrad grad;
  const int slice = blockIdx.x & ((1 << log_slices) - 1);
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x >> log_slices;
  const float c = log2_scale(p.scale);
  pdl_wait();
  pdl_trigger();
  const float w = p.weight[t];
  const S sl(p.logits, t * p.ld, (int)p.V, slice, log_slices);
  char* g = static_cast<char*>(p.g) + t * p.ldg * S::kSize;
  auto put = [&](int j, const F2* v) {
    const int64_t e = sl.e0 + (int64_t)j * S::kVec;
    if constexpr (kAligned) {
      reinterpret_cast<uint4*>(g + (int64_t)sl.e0 * S::kSize)[j] = narrow<kBf16>(v);
    } else {
#pragma unroll
      for (int k = 0; k < S::kVec / 2; ++k) {
        const float2 x = split(v[k]);
        store_elem(g, kBf16, e + 2 * k, x.x);
        store_elem(g, kBf16, e + 2 * k + 1, x.y);
      }
    }
  };
  if (w == 0.f) {  // the same for the whole cluster
    if (p.g) {
      const F2 zero[S::kVec / 2] = {};
      for (int j = tid; j < sl.n; j += kThreads) put(j, zero);
      if (sl.edge >= 0) store_elem(g, kBf16, sl.edge, 0.f);
    }
    if (slice == 0 && tid == 0) {
      p.part[t] = p.part[p.T + t] = p.part[2 * p.T + t] = 0.f;
      if (p.logp) p.logp[t] = 0.f;
    }
    return;
  }
  if (log_slices) cluster_started_arrive();
  int64_t a = -1;
  float logit = 0.f, old = 0.f, adv = 0.f, ref = 0.f;
  if (tid < 32) {
    a = p.actions[t];
    old = p.old_logp[t], adv = p.advantage[t];
    if (p.ref_logp) ref = p.ref_logp[t];
    if (a >= 0 && a < p.V) logit = sl.elem(a);
  }
  uint4 raw[kGroups][S::kGroup];
  float edge;
  MaxSum pair = slice_pair<kBf16, kHeld>(sl, c, raw, edge, warp_pair);
  pair = cluster_pair(pair, c, slice, log_slices, slots);
  if (tid < 32) {
    const bool known = a >= 0 && a < p.V;
    const float lp = known ? token_logp(logit, pair, p.scale) : NAN;
    const float r = expf(lp - old), inner = r * adv;
    const float outer = fminf(fmaxf(r, 1.f - p.clip_low), 1.f + p.clip_high) * adv;
    const bool clipped = outer < inner;
    const float pg = clipped ? -outer : -inner;
    float dlp = clipped ? 0.f : -inner, kl = 0.f;
    if (p.ref_logp) {
      const float d = ref - lp, e = expm1f(d);
      kl = e - d;
      if (p.kl_coef != 0.f) dlp -= p.kl_coef * e;
    }
    const float coef = w * dlp * p.grad_scale * p.scale;
    if (tid == 0) {
      grad = {-pair.m, -coef / pair.s, -coef * expm1f(lp), a};
      if (slice == 0) {
        p.part[t] = w * pg;
        p.part[p.T + t] = w * kl;
        p.part[2 * p.T + t] = clipped ? w : 0.f;
        if (p.logp) p.logp[t] = lp;
        if (!known) raise_flag(p.status, HLQ_DEV_BADCODE);
        if (!isfinite(coef)) raise_flag(p.status, HLQ_DEV_NONFINITE);
      }
    }
  }
  if (!p.g) return;
  __syncthreads();
  const RowGrad gr = grad;
  const F2 c2 = f2(c), neg = f2(gr.neg_m), k2 = f2(gr.k);
  auto gradient = [&](uint4 r, F2* v) {
    widen<kBf16>(r, v);
#pragma unroll
    for (int k = 0; k < S::kVec / 2; ++k) {
      const float2 x = split((v[k] + neg) * c2);
      v[k] = f2(ex2(x.x), ex2(x.y)) * k2;
    }
  };
  for (int b = 0; b < (kHeld ? 1 : sl.n); b += kGroups * S::kStep) {
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const int j = b + q * S::kStep;
      if constexpr (!kHeld) sl.load(j, raw[q]);
#pragma unroll
      for (int i = 0; i < S::kGroup; ++i) {
        if (j + i * kThreads + tid < sl.n) {
          F2 v[S::kVec / 2];
          gradient(raw[q][i], v);
          put(j + i * kThreads + tid, v);
        }
      }
    }
  }
  if (sl.edge >= 0) store_elem(g, kBf16, sl.edge, ex2((edge + gr.neg_m) * c) * gr.k);
  // the action's element, by the thread that has just written it
  const int64_t e = gr.action - sl.e0;
  const bool mine = e >= 0 && e < (int64_t)sl.n * S::kVec ? (int)(e / S::kVec) % kThreads == tid
                                                          : gr.action >= 0 && gr.action == sl.edge;
  if (mine) store_elem(g, kBf16, gr.action, gr.at_action);
}

// stats = sums over the rows in a fixed order (in fp32: a tree over 1024
// partial sums; fp64 is far slower here than all the rest of this kernel).  One
// CTA, whose time is the latency of its loads, so each thread has twelve of
// them under way.
constexpr int kStatsThreads = 1024;

__global__ void __launch_bounds__(kStatsThreads) policy_stats_kernel(PolicyLoss p) {
  __shared__ float red[3][kStatsThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  float s[3] = {0.f, 0.f, 0.f};
  for (int64_t t = tid; t < p.T; t += 4 * kStatsThreads) {
    float v[3][4];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t r = t + i * kStatsThreads;
        v[k][i] = r < p.T ? p.part[k * p.T + r] : 0.f;
      }
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] += (v[k][0] + v[k][1]) + (v[k][2] + v[k][3]);
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    if (lane == 0) red[k][warp] = s[k];
  }
  __syncthreads();
  if (warp > 0) return;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    s[k] = red[k][lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  }
  if (lane == 0) {
    p.stats[0] = p.ref_logp && p.kl_coef != 0.f ? fmaf(p.kl_coef, s[1], s[0]) : s[0];
    p.stats[1] = s[0];
    p.stats[2] = s[1];
    p.stats[3] = s[2];
  }
}

// The slices of a row: as many (a power of two, 8 at most) as threads hold.
int row_slices_log(int64_t V) {
  int n = 0;
  while ((1 << n) < kMostSlices && V > ((int64_t)kSliceElems << n)) ++n;
  return n;
}

template <typename P>
cudaError_t launch_clusters(void (*kernel)(P, int), const P& p, int log_slices, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.T << log_slices));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1 << log_slices;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = log_slices ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, log_slices);
}

}  // namespace

int64_t loss_most_rows(int64_t V) { return (((int64_t)1 << 31) - 1) >> row_slices_log(V); }

cudaError_t launch_token_logprobs(const TokenLogprobs& p, cudaStream_t st) {
  const int log_slices = row_slices_log(p.V), sms = device_sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  const int64_t ctas = (int64_t)sms * (p.bf16 ? 3 : 2);
  if (p.T < ctas)
    return launch_clusters(p.bf16 ? logprobs_cluster_kernel<true> : logprobs_cluster_kernel<false>,
                           p, log_slices, st);
  return launch_pdl(p.bf16 ? logprobs_stream_kernel<true> : logprobs_stream_kernel<false>,
                    dim3((unsigned)ctas), dim3(kThreads), 0, st, p, log_slices);
}

cudaError_t launch_policy_rows(const PolicyLoss& p, cudaStream_t st) {
  const int log_slices = row_slices_log(p.V);
  const bool held = p.V <= (int64_t)kSliceElems << log_slices;
  const uint64_t size = p.bf16 ? 2 : 4;
  const bool aligned =
      (reinterpret_cast<uintptr_t>(p.g) - reinterpret_cast<uintptr_t>(p.logits)) % 16 == 0 &&
      (p.T <= 1 || (uint64_t)(p.ldg - p.ld) * size % 16 == 0);
  auto pick = [&](auto b) {
    constexpr bool kB = decltype(b)::value;
    return held ? aligned ? policy_rows_kernel<kB, true, true> : policy_rows_kernel<kB, true, false>
                : aligned ? policy_rows_kernel<kB, false, true>
                          : policy_rows_kernel<kB, false, false>;
  };
  return launch_clusters(p.bf16 ? pick(std::true_type{}) : pick(std::false_type{}), p, log_slices,
                         st);
}

cudaError_t launch_policy_stats(const PolicyLoss& p, cudaStream_t st) {
  return launch_pdl(policy_stats_kernel, dim3(1), dim3(kStatsThreads), 0, st, p);
}

}  // namespace hlq
