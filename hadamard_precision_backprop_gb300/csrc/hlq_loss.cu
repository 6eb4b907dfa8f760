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
// A cluster of 1 to 8 CTAs holds a row in registers, 64 elements a thread:
// the row is read once, each thread takes the maximum of its elements and the
// sum of exp(z - maximum), these pairs are joined over the warp, the CTA and
// (through distributed shared memory) the cluster, and the gradient is
// computed from the registers and written.  The split depends on the row's
// length and alignment alone, not on the number of rows or on the operator: a
// token's log-probability has the same bits in both, so that the ratio of an
// unchanged policy is exactly 1.
#include <type_traits>

#include "hlq_device.cuh"
#include "hlq_kernels.h"
#include "hlq_rows.cuh"
#include "hlq_tma.cuh"

namespace hlq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kHeld = 64;                      // elements a thread holds
constexpr int kMostCtas = 8;
constexpr int kCtaElems = kThreads * kHeld;    // elements a CTA holds

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// sum_i exp2(c z_i) as exp2(c m) s, m the maximum (-inf: nothing yet).
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float fa = a.m == m ? 1.f : ex2((a.m - m) * c);
  const float fb = b.m == m ? 1.f : ex2((b.m - m) * c);
  return {m, a.s * fa + b.s * fb};
}

// exp2(c (z - m)) as exp2(fma(z, c, bias)) * fix: bias = -(c m) rounded, fix
// the exact rest of that product, so that one fma a term loses nothing.
struct ExpArg {
  float bias, fix;
};
__device__ __forceinline__ ExpArg exp_arg(float m, float c) {
  const float bias = -(m * c);
  return {bias, ex2(-fmaf(m, c, bias))};
}

// One CTA's part of a row: `n` 16-byte vectors from element `e0` of the row,
// and on the first CTA the up to 2 x 7 single elements before the first and
// after the last vector of the row (thread j < 8: element j, j >= 8: the
// (j - 8)th after the vectors).
template <bool kBf16>
struct Slice {
  static constexpr int kVec = kBf16 ? 8 : 4, kNum = kHeld / kVec;
  const char* row;
  int64_t e0;
  int n;
  int64_t edge;  // this thread's single element; -1: none
  __device__ __forceinline__ Slice(const void* base, int64_t offset, int64_t V, int rank, int ctas) {
    constexpr int kSize = kBf16 ? 2 : 4;
    row = static_cast<const char*>(base) + offset * kSize;
    int64_t head = (16 - (reinterpret_cast<uintptr_t>(row) & 15)) % 16 / kSize;
    if (head > V) head = V;
    const int64_t vecs = (V - head) / kVec, per = (vecs + ctas - 1) / ctas;
    const int64_t v0 = min(rank * per, vecs), v1 = min(v0 + per, vecs);
    e0 = head + v0 * kVec;
    n = (int)(v1 - v0);
    edge = -1;
    if (rank == 0 && threadIdx.x < 16) {
      const int64_t j = threadIdx.x, after = head + vecs * kVec + j - 8;
      if (j < 8 ? j < head : after < V) edge = j < 8 ? j : after;
    }
  }
  __device__ __forceinline__ const uint4* vec(int i) const {
    return reinterpret_cast<const uint4*>(row + e0 * (kBf16 ? 2 : 4)) + i;
  }
  __device__ __forceinline__ float elem(int64_t e) const { return load_elem(row, kBf16, e); }
};

template <bool kBf16>
__device__ __forceinline__ void widen(uint4 r, float* v) {
  if constexpr (kBf16) {
    const F8 f = widen8(r);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = f.v[k];
  } else {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
}

// The CTA's pair over its slice, in thread 0's warp.  With kResident the
// slice fits the registers `raw`; otherwise they are reused block by block.
template <bool kBf16, bool kResident>
__device__ __forceinline__ MaxSum slice_pair(const Slice<kBf16>& sl, float c, uint4* raw,
                                             float& edge, MaxSum* warp_pair) {
  using S = Slice<kBf16>;
  const int tid = threadIdx.x, lane = tid & 31;
  MaxSum p = {-INFINITY, 0.f};
  edge = -INFINITY;
  if (sl.edge >= 0) edge = sl.elem(sl.edge);
  for (int b = 0; b < (kResident ? 1 : sl.n); b += S::kNum * kThreads) {
#pragma unroll
    for (int i = 0; i < S::kNum; ++i) {
      const int j = b + i * kThreads + tid;
      if (j < sl.n) raw[i] = *sl.vec(j);
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < S::kNum; ++i) {
      if (b + i * kThreads + tid < sl.n) {
        float v[S::kVec];
        widen<kBf16>(raw[i], v);
#pragma unroll
        for (int k = 0; k < S::kVec; ++k) m = fmaxf(m, v[k]);
      }
    }
    // the difference first: the maximum itself counts exactly 1
    const float top = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < S::kNum; ++i) {
      if (b + i * kThreads + tid < sl.n) {
        float v[S::kVec];
        widen<kBf16>(raw[i], v);
#pragma unroll
        for (int k = 0; k < S::kVec; ++k) s += ex2((v[k] - top) * c);
      }
    }
    p = kResident ? MaxSum{m, s} : join(p, {m, s}, c);
  }
  if (sl.edge >= 0) p = join(p, {edge, edge == -INFINITY ? 0.f : ex2((edge - edge) * c)}, c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    p = join(p, {__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o)}, c);
  if (lane == 0) warp_pair[tid >> 5] = p;
  __syncthreads();
  if (tid < 32) {
    p = warp_pair[lane % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1)
      p = join(p, {__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o)}, c);
  }
  return p;
}

// The row's pair, in the first warp of every CTA of the cluster.
__device__ __forceinline__ MaxSum row_pair(MaxSum p, float c, int rank, int ctas, MaxSum* slots) {
  if (ctas == 1) return p;
  if ((int)threadIdx.x < ctas) {
    const uint32_t at = cluster_map(saddr(slots + rank), threadIdx.x);
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(p.m), "f"(p.s)
                 : "memory");
  }
  cluster_sync();
  p = slots[0];
  for (int i = 1; i < ctas; ++i) p = join(p, slots[i], c);
  return p;
}

__device__ __forceinline__ float token_logp(float logit, MaxSum p, float scale) {
  return scale * (logit - p.m) - logf(p.s);
}

template <bool kBf16, bool kResident>
__global__ void __launch_bounds__(kThreads, kBf16 ? 3 : 2) token_logprobs_kernel(TokenLogprobs p, int ctas) {
  __shared__ MaxSum warp_pair[kWarps], slots[kMostCtas];
  const int rank = ctas > 1 ? (int)cluster_rank() : 0;
  const int64_t t = blockIdx.x / ctas;
  const float c = p.scale * 1.4426950408889634f;
  pdl_wait();
  const Slice<kBf16> sl(p.logits, t * p.ld, p.V, rank, ctas);
  int64_t a = -1;
  float logit = 0.f;
  if (rank == 0 && threadIdx.x == 0) {
    a = p.targets[t];
    if (a >= 0 && a < p.V) logit = sl.elem(a);
  }
  uint4 raw[Slice<kBf16>::kNum];
  float edge;
  MaxSum pair = slice_pair<kBf16, kResident>(sl, c, raw, edge, warp_pair);
  pair = row_pair(pair, c, rank, ctas, slots);
  pdl_trigger();
  if (rank == 0 && threadIdx.x == 0) {
    const bool known = a >= 0 && a < p.V;
    p.logp[t] = known ? token_logp(logit, pair, p.scale) : NAN;
    const float lse = p.scale * pair.m + logf(pair.s);
    if (p.lse) p.lse[t] = lse;
    if (!known) raise_flag(p.status, HLQ_DEV_BADCODE);
    if (!isfinite(lse)) raise_flag(p.status, HLQ_DEV_NONFINITE);
  }
}

// What the first warp hands to its CTA: p_v = exp2(fma(z, c, bias)) * k, and
// the gradient -coef p_v except at the action.
struct RowGrad {
  float bias, k, at_action;
  int64_t action;
};

template <bool kBf16>
__device__ __forceinline__ uint4 narrow(const float* v) {
  if constexpr (kBf16)
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                      pack_bf16(v[6], v[7]));
  else
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
}

// g's rows begin at the same offset from a 16-byte boundary as the logits'
// (kAligned), or are written element by element.
template <bool kBf16, bool kResident, bool kAligned>
__global__ void __launch_bounds__(kThreads, kBf16 ? 3 : 2) policy_rows_kernel(PolicyLoss p, int ctas) {
  using S = Slice<kBf16>;
  __shared__ MaxSum warp_pair[kWarps], slots[kMostCtas];
  __shared__ RowGrad grad;
  const int rank = ctas > 1 ? (int)cluster_rank() : 0;
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x / ctas;
  const float c = p.scale * 1.4426950408889634f;
  pdl_wait();
  const float w = p.weight[t];
  const S sl(p.logits, t * p.ld, p.V, rank, ctas);
  char* g = static_cast<char*>(p.g) + t * p.ldg * (kBf16 ? 2 : 4);
  auto put = [&](int j, const float* v) {
    const int64_t e = sl.e0 + (int64_t)j * S::kVec;
    if constexpr (kAligned) {
      *reinterpret_cast<uint4*>(g + e * (kBf16 ? 2 : 4)) = narrow<kBf16>(v);
    } else {
#pragma unroll
      for (int k = 0; k < S::kVec; ++k) store_elem(g, kBf16, e + k, v[k]);
    }
  };
  if (w == 0.f) {  // the same for the whole cluster
    if (p.g) {
      float zero[S::kVec] = {};
      for (int j = tid; j < sl.n; j += kThreads) put(j, zero);
      if (sl.edge >= 0) store_elem(g, kBf16, sl.edge, 0.f);
    }
    if (rank == 0 && tid == 0) {
      p.part[t] = p.part[p.T + t] = p.part[2 * p.T + t] = 0.f;
      if (p.logp) p.logp[t] = 0.f;
    }
    return;
  }
  int64_t a = -1;
  float logit = 0.f, old = 0.f, adv = 0.f, ref = 0.f;
  if (tid < 32) {
    a = p.actions[t];
    old = p.old_logp[t], adv = p.advantage[t];
    if (p.ref_logp) ref = p.ref_logp[t];
    if (a >= 0 && a < p.V) logit = sl.elem(a);
  }
  uint4 raw[S::kNum];
  float edge;
  MaxSum pair = slice_pair<kBf16, kResident>(sl, c, raw, edge, warp_pair);
  pair = row_pair(pair, c, rank, ctas, slots);
  pdl_trigger();
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
      const ExpArg x = exp_arg(pair.m, c);
      grad = {x.bias, -coef * (x.fix / pair.s), -coef * expm1f(lp), a};
      if (rank == 0) {
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
  for (int b = 0; b < (kResident ? 1 : sl.n); b += S::kNum * kThreads) {
    if constexpr (!kResident) {
#pragma unroll
      for (int i = 0; i < S::kNum; ++i) {
        const int j = b + i * kThreads + tid;
        if (j < sl.n) raw[i] = *sl.vec(j);
      }
    }
#pragma unroll
    for (int i = 0; i < S::kNum; ++i) {
      const int j = b + i * kThreads + tid;
      if (j < sl.n) {
        float v[S::kVec];
        widen<kBf16>(raw[i], v);
#pragma unroll
        for (int k = 0; k < S::kVec; ++k) v[k] = ex2(fmaf(v[k], c, gr.bias)) * gr.k;
        put(j, v);
      }
    }
  }
  if (sl.edge >= 0) store_elem(g, kBf16, sl.edge, ex2(fmaf(edge, c, gr.bias)) * gr.k);
  // the action's element, by the thread that has just written it
  const int64_t e = gr.action - sl.e0;
  const bool mine = e >= 0 && e < (int64_t)sl.n * S::kVec ? (int)(e / S::kVec) % kThreads == tid
                                                          : gr.action >= 0 && gr.action == sl.edge;
  if (mine) store_elem(g, kBf16, gr.action, gr.at_action);
}

// stats = sums over the rows in a fixed order, in fp64.
__global__ void __launch_bounds__(kThreads) policy_stats_kernel(PolicyLoss p) {
  __shared__ double red[3][kThreads];
  pdl_wait();
  for (int k = 0; k < 3; ++k) {
    double s = 0.0;
    for (int64_t t = threadIdx.x; t < p.T; t += kThreads) s += ld_dep_f32(p.part + k * p.T + t);
    red[k][threadIdx.x] = s;
  }
  for (int o = kThreads / 2; o > 0; o >>= 1) {
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

// CTAs of a row: as many (a power of two) as hold it in registers, 8 at most.
int row_ctas(int64_t V) {
  int n = 1;
  while (n < kMostCtas && V > (int64_t)n * kCtaElems) n *= 2;
  return n;
}

template <typename P>
cudaError_t launch_rows(void (*kernel)(P, int), const P& p, int ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.T * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p, ctas);
}

}  // namespace

int64_t loss_most_rows(int64_t V) { return (((int64_t)1 << 31) - 1) / row_ctas(V); }

cudaError_t launch_token_logprobs(const TokenLogprobs& p, cudaStream_t st) {
  const int ctas = row_ctas(p.V);
  const bool resident = p.V <= (int64_t)ctas * kCtaElems;
  return launch_rows(p.bf16 ? resident ? token_logprobs_kernel<true, true>
                                       : token_logprobs_kernel<true, false>
                            : resident ? token_logprobs_kernel<false, true>
                                       : token_logprobs_kernel<false, false>,
                     p, ctas, st);
}

cudaError_t launch_policy_rows(const PolicyLoss& p, cudaStream_t st) {
  const int ctas = row_ctas(p.V);
  const bool resident = p.V <= (int64_t)ctas * kCtaElems;
  const uint64_t size = p.bf16 ? 2 : 4;
  const bool aligned =
      (reinterpret_cast<uintptr_t>(p.g) - reinterpret_cast<uintptr_t>(p.logits)) % 16 == 0 &&
      (p.T <= 1 || (uint64_t)(p.ldg - p.ld) * size % 16 == 0);
  auto pick = [&](auto b) {
    constexpr bool kB = decltype(b)::value;
    return resident ? aligned ? policy_rows_kernel<kB, true, true> : policy_rows_kernel<kB, true, false>
                    : aligned ? policy_rows_kernel<kB, false, true>
                              : policy_rows_kernel<kB, false, false>;
  };
  return launch_rows(p.bf16 ? pick(std::true_type{}) : pick(std::false_type{}), p, ctas, st);
}

cudaError_t launch_policy_stats(const PolicyLoss& p, cudaStream_t st) {
  return launch_pdl(policy_stats_kernel, dim3(1), dim3(kThreads), 0, st, p);
}

}  // namespace hlq
