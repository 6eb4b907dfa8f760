// hlq_clip.cu -- the global norm of many gradients and their clipping
// (hlq_clip_grad_norm): norm = sqrt(sum over all elements of g^2),
// coef = min(1, max_norm / (norm + 1e-6)), out = coef g.
//
// The tensors' table travels as a kernel parameter: nothing is copied to the
// device beforehand, and a captured call replays with the addresses it was
// captured with.  The tensors are cut into chunks of 8192 elements; a CTA
// takes a run of consecutive chunks, and each of its threads 32 elements of a
// chunk, all loaded before the first is used.
//
// Bound by HBM: the gradients are read for the norm and again for the product,
// because no chip holds them in between (what L2 still holds is read first).
// 236 M fp32 gradients in 192 tensors, written as bf16 (2.36 GB in the two
// passes): 350 us, 1.01 of the measured copy rate; the bytes read once and
// written once would be 212 us.  A few small tensors take the time of two
// launches (9 us with the host's work for 24 of them).  54 M gradients written
// as bf16: 76 us, 89 where the outputs begin anywhere in a flat buffer (the ends
// of each warp's run are stored one by one).  Without the bound on registers the
// second pass takes 104 of them and two CTAs run on an SM: 81 and 111 us.
#include "hlq_device.cuh"
#include "hlq_kernels.h"
#include "hlq_rows.cuh"

namespace hlq {
namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;  // 64 registers a thread
constexpr int kQuads = kClipChunk / kThreads / 4;  // groups of four a thread

// The tensor that holds chunk `k` of the concatenation: the last one whose
// first chunk is <= k (tensors without elements are not in the table).
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

// A tensor's elements are taken in groups of four that are aligned in its
// input: the up to three elements before the first group go one by one with
// the tensor's first chunk, and chunk c holds the 8192 elements from
// head + 8192 c on.  Group (i, thread) of a chunk begins at its element
// place(i).
__device__ __forceinline__ int head_of(const void* p, bool bf16) {
  return (int)(4 - ((reinterpret_cast<uintptr_t>(p) >> (bf16 ? 1 : 2)) & 3)) & 3;
}
struct Chunk {
  int head;    // single elements before the tensor's first group
  int64_t e0;  // the chunk's first element
  int n;       // its elements; none where the head is all there is
};
__device__ __forceinline__ Chunk chunk_of(const ClipTable& tab, int i, int64_t k, bool bf16) {
  Chunk c;
  c.head = head_of(tab.in[i], bf16);
  c.e0 = c.head + (k - tab.first[i]) * kClipChunk;
  c.n = (int)max((int64_t)0, min((int64_t)kClipChunk, tab.numel[i] - c.e0));
  return c;
}
__device__ __forceinline__ int place(int i) { return (i * kThreads + (int)threadIdx.x) * 4; }

__device__ __forceinline__ void load_four(const void* in, bool bf16, int64_t e, float* v) {
  if (bf16) {
    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(in) + e);
    v[0] = bf16_lo(r.x), v[1] = bf16_hi(r.x), v[2] = bf16_lo(r.y), v[3] = bf16_hi(r.y);
  } else {
    const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(in) + e);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  }
}
__device__ __forceinline__ void store_four(void* out, bool bf16, int64_t e, const float* v) {
  if (bf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + e) =
        make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(out) + e) = make_float4(v[0], v[1], v[2], v[3]);
}

// This thread's groups of a chunk, zeros past its end.
__device__ __forceinline__ void load_chunk(const void* in, bool bf16, const Chunk& c,
                                           float (&v)[kQuads * 4]) {
  if (c.n == kClipChunk) {
    if (bf16) {
#pragma unroll
      for (int i = 0; i < kQuads; ++i) load_four(in, true, c.e0 + place(i), v + i * 4);
    } else {
#pragma unroll
      for (int i = 0; i < kQuads; ++i) load_four(in, false, c.e0 + place(i), v + i * 4);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      if (place(i) + 4 <= c.n) {
        load_four(in, bf16, c.e0 + place(i), v + i * 4);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[i * 4 + k] = place(i) + k < c.n ? load_elem(in, bf16, c.e0 + place(i) + k) : 0.f;
      }
    }
  }
}

// The same out again.  Where the output's groups of four begin `shift` elements
// after the input's, a warp's run of 128 elements is passed on by that many
// lanes' worth of values, so that all but its ends are still stored by fours.
__device__ __forceinline__ void store_chunk(void* out, bool bf16, const Chunk& c, int shift,
                                            const float (&v)[kQuads * 4]) {
  const int lane = threadIdx.x & 31;
  auto singly = [&](int i, int from, int to) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k >= from && k < to && place(i) + k < c.n)
        store_elem(out, bf16, c.e0 + place(i) + k, v[i * 4 + k]);
  };
  if (shift == 0 && c.n == kClipChunk) {
    if (bf16) {
#pragma unroll
      for (int i = 0; i < kQuads; ++i) store_four(out, true, c.e0 + place(i), v + i * 4);
    } else {
#pragma unroll
      for (int i = 0; i < kQuads; ++i) store_four(out, false, c.e0 + place(i), v + i * 4);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    if (shift == 0) {
      if (place(i) + 4 <= c.n)
        store_four(out, bf16, c.e0 + place(i), v + i * 4);
      else
        singly(i, 0, 4);
    } else if (place(i) - lane * 4 + 128 <= c.n) {  // the same for the whole warp
      float next[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) next[k] = __shfl_down_sync(0xffffffffu, v[i * 4 + k], 1);
      const float* a = v + i * 4;
      const float g[4] = {shift == 1 ? a[1] : shift == 2 ? a[2] : a[3],
                          shift == 1 ? a[2] : shift == 2 ? a[3] : next[0],
                          shift == 1 ? a[3] : shift == 2 ? next[0] : next[1],
                          shift == 1 ? next[0] : shift == 2 ? next[1] : next[2]};
      if (lane < 31)
        store_four(out, bf16, c.e0 + place(i) + shift, g);
      else
        singly(i, shift, 4);
      if (lane == 0) singly(i, 0, shift);
    } else {
      singly(i, 0, 4);
    }
  }
}

// Sums of squares in fp32 where that neither overflows nor loses small terms:
// a thread's 32 elements give between 2^-95 (any square that went below 2^-126
// is then beneath the sum's last bit) and 2^100.  Else, and that is rare, in
// fp64, which is slow here.  `sum` and `rest` are a running fp32 sum and what
// its roundings lost.
struct Squares {
  float sum = 0.f, rest = 0.f;
  double wide = 0.0;
  __device__ __forceinline__ void add(const float (&v)[kQuads * 4]) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kQuads * 4; ++i) s[i & 3] = fmaf(v[i], v[i], s[i & 3]);
    const float f = (s[0] + s[1]) + (s[2] + s[3]);
    if (f >= 0x1p-95f && f <= 0x1p100f) {
      const float y = f - rest, t = sum + y;
      rest = (t - sum) - y;
      sum = t;
      return;
    }
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kQuads * 4; ++i) any |= __float_as_uint(v[i]) << 1;
    if (any == 0) return;
#pragma unroll 1
    for (int i = 0; i < kQuads * 4; ++i) wide += square(v, i);
  }
  static __device__ __forceinline__ double square(const float (&v)[kQuads * 4], int i) {
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < kQuads * 4; ++k) x = k == i ? v[k] : x;
    return (double)x * x;
  }
};

// A CTA's partial result is the norm of its elements: an fp32 number wherever
// the whole norm is one.
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    clip_norm_kernel(const __grid_constant__ ClipTable tab, float* part) {
  __shared__ double red[kThreads / 32];
  pdl_wait();
  const int64_t k0 = tab.chunks * blockIdx.x / gridDim.x;
  const int64_t k1 = tab.chunks * (blockIdx.x + 1) / gridDim.x;
  int i = tensor_of(tab, k0);
  Squares sq;
  for (int64_t k = k0; k < k1; ++k) {
    if (i + 1 < tab.n && tab.first[i + 1] <= k) ++i;  // every tensor has a chunk
    const bool bf16 = tab.flags[i] & kClipInBf16;
    const Chunk c = chunk_of(tab, i, k, bf16);
    float v[kQuads * 4];
    load_chunk(tab.in[i], bf16, c, v);
    sq.add(v);
    if (c.head > 0 && k == tab.first[i]) {
      float h[kQuads * 4] = {};
      if ((int)threadIdx.x < c.head && threadIdx.x < tab.numel[i])
        h[0] = load_elem(tab.in[i], bf16, threadIdx.x);
      sq.add(h);
    }
  }
  // the warps' sums in fp32 (2^100 times all elements of a run could overflow
  // there, so above 2^100 in fp64 as well)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool wide = __syncthreads_or(sq.wide != 0.0 || sq.sum > 0x1p100f);
  float s = sq.sum - sq.rest;
  double d = 0.0;
  if (!wide) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) red[warp] = s;
  } else {
    d = sq.wide + (double)s;
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) red[warp] = d;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kThreads / 32; ++k) red[0] += red[k];
    part[blockIdx.x] = (float)sqrt(red[0]);
  }
}

// The coefficient from the CTAs' norms, in the first warp; with `write` it also
// writes norm and coefficient.
__device__ __forceinline__ float clip_coef(const ClipSums& q, bool write) {
  const int lane = threadIdx.x & 31;
  float top = 0.f, s = 0.f;
  bool nan = false;
#pragma unroll 8
  for (int i = lane; i < q.n; i += 32) {
    const float v = q.part[i];
    top = fmaxf(top, v);
    nan |= isnan(v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  nan = __any_sync(0xffffffffu, nan);
  float norm = nan ? NAN : top;  // 0 and infinity as they are
  if (!nan && top > 0.f && top < INFINITY) {
    // relative to a power of two near the largest: exact, and in range
    const int e = ilogbf(top);
#pragma unroll 8
    for (int i = lane; i < q.n; i += 32) {
      const float v = ldexpf(q.part[i], -e);
      s = fmaf(v, v, s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    norm = ldexpf(sqrtf(s), e);
  }
  float coef = q.max_norm / (norm + 1e-6f);
  // a NaN stays; without a limit an infinite norm clips nothing either
  coef = coef > 1.f || (q.max_norm == INFINITY && norm == INFINITY) ? 1.f : coef;
  if (write && lane == 0) {
    q.norm_coef[0] = norm;
    q.norm_coef[1] = coef;
    if (!isfinite(norm)) raise_flag(q.status, HLQ_DEV_NONFINITE);
  }
  return coef;
}

// The norm and the coefficient alone: one warp.
__global__ void __launch_bounds__(32) clip_coef_kernel(ClipSums q) {
  pdl_wait();
  clip_coef(q, true);
}

// The runs and their chunks in the opposite order of the norm's pass: what
// that pass read last is still in L2.  Each CTA adds the partial sums itself
// (a few thousand at most, from L2), which costs less than a launch between.
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    clip_scale_kernel(const __grid_constant__ ClipTable tab, const __grid_constant__ ClipSums q,
                      int first) {
  __shared__ float shared_coef;
  pdl_wait();
  if (threadIdx.x < 32) {
    const float c = clip_coef(q, first && blockIdx.x == 0);
    if (threadIdx.x == 0) shared_coef = c;
  }
  __syncthreads();
  const float coef = shared_coef;
  const int64_t k0 = tab.chunks * blockIdx.x / gridDim.x;
  const int64_t k1 = tab.chunks * (blockIdx.x + 1) / gridDim.x;
  if (k1 == k0) return;
  int i = tensor_of(tab, k1 - 1);
  for (int64_t k = k1 - 1; k >= k0; --k) {
    if (tab.first[i] > k) --i;
    const unsigned char fl = tab.flags[i];
    const bool in_bf16 = fl & kClipInBf16, out_bf16 = fl & kClipOutBf16;
    // in place, by a coefficient of 1: already there
    if (coef == 1.f && tab.in[i] == tab.out[i] && in_bf16 == out_bf16) continue;
    void* out = tab.out[i];
    const Chunk c = chunk_of(tab, i, k, in_bf16);
    float v[kQuads * 4];
    load_chunk(tab.in[i], in_bf16, c, v);
#pragma unroll
    for (int q = 0; q < kQuads * 4; ++q) v[q] *= coef;
    const int shift = (head_of(out, out_bf16) - c.head) & 3;
    store_chunk(out, out_bf16, c, shift, v);
    if ((int)threadIdx.x < c.head && k == tab.first[i] && threadIdx.x < tab.numel[i])
      store_elem(out, out_bf16, threadIdx.x, coef * load_elem(tab.in[i], in_bf16, threadIdx.x));
  }
}

}  // namespace

// kCtasPerSm CTAs an SM: 128 KB of loads in flight.  Neither pass
// lets the next kernel start before its own CTAs are done: CTAs of the second
// that came early would crowd on the SMs that the first left first, five on
// some and three on others (376 us instead of 356 for 236 M fp32 gradients).
int clip_grid(int64_t chunks, int sms) {
  const int64_t most = (int64_t)sms * kCtasPerSm;
  return (int)(chunks < 1 ? 1 : chunks < most ? chunks : most);
}

cudaError_t launch_clip_norm(const ClipTable& tab, float* part, int grid, cudaStream_t st) {
  return launch_pdl(clip_norm_kernel, dim3(grid), dim3(kThreads), 0, st, tab, part);
}

cudaError_t launch_clip_coef(const ClipSums& q, cudaStream_t st) {
  return launch_pdl(clip_coef_kernel, dim3(1), dim3(32), 0, st, q);
}

cudaError_t launch_clip_scale(const ClipTable& tab, const ClipSums& q, bool first, int grid,
                              cudaStream_t st) {
  return launch_pdl(clip_scale_kernel, dim3(grid), dim3(kThreads), 0, st, tab, q, first ? 1 : 0);
}

}  // namespace hlq
