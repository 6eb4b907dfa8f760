// hlq_attn_simt.cu -- attention and its backward pass on CUDA cores, in fp32:
// every type, head size up to 256, stride and alignment.  The tensor-core
// kernels take bf16 heads that TMA can read; the rest comes here.
//
//   s_ij = scale q_i . k_j          lse_i = log sum_j exp(s_ij)
//   out_i = sum_j exp(s_ij - lse_i) v_j
//   p_ij = exp(s_ij - lse_i)        delta_i = g_out_i . out_i
//   ds_ij = p_ij (g_out_i . v_j - delta_i)
//   g_q_i = scale sum_j ds_ij k_j,  g_k_j = scale sum_i ds_ij q_i,
//   g_v_j = sum_i p_ij g_out_i
//
// One CTA of 8 x 16 or 16 x 16 threads has a tile of rows (queries; keys in the keys'
// pass) in shared memory and goes over tiles of the other side.  Thread
// (ty, tx) has rows ty RM .., columns tx, tx + 16, .. of a tile of scores and
// columns 4 tx + 64 c .. (2 tx .. of 32) of a row of results, so that a row belongs
// to half a warp: maxima and sums are shuffles, and the probabilities go through
// shared memory without a barrier.  The backward pass goes over the keys' tiles
// (g_k, g_v) and over the queries' tiles (g_q) in CTAs of their own: two products
// more than one pass with atomics would take, and equal calls give equal bits.
//
// What bounds it is shared memory: a thread's 4 x 4 scores take 8 loads of 16 bytes
// for 64 multiplications, so a warp's loads (512 bytes each, whether lanes read
// the same or not) 32 clocks of the SM at 128 bytes a clock for 64 clocks of one of
// its four schedulers.  The multiplications fill half of their pipe (8 x 700 tokens,
// 6 heads of 64); 8 x 4 scores need so many registers that too few warps are left
// (64 rows, 128 threads, D 64 backward: 805 us against 769).  4 x 1024 tokens, 8
// heads: 34 TFLOP/s forward and 28 (of five products) backward for heads of 64, 32
// and 26 for heads of 128.  Above 128 the tile is that of 256 whatever the head's size:
// in bf16 1.6 ms forward (22 TFLOP/s for heads of 256, 11 for 136) and 5.9 backward
// (14, 8).
#include <cmath>

#include "hlq_attn.cuh"
#include "hlq_host.h"
#include "hlq_rows.cuh"

namespace hlq {
namespace {

// kT threads with a tile of BM rows of the CTA's own side, and BN of the other side;
// heads up to D, kC CTAs an SM.
template <int D, int BM, int BN, int kT, int kC>
struct Cfg {
  static constexpr int DP = D;
  static constexpr int kThreads = kT, kCtas = kC;
  static constexpr int kLd = DP + 4;  // floats: rows 4 banks apart
  static constexpr int kBM = BM, kBN = BN;
  static constexpr int kRM = kBM * 16 / kThreads, kRN = kBN / 16, kRD = DP / 16;
  static constexpr int kVec = DP == 32 ? 2 : 4;  // columns of a result together
  static constexpr int kLdP = kBN + 4;
  static constexpr size_t kFwd = 4 * (size_t)(kBM * kLd + 2 * kBN * kLd + kBM * kLdP);
  static constexpr size_t kBwd = 4 * (size_t)(2 * kBM * kLd + 2 * kBN * kLd + kBM * kLdP);
};

// Rows row0 .. row0 + n of head h as fp32, zeros in the rest of the tile.  By
// four where heads begin on 16-byte boundaries and are of whole fours.
template <class C>
__device__ __forceinline__ void load_tile(float* dst, const Heads& x, bool bf16, int64_t row0,
                                          int n, int rows, int h, int D) {
  constexpr int DP = C::DP;
  const int64_t at = row0 * x.token + (int64_t)h * x.head;
  if (D % 4 == 0 && reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && x.token % 4 == 0 &&
      x.head % 4 == 0) {
#pragma unroll 4
    for (int i = threadIdx.x; i < rows * DP / 4; i += C::kThreads) {
      const int r = i / (DP / 4), d = i % (DP / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < n && d < D) {
        if (bf16) {
          const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x.p) + at + r * x.token + d);
          v = make_float4(bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y));
        } else {
          v = *reinterpret_cast<const float4*>(static_cast<const float*>(x.p) + at + r * x.token + d);
        }
      }
      *reinterpret_cast<float4*>(dst + r * C::kLd + d) = v;
    }
    return;
  }
  for (int i = threadIdx.x; i < rows * DP; i += C::kThreads) {
    const int r = i / DP, d = i % DP;
    dst[r * C::kLd + d] =
        r < n && d < D ? load_elem(x.p, bf16, at + r * x.token + d) : 0.f;
  }
}

// acc[i][j] = A[row i] . B[row j], rows as in the note at the top.  Two fp32 in
// one instruction: the sums of the even and of the odd columns, added at the end.
template <class C, int RM, int RN>
__device__ __forceinline__ void rows_by_rows(const float* a, const float* b, int ty, int tx,
                                             float (&acc)[RM][RN]) {
  constexpr int kLd = C::kLd, DP = C::DP;
  F2 two[RM][RN];
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < RN; ++j) two[i][j] = f2(0.f);
#pragma unroll 4
  for (int d = 0; d < DP; d += 4) {
    ulonglong2 u[RM], w[RN];
#pragma unroll
    for (int i = 0; i < RM; ++i)
      u[i] = *reinterpret_cast<const ulonglong2*>(a + (ty * RM + i) * kLd + d);
#pragma unroll
    for (int j = 0; j < RN; ++j)
      w[j] = *reinterpret_cast<const ulonglong2*>(b + (tx + 16 * j) * kLd + d);
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
      for (int j = 0; j < RN; ++j)
        two[i][j] = fma2({u[i].y}, {w[j].y}, fma2({u[i].x}, {w[j].x}, two[i][j]));
  }
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < RN; ++j) {
      const float2 s = split(two[i][j]);
      acc[i][j] = s.x + s.y;
    }
}

// acc[i][V c + e] += sum_j P[row i][j] B[j][16 V c + V tx + e], V = kVec; acc by
// pairs of columns.
template <class C, int RM, int BN>
__device__ __forceinline__ void rows_by_columns(const float* P, const float* b, int ty, int tx,
                                                F2 (&acc)[RM][C::kRD / 2]) {
  constexpr int kLd = C::kLd, kLdP = BN + 4, kVec = C::kVec;
#pragma unroll 2
  for (int j = 0; j < BN; j += 4) {
    float p[RM][4];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(P + (ty * RM + i) * kLdP + j);
      p[i][0] = v.x, p[i][1] = v.y, p[i][2] = v.z, p[i][3] = v.w;
    }
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
      for (int c = 0; c < C::kRD / kVec; ++c) {
        const float* at = b + (j + jj) * kLd + 16 * kVec * c + kVec * tx;
        F2 v[kVec / 2];
        if constexpr (kVec == 4) {
          const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(at);
          v[0].b = w.x, v[1].b = w.y;
        } else {
          v[0].b = *reinterpret_cast<const unsigned long long*>(at);
        }
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
          for (int e = 0; e < kVec / 2; ++e)
            acc[i][kVec / 2 * c + e] = fma2(f2(p[i][jj]), v[e], acc[i][kVec / 2 * c + e]);
      }
  }
}

template <class C, int RM>
__device__ __forceinline__ void store_rows(const Heads& x, bool bf16, int64_t row0, int n, int h,
                                           int D, int ty, int tx, float factor,
                                           const F2 (&acc)[RM][C::kRD / 2]) {
  constexpr int kVec = C::kVec;
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int r = ty * RM + i;
    if (r >= n) continue;
    const int64_t at = (row0 + r) * x.token + (int64_t)h * x.head;
#pragma unroll
    for (int c = 0; c < C::kRD; c += 2) {
      const int d = 16 * kVec * (c / kVec) + kVec * tx + c % kVec;
      const float2 v = split(acc[i][c / 2]);
      if (d < D) store_elem(x.p, bf16, at + d, factor * v.x);
      if (d + 1 < D) store_elem(x.p, bf16, at + d + 1, factor * v.y);
    }
  }
}

template <class C, int RM>
__device__ __forceinline__ void clear(F2 (&acc)[RM][C::kRD / 2]) {
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int c = 0; c < C::kRD / 2; ++c) acc[i][c] = f2(0.f);
}

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas) attn_fwd_simt_kernel(const Attn p) {
  constexpr int BM = C::kBM, BN = C::kBN, RM = C::kRM, RN = C::kRN;
  extern __shared__ float smem[];
  float *sq = smem, *sk = sq + BM * C::kLd, *sv = sk + BN * C::kLd, *sp = sv + BN * C::kLd;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  pdl_wait();
  const uint32_t tile = blockIdx.x / p.by_hq;
  const int h = (int)(blockIdx.x - tile * p.Hq), hk = (int)((uint32_t)h / p.by_group);
  AttnTile t;
  const int past = find_tile<false, BM>(p, (int)tile, t);
  if (past >= 0) {  // rows of no sequence
    outside_rows<false>(p, BM, past, [&](int row, int d) {
      if (d == 0) p.lse[(int64_t)row * p.Hq + h] = -INFINITY;
      store_elem(p.out.p, p.bf16, row * p.out.token + h * p.out.head + d, 0.f);
    });
    return;
  }
  const int n = min(BM, t.nq - t.row0);
  const int keys = keys_of(p, t, t.row0 + n - 1);  // the last row sees the most
  load_tile<C>(sq, p.q, p.bf16, t.q0 + t.row0, n, BM, h, p.D);
  float m[RM], l[RM];
  F2 acc[RM][C::kRD / 2];
  clear<C, RM>(acc);
#pragma unroll
  for (int i = 0; i < RM; ++i) m[i] = -INFINITY, l[i] = 0.f;
  const float c2 = p.scale * kLog2e;
  for (int j0 = 0; j0 < keys; j0 += BN) {
    __syncthreads();  // the tiles before have been read
    const int nk = min(BN, keys - j0);
    load_tile<C>(sk, p.k, p.bf16, t.k0 + j0, nk, BN, hk, p.D);
    load_tile<C>(sv, p.v, p.bf16, t.k0 + j0, nk, BN, hk, p.D);
    __syncthreads();
    float s[RM][RN];
    rows_by_rows<C, RM, RN>(sq, sk, ty, tx, s);
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int sees = keys_of(p, t, t.row0 + ty * RM + i) - j0;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < RN; ++j) {
        s[i][j] = tx + 16 * j < sees ? s[i][j] * c2 : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
      top = fmaxf(m[i], half_warp_max(top));
      const float base = top == -INFINITY ? 0.f : top;  // nothing seen so far
      const float keep = exp2f(m[i] - base);
      m[i] = top;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < RN; ++j) {
        const float e = exp2f(s[i][j] - base);
        sum += e;
        sp[(ty * RM + i) * C::kLdP + tx + 16 * j] = e;
      }
      l[i] = l[i] * keep + half_warp_sum(sum);
#pragma unroll
      for (int c = 0; c < C::kRD / 2; ++c) acc[i][c] = acc[i][c] * f2(keep);
    }
    __syncwarp();
    rows_by_columns<C, RM, BN>(sp, sv, ty, tx, acc);
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // an empty row is zeros
#pragma unroll
    for (int c = 0; c < C::kRD / 2; ++c) acc[i][c] = acc[i][c] * f2(inv);
    const int r = ty * RM + i;
    if (tx == 0 && r < n)
      p.lse[(int64_t)(t.q0 + t.row0 + r) * p.Hq + h] =
          l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
  }
  store_rows<C, RM>(p.out, p.bf16, t.q0 + t.row0, n, h, p.D, ty, tx, 1.f, acc);
}

// delta = g_out . out (of g_out as bf16 where the products take it so: the gradients
// are then exactly those of the rounded g_out), and lse in units of log 2, both [Hq, Tq] (a tile's
// values are together); +infinity for a row that sees nothing, so that all its
// probabilities are 0.  With p.gout16 g_out rounded to bf16 as well.  What rows of
// no sequence give is used nowhere.
//
// kLanes lanes have eight of a row's elements each, 16 bytes (32) at a time, a
// warp has some heads of a token one after the other, and a CTA eight tokens,
// whose values it stores together: 44 us for 16384 tokens x 32 heads of 128 in bf16
// (268 MB: 0.9 of the copy rate), against 72 with the elements widened as they
// come (fewer CTAs an SM) and 97 with a warp on several tokens of one head.
template <bool kG, bool kO, int kLanes>
__global__ void __launch_bounds__(256) attn_bwd_rows_kernel(const Attn p) {
  constexpr int kRows = 4, kGroups = 32 / kLanes, kHeads = kRows * kGroups;
  __shared__ float all[2][kHeads][8 + 1];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, part = lane % kLanes;
  const uint32_t blocks = (p.Hq + kHeads - 1) / kHeads, group = blockIdx.x / blocks;
  const int h0 = (int)(blockIdx.x - group * blocks) * kHeads;
  const int64_t t0 = (int64_t)group * 8, t = t0 + warp;
  const bool here = t < p.Tq && 8 * part < p.D;
  // as they come, and all on their way before the first is widened
  uint4 g[kRows][kG ? 1 : 2], o[kRows][kO ? 1 : 2];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int h = h0 + r * kGroups + lane / kLanes;
    if (here && h < p.Hq) {
      const int64_t at = t * p.gout.token + h * p.gout.head + 8 * part;
      const int64_t ao = t * p.out.token + h * p.out.head + 8 * part;
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p.gout.p) + at * (kG ? 2 : 4));
      const uint4* u = reinterpret_cast<const uint4*>(static_cast<const char*>(p.out.p) + ao * (kO ? 2 : 4));
#pragma unroll
      for (int k = 0; k < (kG ? 1 : 2); ++k) g[r][k] = q[k];
#pragma unroll
      for (int k = 0; k < (kO ? 1 : 2); ++k) o[r][k] = u[k];
    }
  }
  if (lane < kHeads && t < p.Tq && h0 + lane < p.Hq) {
    const float lse = p.lse[t * p.Hq + h0 + lane];
    all[1][lane][warp] = lse == -INFINITY ? INFINITY : lse * kLog2e;
  }
  const auto floats = [](const uint4* v) {
    return join8(*reinterpret_cast<const float4*>(v), *reinterpret_cast<const float4*>(v + 1));
  };
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int h = h0 + r * kGroups + lane / kLanes;
    float sum = 0.f;
    if (here && h < p.Hq) {
      F8 a, b;
      if constexpr (kG) a = widen8(g[r][0]);
      else a = floats(g[r]);
      if constexpr (kO) b = widen8(o[r][0]);
      else b = floats(o[r]);
      if (!kG && p.gout16.p) {
        const int64_t at = t * p.gout16.token + h * p.gout16.head + 8 * part;
        store8(p.gout16.p, true, at, a);
#pragma unroll
        for (int k = 0; k < 8; ++k) a.v[k] = __bfloat162float(__float2bfloat16_rn(a.v[k]));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fmaf(a.v[k], b.v[k], sum);
    }
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (part == 0) all[0][r * kGroups + lane / kLanes][warp] = sum;
  }
  __syncthreads();
  const int i = threadIdx.x;
  if (i < kHeads * 8 && h0 + i / 8 < p.Hq && t0 + i % 8 < p.Tq) {
    const int64_t at = (int64_t)(h0 + i / 8) * p.Tq + t0 + i % 8;
    p.delta[at] = all[0][i / 8][i % 8];
    p.lse2[at] = all[1][i / 8][i % 8];
  }
}

// The same for any alignment: eight lanes have the elements of a row in turn.
__global__ void __launch_bounds__(256) attn_bwd_rows_any_kernel(const Attn p) {
  constexpr int kLanes = 8;
  pdl_trigger();
  pdl_wait();
  const int part = threadIdx.x % kLanes;
  const int64_t first = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
  const bool there = first < (int64_t)p.Tq * p.Hq;
  const int64_t t = there ? first / p.Hq : 0;
  const int h = there ? (int)(first - t * p.Hq) : 0;
  const int64_t go = t * p.gout.token + h * p.gout.head, oo = t * p.out.token + h * p.out.head;
  float sum = 0.f;
  if (there)
    for (int d = part; d < p.D; d += kLanes) {
      float g = load_elem(p.gout.p, p.gout_bf16, go + d);
      if (p.gout16.p) {
        store_elem(p.gout16.p, true, t * p.gout16.token + h * p.gout16.head + d, g);
        g = __bfloat162float(__float2bfloat16_rn(g));
      }
      sum = fmaf(g, load_elem(p.out.p, p.bf16, oo + d), sum);
    }
#pragma unroll
  for (int d = kLanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (there && part == 0) {
    const float lse = p.lse[first];
    p.delta[(int64_t)h * p.Tq + t] = sum;
    p.lse2[(int64_t)h * p.Tq + t] = lse == -INFINITY ? INFINITY : lse * kLog2e;
  }
}

// g_k and g_v of a tile of keys: over the query heads that share the key head
// and the tiles of queries that see it.  Rows are keys, columns queries.
template <class C>
__device__ __forceinline__ void keys_body(const Attn& p, uint32_t block) {
  constexpr int BM = C::kBM, BN = C::kBN, RM = C::kRM, RN = C::kRN;
  extern __shared__ float smem[];
  float *sk = smem, *sv = sk + BM * C::kLd, *sq = sv + BM * C::kLd, *sg = sq + BN * C::kLd,
        *sp = sg + BN * C::kLd;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  pdl_wait();
  const uint32_t tile = block / p.by_hk;
  const int hk = (int)(block - tile * p.Hk), group = p.group;
  AttnTile t;
  const int past = find_tile<true, BM>(p, (int)tile, t);
  if (past >= 0) {
    outside_rows<true>(p, BM, past, [&](int row, int d) {
      store_elem(p.gk.p, p.g_bf16, row * p.gk.token + hk * p.gk.head + d, 0.f);
      store_elem(p.gv.p, p.g_bf16, row * p.gv.token + hk * p.gv.head + d, 0.f);
    });
    return;
  }
  const int n = min(BM, t.nk - t.row0);
  load_tile<C>(sk, p.k, p.bf16, t.k0 + t.row0, n, BM, hk, p.D);
  load_tile<C>(sv, p.v, p.bf16, t.k0 + t.row0, n, BM, hk, p.D);
  F2 gk[RM][C::kRD / 2], gv[RM][C::kRD / 2];
  clear<C, RM>(gk);
  clear<C, RM>(gv);
  // the first query that sees the tile's first key
  const int first = p.causal ? max(0, t.row0 + (t.nq - t.nk)) / BN * BN : 0;
  const float c2 = p.scale * kLog2e;
  for (int h = hk * group; h < (hk + 1) * group; ++h)
    for (int i0 = first; i0 < t.nq; i0 += BN) {
      __syncthreads();
      const int nq = min(BN, t.nq - i0);
      load_tile<C>(sq, p.q, p.bf16, t.q0 + i0, nq, BN, h, p.D);
      load_tile<C>(sg, p.gout, p.gout_bf16, t.q0 + i0, nq, BN, h, p.D);
      __syncthreads();
      float s[RM][RN], dp[RM][RN];
      rows_by_rows<C, RM, RN>(sk, sq, ty, tx, s);
      rows_by_rows<C, RM, RN>(sv, sg, ty, tx, dp);
#pragma unroll
      for (int j = 0; j < RN; ++j) {
        const int i = i0 + tx + 16 * j;  // the query
        const bool there = i < t.nq;
        const int64_t at = (int64_t)h * p.Tq + t.q0 + i;
        const float lse2 = there ? ld_dep_f32(p.lse2 + at) : INFINITY;
        const float delta = there ? ld_dep_f32(p.delta + at) : 0.f;
        const int sees = there ? keys_of(p, t, i) - t.row0 : 0;
#pragma unroll
        for (int r = 0; r < RM; ++r) {
          const float e = ty * RM + r < sees ? exp2f(s[r][j] * c2 - lse2) : 0.f;
          sp[(ty * RM + r) * C::kLdP + tx + 16 * j] = e;
          dp[r][j] = ty * RM + r < sees ? e * (dp[r][j] - delta) : 0.f;
        }
      }
      __syncwarp();
      rows_by_columns<C, RM, BN>(sp, sg, ty, tx, gv);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < RN; ++j)
#pragma unroll
        for (int r = 0; r < RM; ++r) sp[(ty * RM + r) * C::kLdP + tx + 16 * j] = dp[r][j];
      __syncwarp();
      rows_by_columns<C, RM, BN>(sp, sq, ty, tx, gk);
      __syncwarp();
    }
  store_rows<C, RM>(p.gk, p.g_bf16, t.k0 + t.row0, n, hk, p.D, ty, tx, p.scale, gk);
  store_rows<C, RM>(p.gv, p.g_bf16, t.k0 + t.row0, n, hk, p.D, ty, tx, 1.f, gv);
}

// g_q of a tile of queries.
template <class C>
__device__ __forceinline__ void queries_body(const Attn& p, uint32_t block) {
  constexpr int BM = C::kBM, BN = C::kBN, RM = C::kRM, RN = C::kRN;
  extern __shared__ float smem[];
  float *sq = smem, *sg = sq + BM * C::kLd, *sk = sg + BM * C::kLd, *sv = sk + BN * C::kLd,
        *sd = sv + BN * C::kLd;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  pdl_wait();
  const uint32_t tile = block / p.by_hq;
  const int h = (int)(block - tile * p.Hq), hk = (int)((uint32_t)h / p.by_group);
  AttnTile t;
  const int past = find_tile<false, BM>(p, (int)tile, t);
  if (past >= 0) {
    outside_rows<false>(p, BM, past, [&](int row, int d) {
      store_elem(p.gq.p, p.g_bf16, row * p.gq.token + h * p.gq.head + d, 0.f);
    });
    return;
  }
  const int n = min(BM, t.nq - t.row0);
  const int keys = keys_of(p, t, t.row0 + n - 1);
  load_tile<C>(sq, p.q, p.bf16, t.q0 + t.row0, n, BM, h, p.D);
  load_tile<C>(sg, p.gout, p.gout_bf16, t.q0 + t.row0, n, BM, h, p.D);
  F2 gq[RM][C::kRD / 2];
  float lse2[RM], delta[RM];
  clear<C, RM>(gq);
#pragma unroll
  for (int r = 0; r < RM; ++r) {
    const bool there = ty * RM + r < n;
    const int64_t at = (int64_t)h * p.Tq + t.q0 + t.row0 + ty * RM + r;
    lse2[r] = there ? ld_dep_f32(p.lse2 + at) : INFINITY;
    delta[r] = there ? ld_dep_f32(p.delta + at) : 0.f;
  }
  const float c2 = p.scale * kLog2e;
  for (int j0 = 0; j0 < keys; j0 += BN) {
    __syncthreads();
    const int nk = min(BN, keys - j0);
    load_tile<C>(sk, p.k, p.bf16, t.k0 + j0, nk, BN, hk, p.D);
    load_tile<C>(sv, p.v, p.bf16, t.k0 + j0, nk, BN, hk, p.D);
    __syncthreads();
    float s[RM][RN], dp[RM][RN];
    rows_by_rows<C, RM, RN>(sq, sk, ty, tx, s);
    rows_by_rows<C, RM, RN>(sg, sv, ty, tx, dp);
#pragma unroll
    for (int r = 0; r < RM; ++r) {
      const int sees = keys_of(p, t, t.row0 + ty * RM + r) - j0;
#pragma unroll
      for (int j = 0; j < RN; ++j)
        sd[(ty * RM + r) * C::kLdP + tx + 16 * j] =
            tx + 16 * j < sees ? exp2f(s[r][j] * c2 - lse2[r]) * (dp[r][j] - delta[r]) : 0.f;
    }
    __syncwarp();
    rows_by_columns<C, RM, BN>(sd, sk, ty, tx, gq);
    __syncwarp();
  }
  store_rows<C, RM>(p.gq, p.g_bf16, t.q0 + t.row0, n, h, p.D, ty, tx, p.scale, gq);
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
    attn_bwd_simt_kernel(const Attn p, uint32_t keys_ctas) {
  if (blockIdx.x < keys_ctas)
    keys_body<C>(p, blockIdx.x);
  else
    queries_body<C>(p, blockIdx.x - keys_ctas);
}

template <class C>
cudaError_t launch_fwd(const Attn& p, cudaStream_t st) {
  const int64_t grid = most_tiles(p, false, C::kBM) * p.Hq;
  if (grid == 0) return cudaSuccess;
  cudaError_t e = allow_smem<attn_fwd_simt_kernel<C>>(C::kFwd);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_fwd_simt_kernel<C>, dim3((unsigned)grid), dim3(C::kThreads), C::kFwd,
                    st, p);
}

template <class C>
cudaError_t launch_bwd(const Attn& p, cudaStream_t st) {
  const int64_t keys = most_tiles(p, true, C::kBM) * p.Hk;
  const int64_t grid = keys + most_tiles(p, false, C::kBM) * p.Hq;
  if (grid == 0) return cudaSuccess;
  cudaError_t e = allow_smem<attn_bwd_simt_kernel<C>>(C::kBwd);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_bwd_simt_kernel<C>, dim3((unsigned)grid), dim3(C::kThreads), C::kBwd,
                    st, p, (uint32_t)keys);
}

template <bool kG, bool kO>
cudaError_t launch_rows(const Attn& p, cudaStream_t st) {
  const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32;
  const int64_t heads = 4 * (32 / lanes);
  const unsigned grid = (unsigned)((p.Tq + (int64_t)7) / 8 * ((p.Hq + heads - 1) / heads));
  return launch_pdl(lanes == 8    ? attn_bwd_rows_kernel<kG, kO, 8>
                    : lanes == 16 ? attn_bwd_rows_kernel<kG, kO, 16>
                                  : attn_bwd_rows_kernel<kG, kO, 32>,
                    dim3(grid), dim3(256), 0, st, p);
}

}  // namespace

// Tiles by head size.  Forward: 32 rows and 128 threads, three or four CTAs an SM.
// Against 64 rows and 256 threads (D 32: 32 by 32 and 256), four sequences, 8 heads:
// D 32 1024 tokens 148 us against 263, 400 tokens 32 against 52; D 64 254 against
// 267, 50 against 62; D 128 532 against 548, 95 against 116.
cudaError_t launch_attn_simt(const Attn& p, cudaStream_t st) {
  return p.D <= 32    ? launch_fwd<Cfg<32, 32, 64, 128, 4>>(p, st)
         : p.D <= 64  ? launch_fwd<Cfg<64, 32, 64, 128, 3>>(p, st)
         : p.D <= 128 ? launch_fwd<Cfg<128, 32, 32, 128, 3>>(p, st)
                      : launch_fwd<Cfg<256, 32, 32, 256, 1>>(p, st);
}

// Backward: 64 rows and 256 threads where that leaves three CTAs for each SM or more, else
// as forward: D 64 4 x 1024 tokens (8 heads) 769 us against 854, 5 x 129 (6 heads) 50
// against 43; D 128 1671 against 1805, 87 against 71.  D up to 32: as forward, but
// where all CTAs of 32 rows run at once each has 256 threads and 32 columns
// (4 x 1024 719 against 456, 5 x 129 23.7 against 29.9).
cudaError_t launch_attn_bwd_simt(const Attn& p, cudaStream_t st) {
  const auto ctas = [&](int rows) {
    return most_tiles(p, true, rows) * p.Hk + most_tiles(p, false, rows) * p.Hq;
  };
  const int64_t sms = device_sm_count();
  if (p.D <= 32)
    return ctas(32) <= 2 * sms ? launch_bwd<Cfg<32, 32, 32, 256, 2>>(p, st)
                               : launch_bwd<Cfg<32, 32, 64, 128, 4>>(p, st);
  if (p.D <= 64)
    return ctas(64) < 3 * sms ? launch_bwd<Cfg<64, 32, 64, 128, 3>>(p, st)
                              : launch_bwd<Cfg<64, 64, 64, 256, 2>>(p, st);
  if (p.D <= 128)
    return ctas(64) < 3 * sms ? launch_bwd<Cfg<128, 32, 32, 128, 3>>(p, st)
                              : launch_bwd<Cfg<128, 64, 32, 256, 2>>(p, st);
  return launch_bwd<Cfg<256, 32, 32, 256, 1>>(p, st);
}

cudaError_t launch_attn_bwd_rows(const Attn& p, cudaStream_t st) {
  const int64_t rows = (int64_t)p.Tq * p.Hq;
  if (rows == 0) return cudaSuccess;
  const auto wide = [&](const Heads& x, bool bf16) {  // rows of whole 16 bytes
    const int64_t per = bf16 ? 8 : 4;
    return p.D % 8 == 0 && reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && x.token % per == 0 &&
           x.head % per == 0;
  };
  if (wide(p.gout, p.gout_bf16) && wide(p.out, p.bf16)) {
    return p.gout_bf16 ? (p.bf16 ? launch_rows<true, true>(p, st) : launch_rows<true, false>(p, st))
                       : (p.bf16 ? launch_rows<false, true>(p, st) : launch_rows<false, false>(p, st));
  }
  return launch_pdl(attn_bwd_rows_any_kernel, dim3((unsigned)((rows + 31) / 32)), dim3(256), 0, st,
                    p);
}

}  // namespace hlq
