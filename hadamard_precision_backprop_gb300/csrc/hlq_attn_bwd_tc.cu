// hlq_attn_bwd_tc.cu -- attention's backward pass in bf16 on the tensor cores
// (tcgen05, TMEM, TMA), heads up to 128.
//
// Two kernels, so that every gradient is summed in one place in a fixed order
// (seven products of a tile of queries and one of keys where five with atomics
// would do):
//
// Keys: a CTA has a tile of 128 keys of a key head and goes over the tiles of
// queries of all query heads that share it.  Rows are keys, columns queries:
//   S' = K Q^T, D' = V G^T (TMEM, fp32)
//   P' = exp2(c S' - lse2), dS' = P' (D' - delta), bf16, in their places
//   g_v += P' G, g_k += dS' Q (TMEM, fp32; P' and dS' are read from TMEM)
// lse2 and delta belong to columns: a warp brings them into shared memory.
//
// Queries: a CTA has a tile of 128 queries of a head and goes over the keys:
//   S = Q K^T, D = G V^T, dS = P (D - delta), g_q += dS K
//
// In both, warps 4 to 11 compute: a thread has a row, warps 4-7 the first 64
// columns and warps 8-11 the others.  The products for one tile run while the
// probabilities of another are computed.
#include <cmath>

#include "hlq_attn_tc.cuh"
#include "hlq_rows.cuh"

namespace hlq {
namespace {

using namespace tc;

constexpr int kThreads = 384;

// 64 columns of this thread's row.
__device__ __forceinline__ void ld64(uint32_t at, uint32_t (&r)[2][32]) {
  ld32(at, r[0]);
  ld32(at + 32, r[1]);
  ld_wait(r[0]);
  ld_wait(r[1]);
}

// A row of a result, `factor` times the fp32 sums.  With `wide` rows are of
// whole 16 bytes.
template <int DP>
__device__ __forceinline__ void store_row(const Heads& x, bool bf16, int wide, int64_t row, int h,
                                          int D, bool there, uint32_t acc, bool zero,
                                          float factor) {
  const int64_t at = row * x.token + (int64_t)h * x.head;
#pragma unroll
  for (int c = 0; c < DP / 32; ++c) {
    uint32_t o[32];
    if (zero) {
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = 0;
    } else {
      __syncwarp();
      ld32(acc + 32 * c, o);
      ld_wait(o);
    }
    if (!there) continue;
    if (wide) {
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        F8 v;
#pragma unroll
        for (int k = 0; k < 8; ++k) v.v[k] = factor * __uint_as_float(o[i + k]);
        if (32 * c + i < D) store8(x.p, bf16, at + 32 * c + i, v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (32 * c + i < D)
          store_elem(x.p, bf16, at + 32 * c + i, factor * __uint_as_float(o[i]));
    }
  }
}

// ---------------------------------------------------------------------------
// Keys
// ---------------------------------------------------------------------------
template <int DP>
struct KeysCfg {
  static constexpr int kChunks = DP / kChunk;
  static constexpr uint32_t kTile = kChunks * kChunkBytes;
  static constexpr int kStages = DP == 64 ? 4 : 2;  // of Q and of G each
  static constexpr int kStats = 2;                  // of lse2 and delta
  static constexpr size_t kSmem =
      1024 + (size_t)(2 + 2 * kStages) * kTile + kStats * 2 * kRows * 4 + 512;
  static constexpr uint32_t kS = 0, kD = 128, kV = 256, kK = 256 + DP, kColumns = 512;
};

struct KeysBars {
  uint64_t kv_full, q_full[4], q_ready[4], q_empty[4], g_full[4], g_ready[4], g_empty[4],
      stat_full[2], stat_empty[2], s_full, p_full, d_full, ds_full, acc_full, drained;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(KeysBars) <= 512, "barriers fit their 512 bytes");

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_keys_tc_kernel(const Attn p, const __grid_constant__ CUtensorMap mq,
                            const __grid_constant__ CUtensorMap mk,
                            const __grid_constant__ CUtensorMap mv,
                            const __grid_constant__ CUtensorMap mg, int wide_k, int wide_v) {
  using C = KeysCfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t *sk = smem, *sv = sk + C::kTile, *sq = sv + C::kTile, *sg = sq + C::kStages * C::kTile;
  float* stats = reinterpret_cast<float*>(sg + C::kStages * C::kTile);  // [kStats][2][128]
  KeysBars& bar = *reinterpret_cast<KeysBars*>(stats + C::kStats * 2 * kRows);
  volatile int* abort_flag = &bar.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bar.kv_full, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bar.q_full[s], 1);
      mbar_init(&bar.q_ready[s], 1);
      mbar_init(&bar.q_empty[s], 1);
      mbar_init(&bar.g_full[s], 1);
      mbar_init(&bar.g_ready[s], 1);
      mbar_init(&bar.g_empty[s], 1);
    }
    for (int s = 0; s < C::kStats; ++s) {
      mbar_init(&bar.stat_full[s], 1);
      mbar_init(&bar.stat_empty[s], 8);
    }
    mbar_init(&bar.s_full, 1);
    mbar_init(&bar.p_full, 8);
    mbar_init(&bar.d_full, 1);
    mbar_init(&bar.ds_full, 8);
    mbar_init(&bar.acc_full, 1);
    mbar_init(&bar.drained, 1);
    bar.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 1) alloc(&bar.tmem, C::kColumns);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem, 0);
  pdl_trigger();
  pdl_wait();

  const int hk = blockIdx.x % p.Hk, group = p.Hq / p.Hk;
  AttnTile t;
  const int past = find_tile<true>(p, kRows, blockIdx.x / p.Hk, t);
  const auto wait = [&](uint64_t* b, uint32_t phase) {
    return wait_for(b, phase, abort_flag, p.status);
  };
  // tiles of queries of a head: from the one with the first query that sees the
  // tile's first key
  int first = 0, per_head = 0;
  if (past < 0) {
    if (p.causal) first = max(0, t.row0 + t.nq - t.nk) / kRows;
    per_head = max(0, (t.nq + kRows - 1) / kRows - first);
  }
  const int n = per_head * group;
  // rows of a head's last tile, if it is not full
  const int rest = t.nq % kRows;
  const auto head_of = [&](int it) { return hk * group + it / per_head; };
  const auto tile_of = [&](int it) { return first + it % per_head; };

  if (past >= 0) {
    outside_rows<true>(p, kRows, past, threadIdx.x, kThreads, [&](int row) {
      for (int d = 0; d < p.D; ++d) {
        store_elem(p.gk.p, p.g_bf16, row * p.gk.token + hk * p.gk.head + d, 0.f);
        store_elem(p.gv.p, p.g_bf16, row * p.gv.token + hk * p.gv.head + d, 0.f);
      }
    });
  } else if (warp < 4) {
    fewer_registers<72>();
    if (warp == 0) {
      if (lane == 0 && n > 0) {
        int q_done = 0, g_done = 0;
        mbar_expect_tx(&bar.kv_full, 2 * C::kTile);
        load_tile<C::kChunks>(sk, &mk, &bar.kv_full, hk, t.k0 + t.row0);
        load_tile<C::kChunks>(sv, &mv, &bar.kv_full, hk, t.k0 + t.row0);
        for (int it = 0; it < n; ++it) {
          const int s = it % C::kStages, use = it / C::kStages;
          const int row = t.q0 + tile_of(it) * kRows, h = head_of(it);
          if (use > 0 && !wait(&bar.q_empty[s], use - 1)) break;
          mbar_expect_tx(&bar.q_full[s], C::kTile);
          load_tile<C::kChunks>(sq + s * C::kTile, &mq, &bar.q_full[s], h, row);
          ++q_done;
          if (use > 0 && !wait(&bar.g_empty[s], use - 1)) break;
          mbar_expect_tx(&bar.g_full[s], C::kTile);
          load_tile<C::kChunks>(sg + s * C::kTile, &mg, &bar.g_full[s], h, row);
          ++g_done;
        }
        if (*abort_flag) {
          ring_drain(&bar.kv_full, 1, 1);
          ring_drain(bar.q_full, C::kStages, q_done);
          ring_drain(bar.g_full, C::kStages, g_done);
        }
      }
    } else if (warp == 1) {  // the whole warp, of which one thread issues
      const int steps = (p.D + 15) / 16;
      const uint32_t id = idesc(16 * steps, true);
      const uint32_t ak = by_columns(saddr(sk)), av = by_columns(saddr(sv));
      const uint32_t aq = by_columns(saddr(sq)), ag = by_columns(saddr(sg));
      const uint32_t rq = by_rows(saddr(sq)), rg = by_rows(saddr(sg));
      constexpr uint32_t kStep = C::kTile >> 4;
      bool ok = n > 0 && wait(&bar.kv_full, 0);
      const auto scores = [&](int it) {
        const int s = it % C::kStages;
        ok = wait(&bar.q_ready[s], it / C::kStages);
        if (!ok) return;
        fence_after();
        if (elect_one()) {
          product_of_rows<DP / 16>(tmem + C::kS, ak, aq + s * kStep, steps);
          commit(&bar.s_full);
        }
        __syncwarp();
      };
      const auto gradients = [&](int it) {
        const int s = it % C::kStages;
        ok = wait(&bar.g_ready[s], it / C::kStages);
        if (!ok) return;
        fence_after();
        if (elect_one()) {
          product_of_rows<DP / 16>(tmem + C::kD, av, ag + s * kStep, steps);
          commit(&bar.d_full);
        }
        __syncwarp();
      };
      if (ok) scores(0);
      if (ok) gradients(0);
      for (int it = 0; it < n && ok; ++it) {
        const int s = it % C::kStages;
        const bool reused = it + C::kStages < n;
        ok = wait(&bar.p_full, it);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          product_of_p<64>(tmem + C::kV, tmem + C::kS, rg + s * kStep, id, it > 0);
          if (reused) commit(&bar.g_empty[s]);
        }
        __syncwarp();
        if (it + 1 < n) scores(it + 1);
        if (ok) ok = wait(&bar.ds_full, it);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          product_of_p<64>(tmem + C::kK, tmem + C::kD, rq + s * kStep, id, it > 0);
          if (reused) commit(&bar.q_empty[s]);
        }
        __syncwarp();
        if (it + 1 < n) gradients(it + 1);
      }
      if (n > 0 && elect_one()) {
        if (ok)
          commit(&bar.acc_full);
        else
          drain(&bar.drained);
      }
      __syncwarp();
    } else if (warp == 2) {  // clears the rows behind the sequence's end
      for (int it = 0; it < n; ++it) {
        const int s = it % C::kStages, use = it / C::kStages;
        const bool cut = rest && it % per_head == per_head - 1;
        if (!__all_sync(0xffffffffu, wait(&bar.q_full[s], use))) break;
        if (cut) clear_rows<C::kChunks>(sq + s * C::kTile, rest);
        if (lane == 0) mbar_arrive(&bar.q_ready[s]);
        if (!__all_sync(0xffffffffu, wait(&bar.g_full[s], use))) break;
        if (cut) clear_rows<C::kChunks>(sg + s * C::kTile, rest);
        if (lane == 0) mbar_arrive(&bar.g_ready[s]);
      }
    } else {  // lse2 and delta of the tiles' queries; what is behind the end has P = 0
      for (int it = 0; it < n; ++it) {
        const int s = it % C::kStats, use = it / C::kStats;
        if (use > 0 && !__all_sync(0xffffffffu, wait(&bar.stat_empty[s], use - 1))) break;
        const int i0 = tile_of(it) * kRows;
        const int64_t at = (int64_t)head_of(it) * p.Tq + t.q0 + i0;
        float* to = stats + s * 2 * kRows;
        float v[2][kRows / 32];  // all on their way before the first is stored
#pragma unroll
        for (int i = 0; i < kRows / 32; ++i) {
          const bool there = i0 + 32 * i + lane < t.nq;
          v[0][i] = there ? ld_dep_f32(p.lse2 + at + 32 * i + lane) : INFINITY;
          v[1][i] = there ? ld_dep_f32(p.delta + at + 32 * i + lane) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kRows / 32; ++i) {
          to[32 * i + lane] = v[0][i];
          to[kRows + 32 * i + lane] = v[1][i];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.stat_full[s]);
      }
    }
  } else {
    more_registers<216>();
    const int half = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane, key = t.row0 + r;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + C::kS + lanes + 64 * half, td = tmem + C::kD + lanes + 64 * half;
    const float c2 = p.scale * kLog2e;
    const F2 c22 = f2(c2), minus = f2(-1.f);
    // the first query that sees this row's key, and the tile's last key
    const int from = p.causal ? key + t.nq - t.nk : 0;
    const int last_from = p.causal ? t.row0 + kRows - 1 + t.nq - t.nk : 0;
    bool ok = true;
    for (int it = 0; it < n; ++it) {
      const int s = it % C::kStats;
      const float* lse2 = stats + s * 2 * kRows + 64 * half;
      const int i0 = tile_of(it) * kRows + 64 * half;
      ok = wait(&bar.stat_full[s], it / C::kStats) && wait(&bar.s_full, it);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      fence_after();
      uint32_t x[2][32];
      ld64(ts, x);
      if (i0 < last_from) {  // some row does not see some column
        const int skip = from - i0;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i < skip) x[c][i] = 0xff800000u;
      }
      float prob[64];
      uint32_t e[32];
#pragma unroll
      for (int i = 0; i < 64; i += 4) {
        const float4 l = *reinterpret_cast<const float4*>(lse2 + i);
        const uint32_t(&v)[32] = x[i / 32];
        const int k = i % 32;
        const float2 a = split(fma2(f2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), c22, f2(l.x, l.y) * minus));
        const float2 b = split(fma2(f2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), c22, f2(l.z, l.w) * minus));
        prob[i] = exp2_fast(a.x), prob[i + 1] = exp2_fast(a.y);
        prob[i + 2] = exp2_fast(b.x), prob[i + 3] = exp2_fast(b.y);
        e[i / 2] = bf16x2(prob[i], prob[i + 1]);
        e[i / 2 + 1] = bf16x2(prob[i + 2], prob[i + 3]);
      }
      st32(ts, e);
      st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full);
      ok = __all_sync(0xffffffffu, wait(&bar.d_full, it));
      if (!ok) break;
      fence_after();
      ld64(td, x);
#pragma unroll
      for (int i = 0; i < 64; i += 4) {
        const float4 d = *reinterpret_cast<const float4*>(lse2 + kRows + i);
        const uint32_t(&v)[32] = x[i / 32];
        const int k = i % 32;
        const F2 a = f2(prob[i], prob[i + 1]) *
                     fma2(f2(d.x, d.y), minus, f2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])));
        const F2 b = f2(prob[i + 2], prob[i + 3]) *
                     fma2(f2(d.z, d.w), minus, f2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])));
        e[i / 2] = pack_bf16(a);
        e[i / 2 + 1] = pack_bf16(b);
      }
      st32(td, e);
      st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.ds_full);
        mbar_arrive(&bar.stat_empty[s]);
      }
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, wait(&bar.acc_full, 0));
    if (ok) {
      fence_after();
      const bool there = key < t.nk;
      if (half == 0)
        store_row<DP>(p.gv, p.g_bf16, wide_v, t.k0 + key, hk, p.D, there, tmem + C::kV + lanes,
                      n == 0, 1.f);
      else
        store_row<DP>(p.gk, p.g_bf16, wide_k, t.k0 + key, hk, p.D, there, tmem + C::kK + lanes,
                      n == 0, p.scale);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    dealloc(tmem, C::kColumns);
  }
}

// ---------------------------------------------------------------------------
// Queries
// ---------------------------------------------------------------------------
template <int DP>
struct QueriesCfg {
  static constexpr int kChunks = DP / kChunk;
  static constexpr uint32_t kTile = kChunks * kChunkBytes;
  // K is read by the scores of a tile and, two tiles of scores later, by g_q
  static constexpr int kStagesK = DP == 64 ? 4 : 3, kStagesV = DP == 64 ? 4 : 2;
  static constexpr size_t kSmem = 1024 + (size_t)(2 + kStagesK + kStagesV) * kTile + 512;
  static constexpr uint32_t kS = 0, kD = 256, kQ = 384, kColumns = 512;
};

struct QueriesBars {
  uint64_t qg_full, k_full[4], k_empty[4], v_full[4], v_empty[4], k_last, k_clear, s_full[2],
      d_full, ds_full, acc_full, drained;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(QueriesBars) <= 512, "barriers fit their 512 bytes");

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_queries_tc_kernel(const Attn p, const __grid_constant__ CUtensorMap mq,
                               const __grid_constant__ CUtensorMap mk,
                               const __grid_constant__ CUtensorMap mv,
                               const __grid_constant__ CUtensorMap mg, int wide) {
  using C = QueriesCfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t *sq = smem, *sg = sq + C::kTile, *sk = sg + C::kTile, *sv = sk + C::kStagesK * C::kTile;
  QueriesBars& bar = *reinterpret_cast<QueriesBars*>(sv + C::kStagesV * C::kTile);
  volatile int* abort_flag = &bar.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bar.qg_full, 1);
    for (int s = 0; s < C::kStagesK; ++s) {
      mbar_init(&bar.k_full[s], 1);
      mbar_init(&bar.k_empty[s], 1);
    }
    for (int s = 0; s < C::kStagesV; ++s) {
      mbar_init(&bar.v_full[s], 1);
      mbar_init(&bar.v_empty[s], 1);
    }
    mbar_init(&bar.k_last, 1);
    mbar_init(&bar.k_clear, 1);
    mbar_init(&bar.s_full[0], 1);
    mbar_init(&bar.s_full[1], 1);
    mbar_init(&bar.d_full, 1);
    mbar_init(&bar.ds_full, 8);
    mbar_init(&bar.acc_full, 1);
    mbar_init(&bar.drained, 1);
    bar.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 1) alloc(&bar.tmem, C::kColumns);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem, 0);
  pdl_trigger();
  pdl_wait();

  const int h = blockIdx.x % p.Hq, hk = h / (p.Hq / p.Hk);
  AttnTile t;
  const int past = find_tile<false>(p, kRows, blockIdx.x / p.Hq, t);
  const auto wait = [&](uint64_t* b, uint32_t phase) {
    return wait_for(b, phase, abort_flag, p.status);
  };
  const int keys = past < 0 ? keys_of(p, t, min(t.row0 + kRows, t.nq) - 1) : 0;
  const int n = (keys + kRows - 1) / kRows;
  // rows of the sequence's last tile of keys, if this CTA goes as far and it is not full
  const int rest = n > 0 && t.nk < n * kRows ? t.nk - (n - 1) * kRows : 0;

  if (past >= 0) {
    outside_rows<false>(p, kRows, past, threadIdx.x, kThreads, [&](int row) {
      for (int d = 0; d < p.D; ++d)
        store_elem(p.gq.p, p.g_bf16, row * p.gq.token + h * p.gq.head + d, 0.f);
    });
  } else if (warp < 4) {
    fewer_registers<72>();
    if (warp == 0) {
      if (lane == 0 && n > 0) {
        int k_done = 0, v_done = 0, last_done = 0;
        mbar_expect_tx(&bar.qg_full, 2 * C::kTile);
        load_tile<C::kChunks>(sq, &mq, &bar.qg_full, h, t.q0 + t.row0);
        load_tile<C::kChunks>(sg, &mg, &bar.qg_full, h, t.q0 + t.row0);
        for (int j = 0; j < n; ++j) {
          const int s = j % C::kStagesK, u = j % C::kStagesV;
          if (j >= C::kStagesK && !wait(&bar.k_empty[s], j / C::kStagesK - 1)) break;
          uint64_t* full = rest && j == n - 1 ? &bar.k_last : &bar.k_full[s];
          mbar_expect_tx(full, C::kTile);
          load_tile<C::kChunks>(sk + s * C::kTile, &mk, full, hk, t.k0 + j * kRows);
          ++(full == &bar.k_last ? last_done : k_done);
          if (j >= C::kStagesV && !wait(&bar.v_empty[u], j / C::kStagesV - 1)) break;
          mbar_expect_tx(&bar.v_full[u], C::kTile);
          load_tile<C::kChunks>(sv + u * C::kTile, &mv, &bar.v_full[u], hk, t.k0 + j * kRows);
          ++v_done;
        }
        if (*abort_flag) {
          ring_drain(&bar.qg_full, 1, 1);
          ring_drain(bar.k_full, C::kStagesK, k_done);
          ring_drain(&bar.k_last, 1, last_done);
          ring_drain(bar.v_full, C::kStagesV, v_done);
        }
      }
    } else if (warp == 1) {
      const int steps = (p.D + 15) / 16;
      const uint32_t id = idesc(16 * steps, true);
      const uint32_t aq = by_columns(saddr(sq)), ag = by_columns(saddr(sg));
      const uint32_t ak = by_columns(saddr(sk)), av = by_columns(saddr(sv)), rk = by_rows(saddr(sk));
      constexpr uint32_t kStep = C::kTile >> 4;
      bool ok = n > 0 && wait(&bar.qg_full, 0);
      const auto scores = [&](int j) {
        const int s = j % C::kStagesK;
        ok = rest && j == n - 1 ? wait(&bar.k_clear, 0) : wait(&bar.k_full[s], j / C::kStagesK);
        if (!ok) return;
        fence_after();
        if (elect_one()) {
          product_of_rows<DP / 16>(tmem + C::kS + 128 * (j & 1), aq, ak + s * kStep, steps);
          commit(&bar.s_full[j & 1]);
        }
        __syncwarp();
      };
      const auto gradients = [&](int j) {
        const int u = j % C::kStagesV;
        ok = wait(&bar.v_full[u], j / C::kStagesV);
        if (!ok) return;
        fence_after();
        if (elect_one()) {
          product_of_rows<DP / 16>(tmem + C::kD, ag, av + u * kStep, steps);
          commit(&bar.d_full);
          if (j + C::kStagesV < n) commit(&bar.v_empty[u]);
        }
        __syncwarp();
      };
      if (ok) scores(0);
      if (ok) gradients(0);
      if (ok && n > 1) scores(1);
      for (int j = 0; j < n && ok; ++j) {
        const int s = j % C::kStagesK;
        ok = wait(&bar.ds_full, j);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          product_of_p<64>(tmem + C::kQ, tmem + C::kD, rk + s * kStep, id, j > 0);
          if (j + C::kStagesK < n) commit(&bar.k_empty[s]);
        }
        __syncwarp();
        if (j + 1 < n) gradients(j + 1);
        if (ok && j + 2 < n) scores(j + 2);
      }
      if (n > 0 && elect_one()) {
        if (ok)
          commit(&bar.acc_full);
        else
          drain(&bar.drained);
      }
      __syncwarp();
    } else if (warp == 2) {
      if (rest) {
        if (__all_sync(0xffffffffu, wait(&bar.k_last, 0))) {
          clear_rows<C::kChunks>(sk + ((n - 1) % C::kStagesK) * C::kTile, rest);
          if (lane == 0) mbar_arrive(&bar.k_clear);
        }
      }
    }
  } else {
    more_registers<216>();
    const int half = (warp - 4) >> 2;
    const int row = t.row0 + (warp & 3) * 32 + lane;
    const bool there = row < t.nq;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + C::kS + lanes + 64 * half, td = tmem + C::kD + lanes + 64 * half;
    const float c2 = p.scale * kLog2e;
    const int64_t at = (int64_t)h * p.Tq + t.q0 + row;
    const F2 lse2 = f2(there ? -ld_dep_f32(p.lse2 + at) : -INFINITY);
    const F2 delta = f2(there ? -ld_dep_f32(p.delta + at) : 0.f), c22 = f2(c2);
    const int sees = keys_of(p, t, row), full = keys_of(p, t, t.row0);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int j0 = j * kRows + 64 * half;
      ok = __all_sync(0xffffffffu, wait(&bar.s_full[j & 1], j >> 1));
      if (!ok) break;
      fence_after();
      uint32_t x[2][32];
      ld64(ts + 128 * (j & 1), x);
      const bool cut = j0 + 64 > full;  // some row does not see some column
      float prob[64];
#pragma unroll
      for (int i = 0; i < 64; i += 2) {
        const uint32_t(&v)[32] = x[i / 32];
        const int k = i % 32;
        const float2 a = split(fma2(f2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), c22, lse2));
        prob[i] = exp2_fast(a.x), prob[i + 1] = exp2_fast(a.y);
      }
      ok = __all_sync(0xffffffffu, wait(&bar.d_full, j));
      if (!ok) break;
      fence_after();
      ld64(td, x);
      uint32_t e[32];
#pragma unroll
      for (int i = 0; i < 64; i += 2) {
        const uint32_t(&v)[32] = x[i / 32];
        const int k = i % 32;
        float2 a = split(f2(prob[i], prob[i + 1]) *
                         (f2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])) + delta));
        if (cut) {
          if (i >= sees - j0) a.x = 0.f;
          if (i + 1 >= sees - j0) a.y = 0.f;
        }
        e[i / 2] = bf16x2(a.x, a.y);
      }
      st32(td, e);
      st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.ds_full);
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, wait(&bar.acc_full, 0));
    if (ok && half == 0) {
      fence_after();
      store_row<DP>(p.gq, p.g_bf16, wide, t.q0 + row, h, p.D, there, tmem + C::kQ + lanes, n == 0,
                    p.scale);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    dealloc(tmem, C::kColumns);
  }
}

// Rows of g [T, H, D] of whole 16 bytes.
int wide_rows(const Heads& g, bool bf16, int64_t T, int64_t H, int64_t D) {
  const int64_t per = bf16 ? 8 : 4;
  return D % 8 == 0 && reinterpret_cast<uintptr_t>(g.p) % 16 == 0 &&
         (T <= 1 || g.token % per == 0) && (H <= 1 || g.head % per == 0);
}

struct Maps {
  CUtensorMap q, k, v, g;
};
bool make_maps(Maps* m, const Attn& p) {
  const Heads& g = p.gout16.p ? p.gout16 : p.gout;
  return heads_map(&m->q, p.q, p.Tq, p.Hq, p.D) && heads_map(&m->k, p.k, p.Tk, p.Hk, p.D) &&
         heads_map(&m->v, p.v, p.Tk, p.Hk, p.D) && heads_map(&m->g, g, p.Tq, p.Hq, p.D);
}

template <int DP>
cudaError_t launch_keys(const Attn& p, cudaStream_t st) {
  using C = KeysCfg<DP>;
  const int64_t grid = most_tiles(p, true, kRows) * p.Hk;
  if (grid == 0) return cudaSuccess;
  Maps m;
  if (!make_maps(&m, p)) return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<attn_bwd_keys_tc_kernel<DP>>(C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_bwd_keys_tc_kernel<DP>, dim3((unsigned)grid), dim3(kThreads), C::kSmem,
                    st, p, m.q, m.k, m.v, m.g, wide_rows(p.gk, p.g_bf16, p.Tk, p.Hk, p.D),
                    wide_rows(p.gv, p.g_bf16, p.Tk, p.Hk, p.D));
}

template <int DP>
cudaError_t launch_queries(const Attn& p, cudaStream_t st) {
  using C = QueriesCfg<DP>;
  const int64_t grid = most_tiles(p, false, kRows) * p.Hq;
  if (grid == 0) return cudaSuccess;
  Maps m;
  if (!make_maps(&m, p)) return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<attn_bwd_queries_tc_kernel<DP>>(C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_bwd_queries_tc_kernel<DP>, dim3((unsigned)grid), dim3(kThreads), C::kSmem,
                    st, p, m.q, m.k, m.v, m.g, wide_rows(p.gq, p.g_bf16, p.Tq, p.Hq, p.D));
}

}  // namespace

bool attn_bwd_tc(const Attn& p) {
  return attn_tc(p) && (!p.gout_bf16 || tma_heads(p.gout, p.Tq, p.Hq));
}
cudaError_t launch_attn_bwd_keys_tc(const Attn& p, cudaStream_t st) {
  return p.D <= 64 ? launch_keys<64>(p, st) : launch_keys<128>(p, st);
}
cudaError_t launch_attn_bwd_queries_tc(const Attn& p, cudaStream_t st) {
  return p.D <= 64 ? launch_queries<64>(p, st) : launch_queries<128>(p, st);
}

}  // namespace hlq
