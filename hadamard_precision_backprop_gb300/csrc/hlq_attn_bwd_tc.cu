// hlq_attn_bwd_tc.cu -- attention's backward pass in bf16 on the tensor cores
// (tcgen05, TMEM, TMA), heads up to 128.
//
// Two kinds of CTAs, so that every gradient is summed in one place in a fixed
// order (seven products of a tile of queries and one of keys where five with
// atomics would do):
//
// Keys: a CTA has a tile of 128 keys of a key head and goes over the tiles of
// queries of all query heads that share it.  Rows are keys, columns queries:
//   S' = K Q^T - lse / scale, D' = V G^T - delta (TMEM, fp32)
//   P' = exp2(c S'), dS' = P' D', bf16, in their places
//   g_v += P' G, g_k += dS' Q (TMEM, fp32; P' and dS' are read from TMEM)
// lse and delta belong to columns.  Reading them for each element would take as
// much of shared memory's bandwidth as the operands leave (128 bytes a clock, of
// which the products of S' and D' take all).  So they are summed in with the
// products: as three bf16 numbers (hi + mid + lo, 24 bits) in 16 more columns of
// Q and of G, against ones in those of K and V, one step of 64 clocks each.
//
// Queries: a CTA has a tile of 128 queries of a head and goes over the keys:
//   S = Q K^T, D = G V^T, dS = P (D - delta), g_q += dS K
// D has two places: it is there before the probabilities are.
//
// The products take G, P and dS in bf16.  Where g_out comes as fp32, its rounding
// is the only one: P and dS are two bf16 numbers each (there is room for the second
// beside the first), for three products more.  Errors relative to the gradients'
// norm, with results in bf16 (64 x 197; their own rounding alone is 0.0017): 0.0031
// with one number each, 0.0024 with two, and as much with a g_out of bf16 and one.
//
// In both, warp 0 loads, warp 2 clears rows behind a sequence's end, and the
// warps from 4 on compute: a thread has a row and 32 columns of a tile.  The
// products for one tile run while the probabilities of another are computed.
// Heads up to 64 take the other side in tiles of 64 rows: a CTA then needs half
// of TMEM and of the threads, and two of them on an SM hide each other's
// beginning and end.
//
// 8 sequences of 2048, causal, 32 heads of 128 with 8 of keys: 803 us with the rows'
// pass (0.86 PFLOP/s of five products), tensor pipe busy for 60 %; 64 x 197, 12 heads
// of 64, fp32 g_out: 112 us.  All but the kernels of 128 with one number spill 8 to 48
// bytes.
#include <cmath>

#include "hlq_attn_tc.cuh"
#include "hlq_host.h"
#include "hlq_rows.cuh"

namespace hlq {
namespace {

using namespace tc;

// 32 probabilities or gradients of a row as bf16 pairs, in the first half of the
// columns that they were computed from; with kTwo what the rounding left, as bf16
// again, in the other half.
template <bool kTwo>
__device__ __forceinline__ void put_pairs(uint32_t at, const float (&v)[32]) {
  uint32_t e[16], rest[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    e[i] = bf16x2(v[2 * i], v[2 * i + 1]);
    if (kTwo) rest[i] = bf16x2(v[2 * i] - bf16_lo(e[i]), v[2 * i + 1] - bf16_hi(e[i]));
  }
  st16(at, e);
  if (kTwo) st16(at + 16, rest);
  st_wait();
}

// By head size: rows of a tile of the other side, and the registers of the
// warps that do not compute and of those that do (640 threads of 96 registers:
// 128 x 64 + 512 x 104; 384 of 80: 128 x 48 + 256 x 96).
template <int DP>
struct BwdCfg {
  static constexpr int kN = DP;
  static constexpr int kWarps = kN / 8;  // that compute
  static constexpr int kThreads = 32 * (4 + kWarps), kCtas = kN == 64 ? 2 : 1;
  static constexpr int kFewer = kN == 64 ? 48 : 64, kMore = kN == 64 ? 96 : 104;
  static constexpr int kChunks = DP / kChunk;
  static constexpr uint32_t kTile = kChunks * kChunkBytes;      // of the CTA's side
  static constexpr uint32_t kOther = kChunks * kN * 128;        // of the other side
};

// P or dS as the first operand, 32 columns (two steps) in each 32 columns of
// the fp32 tile that they were computed from; with kTwo what their rounding left
// as well.
template <int kN, bool kTwo>
__device__ __forceinline__ void product_of_parts(uint32_t d, uint32_t p, uint32_t b, uint32_t id,
                                                 bool add) {
#pragma unroll
  for (int two = 0; two < (kTwo ? 2 : 1); ++two)
#pragma unroll
    for (int k = 0; k < kN / 16; ++k)
      mma_ts(d, p + (k >> 1) * 32 + (k & 1) * 8 + 16 * two, desc(b + row_step(k)), id,
             add || k > 0 || two > 0);
}

// What a pass reads, and whether the rows of its results are of whole 16 bytes.
struct Maps {
  CUtensorMap q, k, v, g;
  int wide_q, wide_k, wide_v;
};

// ---------------------------------------------------------------------------
// Keys
// ---------------------------------------------------------------------------
template <int DP>
struct KeysCfg : BwdCfg<DP> {
  using B = BwdCfg<DP>;
  static constexpr int kStages = DP == 64 ? 3 : 2;  // of Q and of G each
  static constexpr int kStats = 2;                  // of lse and delta
  static constexpr uint32_t kMoreN = B::kN * 32;
  static constexpr size_t kSmem =
      1024 + 2 * B::kTile + (size_t)2 * kStages * B::kOther + kMoreBytes + 2 * kStats * kMoreN + 512;
  static constexpr uint32_t kS = 0, kD = B::kN, kV = 2 * B::kN, kK = kV + DP, kColumns = kK + DP;
};

struct KeysBars {
  uint64_t kv_full, q_full[4], q_ready[4], q_empty[4], g_full[4], g_ready[4], g_empty[4],
      stat_full[2], stat_empty[2], s_full, p_full, d_full, ds_full, acc_full, drained;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(KeysBars) <= 512, "barriers fit their 512 bytes");

// With kSplit a cluster of 2^log_split CTAs has the tile of keys, each some of
// the query heads; they add up their sums through each other's shared memory, in
// the order of their ranks.
template <int DP, bool kSplit, bool kTwo>
__device__ __forceinline__ void keys_body(const Attn& p, const Maps& maps, uint32_t block,
                                          int log_split) {
  using C = KeysCfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t *sk = smem, *sv = sk + C::kTile, *sq = sv + C::kTile, *sg = sq + C::kStages * C::kOther;
  uint8_t *ones = sg + C::kStages * C::kOther, *stats = ones + kMoreBytes;  // [kStats][2]
  KeysBars& bar = *reinterpret_cast<KeysBars*>(stats + 2 * C::kStats * C::kMoreN);
  volatile int* abort_flag = &bar.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 64) prefetch(&maps.k), prefetch(&maps.v), prefetch(&maps.q), prefetch(&maps.g);
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
      mbar_init(&bar.stat_empty[s], 1);
    }
    mbar_init(&bar.s_full, 1);
    mbar_init(&bar.p_full, C::kWarps);
    mbar_init(&bar.d_full, 1);
    mbar_init(&bar.ds_full, C::kWarps);
    mbar_init(&bar.acc_full, 1);
    mbar_init(&bar.drained, 1);
    bar.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  // ones in the first three columns, zeros in the rest of all five tiles
  for (int i = threadIdx.x; i < (int)(kMoreBytes + 2 * C::kStats * C::kMoreN) / 16; i += C::kThreads)
    reinterpret_cast<uint4*>(ones)[i] =
        i < (int)kMoreBytes / 16 && i % 16 < 8 ? make_uint4(0x3f803f80u, 0x00003f80u, 0, 0)
                                               : make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 1) {
    alloc(&bar.tmem, C::kColumns);
    // One warp's trigger is the CTA's, and not before it holds its TMEM: a CTA of
    // the next kernel that had taken it instead would wait for this one.
    pdl_trigger();
  }
  pdl_wait();

  const uint32_t unit = kSplit ? block >> log_split : block, tile = unit / p.by_hk;
  const int hk = (int)(unit - tile * p.Hk);
  const int rank = kSplit ? (int)cluster_rank() : 0;
  // of the query heads
  const int h0 = hk * p.group + (kSplit ? rank * p.group >> log_split : 0);
  const int heads = kSplit ? hk * p.group + ((rank + 1) * p.group >> log_split) - h0 : p.group;
  AttnTile t;
  const int past = find_tile<true, kRows>(p, (int)tile, t);
  const auto wait = [&](uint64_t* b, uint32_t phase) {
    return wait_warp(abort_flag, p.status, [&] { return mbar_test(b, phase & 1); });
  };
  const auto wait_alone = [&](uint64_t* b, uint32_t phase) {
    return wait_lane(b, phase, abort_flag, p.status);
  };
  // tiles of queries of a head: from the one with the first query that sees the
  // tile's first key
  int first = 0, per_head = 0;
  if (past < 0) {
    if (p.causal) first = max(0, t.row0 + (t.nq - t.nk)) / C::kN;
    per_head = max(0, (t.nq + C::kN - 1) / C::kN - first);
  }
  const int n = per_head * heads;
  // rows of a head's last tile, if it is not full
  const int rest = past < 0 ? t.nq % C::kN : 0;
  // Thread 0 has set up the barriers, and loads (the first tiles before the others
  // come to the barrier below).
  int q_done = 0, g_done = 0;
  const auto load_q = [&](int it, int h, int i) {
    const int s = it % C::kStages, use = it / C::kStages;
    if (use > 0 && !wait_alone(&bar.q_empty[s], use - 1)) return false;
    mbar_expect_tx(&bar.q_full[s], C::kOther);
    load_tile<C::kChunks, C::kN>(sq + s * C::kOther, &maps.q, &bar.q_full[s], h, t.q0 + i * C::kN);
    ++q_done;
    return true;
  };
  const auto load_g = [&](int it, int h, int i) {
    const int s = it % C::kStages, use = it / C::kStages;
    if (use > 0 && !wait_alone(&bar.g_empty[s], use - 1)) return false;
    mbar_expect_tx(&bar.g_full[s], C::kOther);
    load_tile<C::kChunks, C::kN>(sg + s * C::kOther, &maps.g, &bar.g_full[s], h, t.q0 + i * C::kN);
    ++g_done;
    return true;
  };
  if (threadIdx.x == 0 && n > 0) {
    mbar_expect_tx(&bar.kv_full, 2 * C::kTile);
    load_tile<C::kChunks>(sk, &maps.k, &bar.kv_full, hk, t.k0 + t.row0);
    load_q(0, h0, first);
    load_tile<C::kChunks>(sv, &maps.v, &bar.kv_full, hk, t.k0 + t.row0);
    load_g(0, h0, first);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem, 0);

  if (past >= 0) {
    outside_rows<true>(p, kRows, past, [&](int row, int d) {
      store_elem(p.gk.p, p.g_bf16, row * p.gk.token + hk * p.gk.head + d, 0.f);
      store_elem(p.gv.p, p.g_bf16, row * p.gv.token + hk * p.gv.head + d, 0.f);
    });
  } else if (warp < 4) {
    fewer_registers<C::kFewer>();
    if (warp == 0) {
      if (lane == 0 && n > 0) {
        for (int it = 1, h = h0, i = first + 1; it < n; ++it, ++i) {
          if (i == first + per_head) i = first, ++h;
          if (!load_q(it, h, i) || !load_g(it, h, i)) break;
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
      constexpr uint32_t kStep = C::kOther >> 4, kIdRows = idesc(C::kN, false);
      const uint32_t ak = by_columns(saddr(sk)), av = by_columns(saddr(sv));
      const uint32_t aq = by_columns(saddr(sq)), ag = by_columns(saddr(sg));
      const uint32_t rq = by_rows(saddr(sq), C::kN), rg = by_rows(saddr(sg), C::kN);
      const uint64_t one = more_columns(saddr(ones)), more = more_columns(saddr(stats));
      constexpr uint32_t kMoreStep = C::kMoreN >> 4;
      // by the elected thread
      const auto scores = [&](int it) {
        product_of_rows<DP / 16, C::kN>(tmem + C::kS, ak, aq + (it % C::kStages) * kStep, steps);
        mma_ss(tmem + C::kS, one, more + (it % C::kStats) * 2 * kMoreStep, kIdRows, true);
        commit(&bar.s_full);
      };
      const auto gradients = [&](int it) {
        product_of_rows<DP / 16, C::kN>(tmem + C::kD, av, ag + (it % C::kStages) * kStep, steps);
        mma_ss(tmem + C::kD, one, more + ((it % C::kStats) * 2 + 1) * kMoreStep, kIdRows, true);
        commit(&bar.d_full);
        if (it + C::kStats < n) commit(&bar.stat_empty[it % C::kStats]);
      };
      const auto q_there = [&](int it) {
        return wait_warp(abort_flag, p.status, [&] {
          return mbar_test(&bar.q_ready[it % C::kStages], it / C::kStages & 1) &&
                 mbar_test(&bar.stat_full[it % C::kStats], it / C::kStats & 1);
        });
      };
      const auto g_there = [&](int it) {
        return wait(&bar.g_ready[it % C::kStages], it / C::kStages);
      };
      bool ok = n > 0 && wait(&bar.kv_full, 0) && q_there(0) && g_there(0);
      if (ok) {
        fence_after();
        if (elect_one()) {
          scores(0);
          gradients(0);
        }
        __syncwarp();
      }
      for (int it = 0; it < n && ok; ++it) {
        const int s = it % C::kStages;
        const bool again = it + 1 < n, reused = it + C::kStages < n;
        ok = wait(&bar.p_full, it);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          product_of_parts<C::kN, kTwo>(tmem + C::kV, tmem + C::kS, rg + s * kStep, id, it > 0);
          if (reused) commit(&bar.g_empty[s]);
        }
        __syncwarp();
        if (again) {
          ok = q_there(it + 1);
          if (!ok) break;
          fence_after();
          if (elect_one()) scores(it + 1);
          __syncwarp();
        }
        ok = wait(&bar.ds_full, it);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          product_of_parts<C::kN, kTwo>(tmem + C::kK, tmem + C::kD, rq + s * kStep, id, it > 0);
          if (reused) commit(&bar.q_empty[s]);
        }
        __syncwarp();
        if (again) {
          ok = g_there(it + 1);
          if (!ok) break;
          fence_after();
          if (elect_one()) gradients(it + 1);
          __syncwarp();
        }
      }
      if (n > 0 && elect_one()) {
        if (ok)
          commit(&bar.acc_full);
        else
          drain(&bar.drained);
      }
      __syncwarp();
    } else if (warp == 2) {  // clears the rows behind the sequence's end
      for (int it = 0, left = per_head; it < n; ++it) {
        const int s = it % C::kStages, use = it / C::kStages;
        const bool cut = rest && left == 1;
        left = left == 1 ? per_head : left - 1;
        if (!wait(&bar.q_full[s], use)) break;
        if (cut) clear_rows<C::kChunks, C::kN>(sq + s * C::kOther, rest);
        if (lane == 0) mbar_arrive(&bar.q_ready[s]);
        if (!wait(&bar.g_full[s], use)) break;
        if (cut) clear_rows<C::kChunks, C::kN>(sg + s * C::kOther, rest);
        if (lane == 0) mbar_arrive(&bar.g_ready[s]);
      }
    } else {
      // -lse / scale and -delta of the tiles' queries as three bf16 numbers each;
      // what is behind the end or sees nothing has a score of -3e38
      const float back = 1.f / (p.scale * kLog2e);
      for (int it = 0, h = h0, i = first; it < n; ++it, ++i) {
        const int u = it % C::kStats;
        if (i == first + per_head) i = first, ++h;
        const int i0 = i * C::kN + lane;
        const int64_t at = (int64_t)h * p.Tq + t.q0 + i0;
        float v[2][C::kN / 32];  // all on their way before the first is used
#pragma unroll
        for (int i = 0; i < C::kN / 32; ++i) {
          const bool there = i0 + 32 * i < t.nq;
          v[0][i] = there ? ld_dep_f32(p.lse2 + at + 32 * i) : INFINITY;
          v[1][i] = there ? ld_dep_f32(p.delta + at + 32 * i) : 0.f;
        }
        if (it >= C::kStats && !wait(&bar.stat_empty[u], it / C::kStats - 1))
          break;
#pragma unroll
        for (int i = 0; i < C::kN / 32; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x = k == 0 ? -v[0][i] * back : -v[1][i];
            if (k == 0) x = x > 3e38f ? 3e38f : x < -3e38f ? -3e38f : x;  // NaN stays NaN
            const float hi = __bfloat162float(__float2bfloat16_rn(x));
            const float mid = __bfloat162float(__float2bfloat16_rn(x - hi));
            *reinterpret_cast<uint2*>(stats + (2 * u + k) * C::kMoreN + more_at(32 * i + lane)) =
                make_uint2(bf16x2(hi, mid), bf16x2(x - hi - mid, 0.f));
          }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.stat_full[u]);
      }
    }
    if constexpr (kSplit) {  // the two barriers of the other branch
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else {
    more_registers<C::kMore>();
    const int part = (warp - 4) >> 2;  // of the columns
    const int r = (warp & 3) * 32 + lane, key = t.row0 + r;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + C::kS + lanes + 32 * part, td = tmem + C::kD + lanes + 32 * part;
    const F2 c22 = f2(p.scale * kLog2e);
    // the first query that sees this row's key, and the tile's last key
    const int from = p.causal ? key + (t.nq - t.nk) : 0;
    const int last_from = p.causal ? t.row0 + kRows - 1 + (t.nq - t.nk) : 0;
    bool ok = true;
    for (int it = 0, tile_q = first; it < n; ++it, ++tile_q) {
      if (tile_q == first + per_head) tile_q = first;
      const int i0 = tile_q * C::kN + 32 * part;
      // each lane by itself and one vote: 804 us for 8 x 2048 against 822 with a
      // vote on each try (the warps that issue have those, 5 % faster there)
      ok = __all_sync(0xffffffffu, wait_alone(&bar.s_full, it));
      if (!ok) break;
      fence_after();
      uint32_t x[32];
      float prob[32];
      ld32(ts, x);
      ld_wait(x);
      if (i0 < last_from) {  // some row does not see some column
        const int skip = from - i0;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < skip) x[i] = 0xff800000u;
      }
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 a = split(f2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])) * c22);
        prob[i] = exp2_fast(a.x), prob[i + 1] = exp2_fast(a.y);
      }
      put_pairs<kTwo>(ts, prob);
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full);
      ok = __all_sync(0xffffffffu, wait_alone(&bar.d_full, it));
      if (!ok) break;
      fence_after();
      ld32(td, x);
      ld_wait(x);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 a = split(f2(prob[i], prob[i + 1]) *
                               f2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
        prob[i] = a.x, prob[i + 1] = a.y;
      }
      put_pairs<kTwo>(td, prob);
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.ds_full);
    }
    if (ok && n > 0) ok = wait(&bar.acc_full, 0);
    if (ok) {
      fence_after();
      // all tiles have been read: their place serves for the way out
      const int row0 = t.row0 + (warp & 3) * 32, rows = max(0, min(32, t.nk - row0));
#pragma unroll
      for (int i = part; i < DP / 32; i += C::kWarps / 4) {  // 64 columns of g_v, then of g_k
        const bool second = i >= DP / 64;
        const uint32_t from = tmem + (second ? C::kK : C::kV) + lanes;
        if (kSplit)
          stage_64(smem + (4 * i + (warp & 3)) * 8192, 64 * (i % (DP / 64)), from, n == 0,
                   second ? p.scale : 1.f);
        else
          store_64(smem + (warp - 4) * 8192, second ? p.gk : p.gv, p.g_bf16,
                   second ? maps.wide_k : maps.wide_v, t.k0 + row0, rows, hk, 64 * (i % (DP / 64)), p.D, from,
                   n == 0, n == 0, second ? p.scale : 1.f);
      }
    }
    if constexpr (kSplit) {
      __syncwarp();
      cluster_sync();
      // block b: 64 columns of 32 rows, as 32 x 16 pieces of 16 bytes
      for (int b = rank; b < DP / 8; b += 1 << log_split) {
        const int i = b >> 2;
        const bool second = i >= DP / 64;
        const Heads& x = second ? p.gk : p.gv;
        const int c0 = 64 * (i % (DP / 64));
        for (int e = threadIdx.x - 128; e < 512; e += C::kThreads - 128) {
          const int r = e >> 4, c = e & 15, row = t.row0 + 32 * (b & 3) + r, d = c0 + 4 * c;
          if (row >= t.nk || d >= p.D) continue;
          const uint32_t at = saddr(smem) + b * 8192 + r * 256 + ((c ^ (r & 7)) << 4);
          float4 sum = load_cluster(cluster_map(at, 0));
          for (int k = 1; k < 1 << log_split; ++k) {
            const float4 v = load_cluster(cluster_map(at, k));
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
          }
          const int64_t to = (int64_t)(t.k0 + row) * x.token + (int64_t)hk * x.head + d;
          if (second ? maps.wide_k : maps.wide_v) {
            if (p.g_bf16)
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(x.p) + to) =
                  make_uint2(bf16x2(sum.x, sum.y), bf16x2(sum.z, sum.w));
            else
              *reinterpret_cast<float4*>(static_cast<float*>(x.p) + to) = sum;
          } else {
            store_elem(x.p, p.g_bf16, to, sum.x);
            if (d + 1 < p.D) store_elem(x.p, p.g_bf16, to + 1, sum.y);
            if (d + 2 < p.D) store_elem(x.p, p.g_bf16, to + 2, sum.z);
            if (d + 3 < p.D) store_elem(x.p, p.g_bf16, to + 3, sum.w);
          }
        }
      }
      __syncwarp();
      cluster_sync();  // nobody's shared memory goes before it has been read
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
struct QueriesCfg : BwdCfg<DP> {
  using B = BwdCfg<DP>;
  // K is read by the scores of a tile and, later, by g_q
  static constexpr int kStagesK = DP == 64 ? 4 : 3, kStagesV = DP == 64 ? 3 : 2;
  static constexpr int kDs = 2;  // places of D
  static constexpr size_t kSmem =
      1024 + 2 * B::kTile + (size_t)(kStagesK + kStagesV) * B::kOther + 512;
  static constexpr uint32_t kS = 0, kD = B::kN, kQ = kD + kDs * B::kN, kColumns = kQ + DP;
};

struct QueriesBars {
  uint64_t qg_full, k_full[4], k_empty[4], v_full[4], v_empty[4], k_last, k_clear, s_full, s_empty,
      d_full[2], d_empty[2], ds_full[2], acc_full, drained[2];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(QueriesBars) <= 512, "barriers fit their 512 bytes");

template <int DP, bool kTwo>
__device__ __forceinline__ void queries_body(const Attn& p, const Maps& maps, uint32_t block) {
  using C = QueriesCfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t *sq = smem, *sg = sq + C::kTile, *sk = sg + C::kTile, *sv = sk + C::kStagesK * C::kOther;
  QueriesBars& bar = *reinterpret_cast<QueriesBars*>(sv + C::kStagesV * C::kOther);
  volatile int* abort_flag = &bar.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 64) prefetch(&maps.q), prefetch(&maps.k), prefetch(&maps.g), prefetch(&maps.v);
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
    mbar_init(&bar.s_full, 1);
    mbar_init(&bar.s_empty, C::kWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.d_full[i], 1);
      mbar_init(&bar.d_empty[i], 1);
      mbar_init(&bar.ds_full[i], C::kWarps);
    }
    mbar_init(&bar.acc_full, 1);
    mbar_init(&bar.drained[0], 1);
    mbar_init(&bar.drained[1], 1);
    bar.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    alloc(&bar.tmem, C::kColumns);
    pdl_trigger();  // as in the keys' CTAs
  }
  pdl_wait();

  const uint32_t tile = block / p.by_hq;
  const int h = (int)(block - tile * p.Hq), hk = (int)((uint32_t)h / p.by_group);
  AttnTile t;
  const int past = find_tile<false, kRows>(p, (int)tile, t);
  const auto wait = [&](uint64_t* b, uint32_t phase) {
    return wait_warp(abort_flag, p.status, [&] { return mbar_test(b, phase & 1); });
  };
  const auto wait_alone = [&](uint64_t* b, uint32_t phase) {
    return wait_lane(b, phase, abort_flag, p.status);
  };
  const int keys = past < 0 ? keys_of(p, t, min(t.row0 + kRows, t.nq) - 1) : 0;
  const int n = (keys + C::kN - 1) / C::kN;
  // rows of the sequence's last tile of keys, if this CTA goes as far and it is not full
  const int rest = n > 0 && t.nk < n * C::kN ? t.nk - (n - 1) * C::kN : 0;
  int k_done = 0, v_done = 0, last_done = 0;
  const auto load_k = [&](int j) {
    const int s = j % C::kStagesK;
    if (j >= C::kStagesK && !wait_alone(&bar.k_empty[s], j / C::kStagesK - 1)) return false;
    uint64_t* full = rest && j == n - 1 ? &bar.k_last : &bar.k_full[s];
    mbar_expect_tx(full, C::kOther);
    load_tile<C::kChunks, C::kN>(sk + s * C::kOther, &maps.k, full, hk, t.k0 + j * C::kN);
    ++(full == &bar.k_last ? last_done : k_done);
    return true;
  };
  const auto load_v = [&](int j) {
    const int u = j % C::kStagesV;
    if (j >= C::kStagesV && !wait_alone(&bar.v_empty[u], j / C::kStagesV - 1)) return false;
    mbar_expect_tx(&bar.v_full[u], C::kOther);
    load_tile<C::kChunks, C::kN>(sv + u * C::kOther, &maps.v, &bar.v_full[u], hk, t.k0 + j * C::kN);
    ++v_done;
    return true;
  };
  if (threadIdx.x == 0 && n > 0) {
    mbar_expect_tx(&bar.qg_full, 2 * C::kTile);
    load_tile<C::kChunks>(sq, &maps.q, &bar.qg_full, h, t.q0 + t.row0);
    load_k(0);
    load_tile<C::kChunks>(sg, &maps.g, &bar.qg_full, h, t.q0 + t.row0);
    load_v(0);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem, 0);

  if (past >= 0) {
    outside_rows<false>(p, kRows, past, [&](int row, int d) {
      store_elem(p.gq.p, p.g_bf16, row * p.gq.token + h * p.gq.head + d, 0.f);
    });
  } else if (warp < 4) {
    fewer_registers<C::kFewer>();
    if (warp == 0) {
      if (lane == 0 && n > 0) {
        for (int j = 1; j < n; ++j)
          if (!load_k(j) || !load_v(j)) break;
        if (*abort_flag) {
          ring_drain(&bar.qg_full, 1, 1);
          ring_drain(bar.k_full, C::kStagesK, k_done);
          ring_drain(&bar.k_last, 1, last_done);
          ring_drain(bar.v_full, C::kStagesV, v_done);
        }
      }
    } else if (warp != 2) {  // warp 1: S = Q K^T and D = G V^T; warp 3: g_q += dS K
      const int steps = (p.D + 15) / 16;
      constexpr uint32_t kStep = C::kOther >> 4;
      bool ok = n > 0 && wait(&bar.qg_full, 0);
      if (warp == 1) {
        const uint32_t aq = by_columns(saddr(sq)), ag = by_columns(saddr(sg));
        const uint32_t ak = by_columns(saddr(sk)), av = by_columns(saddr(sv));
        for (int j = 0; j < n && ok; ++j) {
          const int s = j % C::kStagesK, u = j % C::kStagesV;
          ok = (rest && j == n - 1 ? wait(&bar.k_clear, 0) : wait(&bar.k_full[s], j / C::kStagesK)) &&
               (j < 1 || wait(&bar.s_empty, j - 1));  // the scores before have been read
          if (!ok) break;
          fence_after();
          if (elect_one()) {
            product_of_rows<DP / 16, C::kN>(tmem + C::kS, aq, ak + s * kStep, steps);
            commit(&bar.s_full);
          }
          __syncwarp();
          ok = wait(&bar.v_full[u], j / C::kStagesV) &&
               (j < C::kDs || wait(&bar.d_empty[j % C::kDs], j / C::kDs - 1));  // g_q has read dS
          if (!ok) break;
          fence_after();
          if (elect_one()) {
            product_of_rows<DP / 16, C::kN>(tmem + C::kD + C::kN * (j % C::kDs), ag, av + u * kStep, steps);
            commit(&bar.d_full[j % C::kDs]);
            if (j + C::kStagesV < n) commit(&bar.v_empty[u]);
          }
          __syncwarp();
        }
        if (n > 0 && !ok && elect_one()) drain(&bar.drained[0]);
      } else {
        const uint32_t id = idesc(16 * steps, true), rk = by_rows(saddr(sk), C::kN);
        for (int j = 0; j < n && ok; ++j) {
          const int s = j % C::kStagesK;
          ok = wait(&bar.ds_full[j % C::kDs], j / C::kDs);  // and so K is there
          if (!ok) break;
          fence_after();
          if (elect_one()) {
            product_of_parts<C::kN, kTwo>(tmem + C::kQ, tmem + C::kD + C::kN * (j % C::kDs), rk + s * kStep, id, j > 0);
            if (j + C::kDs < n) commit(&bar.d_empty[j % C::kDs]);
            if (j + C::kStagesK < n) commit(&bar.k_empty[s]);
          }
          __syncwarp();
        }
        if (n > 0 && elect_one()) {
          if (ok)
            commit(&bar.acc_full);
          else
            drain(&bar.drained[1]);
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      if (rest) {
        if (wait_warp(abort_flag, p.status, [&] { return mbar_test(&bar.k_last, 0); }, n)) {
          clear_rows<C::kChunks, C::kN>(sk + ((n - 1) % C::kStagesK) * C::kOther, rest);
          if (lane == 0) mbar_arrive(&bar.k_clear);
        }
      }
    }
  } else {
    more_registers<C::kMore>();
    const int part = (warp - 4) >> 2;  // of the columns
    const int row = t.row0 + (warp & 3) * 32 + lane;
    const bool there = row < t.nq;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + C::kS + lanes + 32 * part, td = tmem + C::kD + lanes + 32 * part;
    const int64_t at = (int64_t)h * p.Tq + t.q0 + row;
    const F2 lse2 = f2(there ? -ld_dep_f32(p.lse2 + at) : -INFINITY);
    const F2 delta = f2(there ? -ld_dep_f32(p.delta + at) : 0.f), c22 = f2(p.scale * kLog2e);
    const int sees = keys_of(p, t, row), full = keys_of(p, t, t.row0);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int j0 = j * C::kN + 32 * part;
      ok = __all_sync(0xffffffffu, wait_alone(&bar.s_full, j));
      if (!ok) break;
      fence_after();
      uint32_t x[32];
      float prob[32];
      ld32(ts, x);
      ld_wait(x);
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.s_empty);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 a = split(fma2(f2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), c22, lse2));
        prob[i] = exp2_fast(a.x), prob[i + 1] = exp2_fast(a.y);
      }
      ok = __all_sync(0xffffffffu, wait_alone(&bar.d_full[j % C::kDs], j / C::kDs));
      if (!ok) break;
      fence_after();
      ld32(td + C::kN * (j % C::kDs), x);
      ld_wait(x);
      float ds[32];
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 a = split(f2(prob[i], prob[i + 1]) *
                               (f2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])) + delta));
        ds[i] = a.x, ds[i + 1] = a.y;
      }
      if (j0 + 32 > full) {  // some row does not see some column
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i >= sees - j0) ds[i] = 0.f;
      }
      put_pairs<kTwo>(td + C::kN * (j % C::kDs), ds);
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.ds_full[j % C::kDs]);
    }
    if (ok && n > 0) ok = wait(&bar.acc_full, 0);
    if (ok && part < DP / 64) {
      fence_after();
      const int row0 = t.row0 + (warp & 3) * 32;
      store_64(smem + (warp - 4) * 8192, p.gq, p.g_bf16, maps.wide_q, t.q0 + row0,
               max(0, min(32, t.nq - row0)), h, 64 * part, p.D, tmem + C::kQ + lanes, n == 0, n == 0,
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

// ---------------------------------------------------------------------------
// Kernels
// ---------------------------------------------------------------------------
// Both in one launch, the keys' CTAs first (they are alike in threads, and
// nearly in shared memory): what one leaves of the SMs the other takes.  One
// after the other 64 x 197 (12 heads of 64) took 110 us with the rows' pass where
// this takes 103, one sequence of 300 (8 heads of 64) 18 where this takes 11.
template <int DP, bool kSplit, bool kTwo>
__global__ void __launch_bounds__(BwdCfg<DP>::kThreads, BwdCfg<DP>::kCtas)
    attn_bwd_tc_kernel(const Attn p, const __grid_constant__ Maps keys,
                       const __grid_constant__ Maps queries, uint32_t keys_ctas, uint32_t ctas,
                       int log_split) {
  if (blockIdx.x < keys_ctas)
    keys_body<DP, kSplit, kTwo>(p, keys, blockIdx.x, log_split);
  else if (!kSplit || blockIdx.x < ctas)  // whole clusters are launched
    queries_body<DP, kTwo>(p, queries, blockIdx.x - keys_ctas);
}

// Rows of g [T, H, D] of whole 16 bytes.
int wide_rows(const Heads& g, bool bf16, int64_t T, int64_t H, int64_t D) {
  const int64_t per = bf16 ? 8 : 4;
  return D % 8 == 0 && reinterpret_cast<uintptr_t>(g.p) % 16 == 0 &&
         (T <= 1 || g.token % per == 0) && (H <= 1 || g.head % per == 0);
}

bool make_maps(Maps* m, const Attn& p, int rows_q, int rows_k) {
  const Heads& g = p.gout16.p ? p.gout16 : p.gout;
  m->wide_q = wide_rows(p.gq, p.g_bf16, p.Tq, p.Hq, p.D);
  m->wide_k = wide_rows(p.gk, p.g_bf16, p.Tk, p.Hk, p.D);
  m->wide_v = wide_rows(p.gv, p.g_bf16, p.Tk, p.Hk, p.D);
  return heads_map(&m->q, p.q, p.Tq, p.Hq, p.D, rows_q) &&
         heads_map(&m->k, p.k, p.Tk, p.Hk, p.D, rows_k) &&
         heads_map(&m->v, p.v, p.Tk, p.Hk, p.D, rows_k) &&
         heads_map(&m->g, g, p.Tq, p.Hq, p.D, rows_q);
}

template <int DP, bool kSplit, bool kTwo>
cudaError_t launch(const Attn& p, int log_split, cudaStream_t st) {
  using K = KeysCfg<DP>;
  using Q = QueriesCfg<DP>;
  constexpr size_t kSmem = K::kSmem > Q::kSmem ? K::kSmem : Q::kSmem;
  const int64_t keys = most_tiles(p, true, kRows) * p.Hk << log_split;
  const int64_t ctas = keys + most_tiles(p, false, kRows) * p.Hq;
  if (ctas == 0) return cudaSuccess;
  Maps mk, mq;
  if (!make_maps(&mk, p, K::kN, kRows) || !make_maps(&mq, p, kRows, Q::kN))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<attn_bwd_tc_kernel<DP, kSplit, kTwo>>(kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((ctas - 1) >> log_split) + 1) << log_split);
  cfg.blockDim = dim3(K::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1u << log_split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kSplit ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, attn_bwd_tc_kernel<DP, kSplit, kTwo>, p, mk, mq, (uint32_t)keys,
                            (uint32_t)ctas, log_split);
}

template <int DP, bool kSplit>
cudaError_t launch_types(const Attn& p, int log_split, cudaStream_t st) {
  return p.gout16.p ? launch<DP, kSplit, true>(p, log_split, st)
                    : launch<DP, kSplit, false>(p, log_split, st);
}

}  // namespace

bool attn_bwd_tc(const Attn& p) {
  return attn_tc(p) && (!p.gout_bf16 || tma_heads(p.gout, p.Tq, p.Hq));
}

cudaError_t launch_attn_bwd_tc(const Attn& p, cudaStream_t st) {
  // A cluster for a tile of keys only where there are fewer tiles than SMs twice
  // and each has eight tiles of queries or more: one sequence of 16384 (4 heads of
  // 128 that share one; causal) 738 -> 601 us, 5 of 400 (8 heads of 64 that share
  // one) 57 -> 30; but 8 of 2048 (16 heads of 128, 4 shared ones) 409 -> 459, 40
  // of 60 (4 heads of 64, 2 shared ones) 12 -> 20.
  const int64_t tiles = most_tiles(p, true, kRows) * p.Hk, n = p.D <= 64 ? 64 : 128;
  const int64_t each = (p.Tq / p.batch + n - 1) / n * p.group;
  int split = 0;
  if (each >= 8)
    while (split < 3 && 2 << split <= p.group && tiles << split < 2 * (int64_t)device_sm_count())
      ++split;
  if (split > 0)
    return p.D <= 64 ? launch_types<64, true>(p, split, st) : launch_types<128, true>(p, split, st);
  return p.D <= 64 ? launch_types<64, false>(p, 0, st) : launch_types<128, false>(p, 0, st);
}

}  // namespace hlq
