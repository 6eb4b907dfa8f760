// hlq_attn_fwd_tc.cu -- attention's forward pass in bf16 on the tensor cores
// (tcgen05, TMEM, TMA), heads up to 128.
//
// A CTA has one or two tiles of 128 queries of one head and goes over the keys'
// tiles of 128.  Per tile of keys and of queries:
//   S = Q K^T (TMEM, fp32)  ->  P = exp2(c S - c m), bf16, in the place of S
//   O += P V (TMEM, fp32)
// warp 0 loads (TMA), warps 1 and 3 issue the products of the first and of the
// second tile of queries, warp 2 clears V's rows behind the sequence's end,
// warps 4-7 and 8-11 are the softmax of the tiles, a thread to a row: maximum and
// sum need no shuffles.  While one tile's softmax runs, the products of the other
// one do (of the same CTA, or of the SM's other CTA); the product with V begins
// when half of P is there.
//
// m is the maximum of the tiles so far when it was last taken over; it is taken
// over again only where the row's maximum has risen by more than 8 in units of
// log 2 (P then stays below 2^8, which costs bf16 nothing), so that O is
// rescaled rarely.  Sums are those of the unrounded probabilities, in fp32.
// (Rescaling put off and two tiles' softmax in turns are published steps of the
// algorithm.)
//
// What bounds it: a tile's chain of product, softmax and product, of which two
// run side by side in an SM.  A step of 128 x 128 of a head of 128 is 1024 clocks
// of the tensor pipe (64 for each 128 x 128 x 16) and, for each of the four
// schedulers, 512 of exponentials (4 a warp) and about as many of multiplications,
// maxima, sums and conversions; the reads and writes of TMEM and the waits between
// them are what is left.  Tensor pipe busy for 49 % (4 sequences of 2048).
// Causal, 32 heads of 128 with 8 of keys, 8 sequences of 2048: 257 us (1.07
// PFLOP/s of the half that is not masked), where the beginnings and ends of the CTAs
// that fill an SM one after the other are a good part; 4 heads, one sequence of
// 16384: 184 us (1.49 PFLOP/s), where the longest tile's 128 steps are the time.
// All instances spill 12 to 60 bytes.
#include <cmath>
#include <cstring>

#include "hlq_attn_tc.cuh"
#include "hlq_host.h"
#include "hlq_rows.cuh"

namespace hlq {
namespace {

using namespace tc;

constexpr float kRise = 8.f;

// kQ tiles of queries in a CTA.  Two for one CTA an SM; one for two CTAs an SM,
// which hide each other's beginning and end but bring the keys' tiles into
// shared memory for each tile of queries.
template <int DP, int kQ>
struct FwdCfg {
  static constexpr int kChunks = DP / kChunk;
  static constexpr uint32_t kTile = kChunks * kChunkBytes;
  static constexpr int kStages = (kQ == 2 ? 2 : 1) * (DP == 64 ? 2 : 1);  // of K and of V each
  static constexpr size_t kSmem = 1024 + (size_t)(kQ + 2 * kStages) * kTile + 512;
  static constexpr uint32_t kO = kQ * kRows, kColumns = kQ * 256;
  static constexpr int kThreads = 128 * (1 + kQ), kCtas = 3 - kQ;
  // The softmax of two tiles goes in turns, so that one's products run beside the
  // other's softmax whatever the tiles began with: one sequence of 16384 (4 heads of
  // 128, causal) 184 us, without turns 195 or 231 from one build to the next, with
  // the maxima out of turn 191; 8 of 2048 257 against 258.  Heads of 64, where the
  // products are half as long, lose by it: 2 of 8192 (8 heads) 350 against 320.
  static constexpr bool kTurns = kQ == 2 && DP == 128;
  // of the launch's 168 (384 threads) or 128 (256 threads) a thread
  static constexpr int kFewer = kQ == 2 ? 72 : 56, kMore = kQ == 2 ? 216 : 200;
};

struct FwdBars {
  uint64_t q_full[2], k_full[4], k_empty[4], v_full[4], v_empty[4], v_last, v_clear, s_full[2],
      p_full[2][2], turn[2][4], o_full[2], drained[2];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(FwdBars) <= 512, "barriers fit their 512 bytes");

template <int DP, int kQ>
__global__ void __launch_bounds__(FwdCfg<DP, kQ>::kThreads, FwdCfg<DP, kQ>::kCtas)
    attn_fwd_tc_kernel(const Attn p, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, int wide_out) {
  using C = FwdCfg<DP, kQ>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t *sq = smem, *sk = sq + kQ * C::kTile, *sv = sk + C::kStages * C::kTile;
  FwdBars& bar = *reinterpret_cast<FwdBars*>(sv + C::kStages * C::kTile);
  volatile int* abort_flag = &bar.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int g = 0; g < kQ; ++g) {
      mbar_init(&bar.q_full[g], 1);
      mbar_init(&bar.s_full[g], 1);
      mbar_init(&bar.p_full[g][0], 4);
      mbar_init(&bar.p_full[g][1], 4);
      for (int w = 0; w < 4; ++w) mbar_init(&bar.turn[g][w], 1);
      mbar_init(&bar.o_full[g], 1);
      mbar_init(&bar.drained[g], 1);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bar.k_full[s], 1);
      mbar_init(&bar.k_empty[s], kQ);
      mbar_init(&bar.v_full[s], 1);
      mbar_init(&bar.v_empty[s], kQ);
    }
    mbar_init(&bar.v_last, 1);
    mbar_init(&bar.v_clear, 1);
    bar.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 1) alloc(&bar.tmem, C::kColumns);
  if (threadIdx.x == 64) {
    prefetch(&mq), prefetch(&mk), prefetch(&mv);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem, 0);
  pdl_trigger();
  pdl_wait();

  const uint32_t tile = blockIdx.x / p.by_hq;
  const int h = (int)(blockIdx.x - tile * p.Hq), hk = (int)((uint32_t)h / p.by_group);
  AttnTile t;
  const int past = find_tile<false, kQ * kRows>(p, (int)tile, t);
  const auto wait = [&](uint64_t* b, uint32_t phase) {
    return wait_warp(abort_flag, p.status, [&] { return mbar_test(b, phase & 1); });
  };
  const auto wait_alone = [&](uint64_t* b, uint32_t phase) {
    return wait_lane(b, phase, abort_flag, p.status);
  };
  // tiles of keys that the tiles of queries see
  int tiles[2] = {0, 0};
  if (past < 0)
    for (int g = 0; g < kQ; ++g) {
      const int last = min(t.row0 + (g + 1) * kRows, t.nq) - 1;
      if (last >= t.row0 + g * kRows) tiles[g] = (keys_of(p, t, last) + kRows - 1) / kRows;
    }
  const int n = max(tiles[0], tiles[1]);
  // rows of the sequence's last tile of keys, if this CTA goes as far and it is not full
  const int rest = n > 0 && t.nk < n * kRows ? t.nk - (n - 1) * kRows : 0;

  if (past >= 0) {
    outside_rows<false>(p, kQ * kRows, past, [&](int row, int d) {
      if (d == 0) p.lse[(int64_t)row * p.Hq + h] = -INFINITY;
      store_elem(p.out.p, true, row * p.out.token + h * p.out.head + d, 0.f);
    });
  } else if (warp < 4) {
    fewer_registers<C::kFewer>();
    if (warp == 0) {
      if (lane == 0 && n > 0) {
        int k_done = 0, v_done = 0, last_done = 0;
        const auto load_q = [&](int g) {
          mbar_expect_tx(&bar.q_full[g], C::kTile);
          load_tile<C::kChunks>(sq + g * C::kTile, &mq, &bar.q_full[g], h,
                                t.q0 + t.row0 + g * kRows);
        };
        const auto load_k = [&](int j) {
          const int s = j % C::kStages;
          if (j >= C::kStages && !wait_alone(&bar.k_empty[s], j / C::kStages - 1)) return false;
          mbar_expect_tx(&bar.k_full[s], C::kTile);
          load_tile<C::kChunks>(sk + s * C::kTile, &mk, &bar.k_full[s], hk, t.k0 + j * kRows);
          ++k_done;
          return true;
        };
        const auto load_v = [&](int j) {
          const int s = j % C::kStages;
          if (j >= C::kStages && !wait_alone(&bar.v_empty[s], j / C::kStages - 1)) return false;
          uint64_t* full = rest && j == n - 1 ? &bar.v_last : &bar.v_full[s];
          mbar_expect_tx(full, C::kTile);
          load_tile<C::kChunks>(sv + s * C::kTile, &mv, full, hk, t.k0 + j * kRows);
          ++(full == &bar.v_last ? last_done : v_done);
          return true;
        };
        // only what is waited for: with fewer keys than queries the first tile of
        // queries may see none
        if (tiles[0] > 0) load_q(0);
        load_k(0);
        if (tiles[1] > 0) load_q(1);
        for (int j = 0; j < n; ++j)
          if ((j > 0 && !load_k(j)) || !load_v(j)) break;
        if (*abort_flag) {  // let the copies under way land
          for (int g = 0; g < kQ; ++g) ring_drain(&bar.q_full[g], 1, tiles[g] > 0);
          ring_drain(bar.k_full, C::kStages, k_done);
          ring_drain(bar.v_full, C::kStages, v_done);
          ring_drain(&bar.v_last, 1, last_done);
        }
      }
    } else if (warp == 1 || (kQ == 2 && warp == 3)) {  // the whole warp, of which one thread issues
        const int g = warp >> 1;
        const int steps = (p.D + 15) / 16;
        const uint32_t id = idesc(16 * steps, true);
        const uint32_t aq = by_columns(saddr(sq) + g * C::kTile), ak = by_columns(saddr(sk));
        const uint32_t av = by_rows(saddr(sv)), ts = tmem + g * kRows, to = tmem + C::kO + g * DP;
        constexpr uint32_t kStep = C::kTile >> 4;
        bool ok = tiles[g] == 0 || wait(&bar.q_full[g], 0);
        const auto scores = [&](int j) {
          const int s = j % C::kStages;
          ok = wait(&bar.k_full[s], j / C::kStages);
          if (!ok) return;
          fence_after();
          if (elect_one()) {
            product_of_rows<DP / 16>(ts, aq, ak + s * kStep, steps);
            commit(&bar.s_full[g]);
            if (j + C::kStages < n) commit(&bar.k_empty[s]);
          }
          __syncwarp();
        };
        if (ok && tiles[g] > 0) scores(0);
        for (int j = 0; j < tiles[g] && ok; ++j) {
          const int s = j % C::kStages;
          ok = rest && j == n - 1 ? wait(&bar.v_clear, 0) : wait(&bar.v_full[s], j / C::kStages);
          for (int half = 0; half < 2 && ok; ++half) {
            ok = wait(&bar.p_full[g][half], j);
            if (!ok) break;
            fence_after();
            if (elect_one()) {
              product_of_p(to, ts + 32 * half, av + s * kStep, id, half, j > 0 || half > 0);
              if (half && j == tiles[g] - 1) commit(&bar.o_full[g]);
              if (half && j + C::kStages < n) commit(&bar.v_empty[s]);
            }
            __syncwarp();
          }
          if (ok && j + 1 < tiles[g]) scores(j + 1);
        }
        // tiles of keys that the other tile of queries alone sees
        for (int j = tiles[g]; j + C::kStages < n && ok; ++j) {
          const int s = j % C::kStages;
          ok = wait(&bar.k_full[s], j / C::kStages) && wait(&bar.v_full[s], j / C::kStages);
          if (ok && lane == 0) {
            mbar_arrive(&bar.k_empty[s]);
            mbar_arrive(&bar.v_empty[s]);
          }
        }
        if (!ok && elect_one()) drain(&bar.drained[g]);
        __syncwarp();
    } else if (warp == 2) {
      if (rest) {
        const int s = (n - 1) % C::kStages;
        if (wait_warp(abort_flag, p.status, [&] { return mbar_test(&bar.v_last, 0); }, n)) {
          clear_rows<C::kChunks>(sv + s * C::kTile, rest);
          if (lane == 0) mbar_arrive(&bar.v_clear);
        }
      }
    }
  } else {
    more_registers<C::kMore>();
    const int g = (warp - 4) >> 2;
    const int row = t.row0 + g * kRows + (warp & 3) * 32 + lane;  // of the sequence
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // 32 lanes a warp, in bits 16-31
    const uint32_t ts = tmem + g * kRows + lanes, to = tmem + C::kO + g * DP + lanes;
    const int sees = keys_of(p, t, row);
    // the tile's first row sees the fewest
    const int full = keys_of(p, t, t.row0 + g * kRows) / kRows;
    const float c2 = p.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < tiles[g] && ok; ++j) {
      ok = wait(&bar.s_full[g], j);
      // after the other tile's step before
      if (C::kTurns && ok && j >= 1 - g && j - 1 + g < tiles[1 - g])
        ok = wait(&bar.turn[1 - g][warp & 3], j - 1 + g);
      if (!ok) break;
      fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) ld32(ts + 32 * c, s[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c) ld_wait(s[c]);
      if (j >= full) {
        const int limit = sees - j * kRows;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i >= limit) s[c][i] = 0xff800000u;
      }
      float tops[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        tops[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
        for (int i = 2; i < 32; i += 2)
          tops[c] = max3(tops[c], __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
      }
      float top = max3(tops[0], tops[1], fmaxf(tops[2], tops[3]));
      top = fmaxf(top, m);
      // a row that has seen nothing takes over what it sees
      const bool rises = top > m && !((top - m) * c2 <= kRise);
      if (__any_sync(0xffffffffu, rises)) {
        const float keep = rises ? exp2_fast((m - top) * c2) : 1.f;
        if (rises) m = top;
        l *= keep;
        if (j > 0) {
#pragma unroll
          for (int c = 0; c < DP / 32; ++c) {
            uint32_t o[32];
            ld32(to + 32 * c, o);
            ld_wait(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
            st32(to + 32 * c, o);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : -m * c2;
      const F2 c22 = f2(c2), base2 = f2(base);
      F2 sum = f2(0.f);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t e[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint32_t(&r)[32] = s[2 * half + i / 16];
          const int k = 2 * (i % 16);
          const F2 two = f2(__uint_as_float(r[k]), __uint_as_float(r[k + 1]));
          const float2 x = split(fma2(two, c22, base2));
          const float a = exp2_fast(x.x), b = exp2_fast(x.y);
          sum = sum + f2(a, b);
          e[i] = bf16x2(a, b);
        }
        st32(ts + 32 * half, e);
        st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[g][half]);
      }
      if (C::kTurns && lane == 0) mbar_arrive(&bar.turn[g][warp & 3]);
      const float2 both = split(sum);
      l += both.x + both.y;
    }
    if (tiles[g] > 0 && ok) ok = wait(&bar.o_full[g], 0);
    const bool there = past < 0 && row < t.nq;
    if (ok) {
      fence_after();
      const float inv = 1.f / l;
      if (there)
        p.lse[(int64_t)(t.q0 + row) * p.Hq + h] =
            l == 0.f ? -INFINITY : (m * c2 + log2f(l)) * kLn2;
      // Q has been read: its place serves for the way out.  A row that sees
      // nothing is zeros, whatever TMEM holds.
      const bool none = __all_sync(0xffffffffu, l == 0.f);
      const int first = t.row0 + g * kRows + (warp & 3) * 32;
#pragma unroll
      for (int c = 0; c < DP / 64; ++c)
        store_64(sq + g * C::kTile + (warp & 3) * 4096, p.out, true, wide_out, t.q0 + first,
                 max(0, min(32, t.nq - first)), h, 64 * c, p.D, to, none, l == 0.f, inv);
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

template <int DP, int kQ>
cudaError_t launch(const Attn& p, cudaStream_t st) {
  using C = FwdCfg<DP, kQ>;
  const int64_t grid = most_tiles(p, false, kQ * kRows) * p.Hq;
  if (grid == 0) return cudaSuccess;
  CUtensorMap mq, mk, mv;
  if (!heads_map(&mq, p.q, p.Tq, p.Hq, p.D, kRows) ||
      !heads_map(&mk, p.k, p.Tk, p.Hk, p.D, kRows) ||
      !heads_map(&mv, p.v, p.Tk, p.Hk, p.D, kRows))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<attn_fwd_tc_kernel<DP, kQ>>(C::kSmem);
  if (e != cudaSuccess) return e;
  const int wide_out = p.D % 8 == 0 && tma_heads(p.out, p.Tq, p.Hq);
  return launch_pdl(attn_fwd_tc_kernel<DP, kQ>, dim3((unsigned)grid), dim3(C::kThreads), C::kSmem,
                    st, p, mq, mk, mv, wide_out);
}

PFN_cuTensorMapEncodeTiled_v12000 encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

}  // namespace

bool heads_map(CUtensorMap* map, const Heads& x, int64_t T, int64_t H, int64_t D, int rows) {
  const auto fn = encode();
  if (!fn) return false;
  // a dimension of one element: any stride does
  const cuuint64_t token = T > 1 ? (cuuint64_t)x.token * 2 : 16;
  const cuuint64_t head = H > 1 ? (cuuint64_t)x.head * 2 : 16;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {head, token};
  const cuuint32_t box[3] = {tc::kChunk, 1, (cuuint32_t)rows}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, x.p, dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool attn_tc(const Attn& p) {
  return p.bf16 && p.D <= 128 && p.Tq > 0 && p.Tk > 0 && tma_heads(p.q, p.Tq, p.Hq) &&
         tma_heads(p.k, p.Tk, p.Hk) && tma_heads(p.v, p.Tk, p.Hk);
}

cudaError_t launch_attn_tc(const Attn& p, cudaStream_t st) {
  // Two tiles of queries in a CTA where sequences are long (with a causal mask the
  // two see different numbers of keys) and there are enough of them: 16 of 1024 (16
  // heads of 128) 119 us against 126 with one tile, 12 of 1300 (12 heads) 127 against
  // 136; but 64 of 300 128 against 114.  Causal: 8 of 2000 (8 heads) 69.3 against 69.9;
  // but 12 of 1300 90 against 81, 32 of 512 75 against 67.  Heads of 64: 99 against 104,
  // 105 against 109, 104 against 87; 53.5 against 55.4, 69 against 65, 54 against 51.
  const int64_t pairs = most_tiles(p, false, 2 * kRows) * p.Hq;
  if (p.Tk / p.batch >= (p.causal ? 1792 : 768) && pairs >= device_sm_count())
    return p.D <= 64 ? launch<64, 2>(p, st) : launch<128, 2>(p, st);
  return p.D <= 64 ? launch<64, 1>(p, st) : launch<128, 1>(p, st);
}

}  // namespace hlq
