// hlq_attn.cuh -- what the attention kernels share: one call's arguments, the
// sequences and their tiles.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "hlq_device.cuh"
#include "hlq_kernels.h"

namespace hlq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Queries and keys of one sequence, and the tile of it that a CTA has.
struct AttnTile {
  int q0, nq, k0, nk;  // first row and number of rows
  int row0;            // the tile's first row within the sequence
};

__device__ __forceinline__ uint32_t operator/(uint32_t n, const Div& d) {
  return (uint32_t)((uint64_t)n * d.m >> d.s);
}

// Rows [lo, hi) of sequence b; `bad` where the offsets are not in order (the
// rows are then cut to those that exist).
__device__ __forceinline__ int2 seq_rows(const int32_t* seqs, int b, int T, bool& bad) {
  const int a = (int)ld_dep_u32(reinterpret_cast<const unsigned int*>(seqs) + b);
  const int e = (int)ld_dep_u32(reinterpret_cast<const unsigned int*>(seqs) + b + 1);
  const int lo = min(max(a, 0), T), hi = min(max(e, lo), T);
  bad |= a != lo || e != hi;
  return make_int2(lo, hi);
}

// find_tile for more than kScan sequences.  Sequence b has the tiles from
// offset(b) / rows + b on: as many as it can need, at the price of one that may stay
// without rows.  So a sequence is found by search, 32 ways at a time, and the time
// of a call grows with its tiles (by the steps of find_tile with their number times
// that of the sequences): sequences of 20 tokens, 8 heads of 64, not causal, 10000 of
// them 2.7 ms against 9.0, 1000 of them 276 us against 460; but 300 of them 94 against
// 89, 200 of 100 tokens 105 against 89, and 24 of up to 1500 (16 heads of 80, causal),
// which then are not taken in order of their work, 59 against 48.
constexpr int kScan = 256, kNoChunk = 0x7fffffff;

template <bool kKeys, int rows>
__device__ __forceinline__ int search_tile(const Attn& p, int t, AttnTile& o) {
  const int32_t* seqs = kKeys ? p.seqs_k : p.seqs_q;
  const int T = kKeys ? p.Tk : p.Tq, lane = threadIdx.x & 31;
  bool bad = false;
  if (t < p.batch) {  // each sequence's offsets are looked at by some CTA
    seq_rows(p.seqs_q, t, p.Tq, bad);
    seq_rows(p.seqs_k, t, p.Tk, bad);
  }
  const int front = seq_rows(seqs, 0, T, bad).x;
  const int end = seq_rows(seqs, p.batch - 1, T, bad).y / rows + p.batch;
  int past = -1;
  if (t < front / rows) {
    past = t;
  } else if (t >= end) {
    past = front / rows + t - end;
  } else {
    int lo = 0, hi = p.batch;  // the last one that begins at t or before is among these
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, b = lo + lane * step;
      const bool before = b < hi && seq_rows(seqs, b, T, bad).x / rows + b <= t;
      lo += (31 - __clz(__ballot_sync(0xffffffffu, before) | 1)) * step;
      hi = min(hi, lo + step);
    }
    const int2 q = seq_rows(p.seqs_q, lo, p.Tq, bad), k = seq_rows(p.seqs_k, lo, p.Tk, bad);
    const int2 r = kKeys ? k : q;
    const int n = (r.y - r.x + rows - 1) / rows, i = t - r.x / rows - lo;
    if (i >= 0 && i < n)
      o = {q.x, q.y - q.x, k.x, k.y - k.x, (kKeys ? i : n - 1 - i) * rows};
    else
      past = kNoChunk;
  }
  if (bad) raise_flag(p.status, HLQ_DEV_BADCODE);
  return past;
}

// Tile t of `rows` queries (keys with kKeys) among the tiles of all sequences,
// those with the most work first.  Returns -1, or for a tile of no sequence the
// number of its chunk of the rows outside them.  A whole warp calls it.
//
// With sequences of one length the tiles of all sequences that have the same
// rank follow each other.  Else each lane looks at a sequence of its own, 32 of
// them at a time: with a causal mask the work of a sequence's tiles goes from its
// number of tiles down to one, so for each amount from the most on the tiles that
// have it (a sequence's tiles one after the other: 24 packed sequences of up to
// 1500 tokens ended with a long one that began late); without a mask the tiles of
// a sequence have the same work and follow each other.
template <bool kKeys, int rows>
__device__ __forceinline__ int find_tile(const Attn& p, int t, AttnTile& o) {
  const int T = kKeys ? p.Tk : p.Tq;
  if (!p.seqs_q) {
    const int per = ((kKeys ? p.Lk : p.Lq) + rows - 1) / rows;
    const int rank = (int)((uint32_t)t / p.by_batch), b = t - rank * p.batch;
    o = {b * p.Lq, p.Lq, b * p.Lk, p.Lk, (kKeys ? rank : per - 1 - rank) * rows};
    return -1;
  }
  if (p.batch > kScan) return search_tile<kKeys, rows>(p, t, o);
  const int32_t* seqs = kKeys ? p.seqs_k : p.seqs_q;
  const int lane = threadIdx.x & 31;
  bool bad = false;
  int next[4] = {0, 0, 0, 0};  // tiles of the lane's sequences, of four steps at a time
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    if (b0 % 128 == 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int b = b0 + 32 * k + lane;
        next[k] = 0;
        if (b < p.batch) {
          const int2 r = seq_rows(seqs, b, T, bad);
          next[k] = (r.y - r.x + rows - 1) / rows;
        }
      }
    }
    const int n = next[0];
    next[0] = next[1], next[1] = next[2], next[2] = next[3];
    const int all = __reduce_add_sync(0xffffffffu, n);
    if (t < all) {
      int first, index;  // the sequence's lane, and the tile of it
      if (p.causal) {
        int work = __reduce_max_sync(0xffffffffu, n);
        unsigned mask;
        while (t >= __popc(mask = __ballot_sync(0xffffffffu, n >= work))) {
          t -= __popc(mask);
          --work;
        }
        const bool mine = n >= work && __popc(mask & ((1u << lane) - 1)) == t;
        first = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        index = kKeys ? __shfl_sync(0xffffffffu, n, first) - work : work - 1;
      } else {
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += v;
        }
        first = __ffs(__ballot_sync(0xffffffffu, sum > t)) - 1;
        index = __shfl_sync(0xffffffffu, sum, first) - 1 - t;
      }
      const int2 q = seq_rows(p.seqs_q, b0 + first, p.Tq, bad);
      const int2 k = seq_rows(p.seqs_k, b0 + first, p.Tk, bad);
      if (bad) raise_flag(p.status, HLQ_DEV_BADCODE);
      o = {q.x, q.y - q.x, k.x, k.y - k.x, index * rows};
      return -1;
    }
    t -= all;
  }
  if (bad) raise_flag(p.status, HLQ_DEV_BADCODE);
  return t;
}

// Tiles of all sequences, at most, and those for the rows outside them: sequence
// i has at most n_i / rows + (rows - 1) / rows tiles, and the n rows outside take at
// most n / rows + 1.  (By search: the tiles before the first sequence's and from
// T' / rows + batch on, T' its last row, are no fewer.)
inline int64_t most_tiles(const Attn& p, bool keys, int rows) {
  const int64_t T = keys ? p.Tk : p.Tq;
  if (!p.seqs_q) return (T / p.batch + rows - 1) / rows * p.batch;
  return (T + rows - 1) / rows + p.batch + 1;
}

// Rows of chunk `chunk` of the rows that belong to no sequence (before the
// first and behind the last), a warp for each: calls f(row, d) for this thread's
// elements, d from 0 to D - 1.
template <bool kKeys, typename F>
__device__ __forceinline__ void outside_rows(const Attn& p, int rows, int chunk, F&& f) {
  if (!p.seqs_q) return;
  const int32_t* seqs = kKeys ? p.seqs_k : p.seqs_q;
  const int T = kKeys ? p.Tk : p.Tq;
  bool bad = false;
  const int front = seq_rows(seqs, 0, T, bad).x;
  const int back = max(front, seq_rows(seqs, p.batch - 1, T, bad).y);
  const int64_t first = (int64_t)chunk * rows, n = (int64_t)front + (T - back);
#pragma unroll 1
  for (int64_t i = first + threadIdx.x / 32; i < first + rows && i < n; i += blockDim.x / 32)
#pragma unroll 1
    for (int d = threadIdx.x % 32; d < p.D; d += 32)
      f((int)(i < front ? i : back + (i - front)), d);
}

// Keys that query i of a tile's sequence sees: the last query sees all of
// them, each one before it one fewer.  (The difference first: a sum of two
// lengths may leave 32 bits.)
__device__ __forceinline__ int keys_of(const Attn& p, const AttnTile& t, int i) {
  return p.causal ? max(0, min(t.nk, i + 1 + (t.nk - t.nq))) : t.nk;
}

}  // namespace hlq
