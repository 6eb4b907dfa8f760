// hlq_attn_tc.cuh -- tensor-core pieces of the attention kernels (tcgen05, TMEM,
// TMA tiles of heads).
//
// A tile of R rows of a head lies in shared memory as TMA writes it with the
// 128-byte swizzle: chunk c (columns 64 c .. 64 c + 63) is R rows of 128 bytes,
// chunks R x 128 bytes apart.  The same tile serves as an operand whose rows
// are the product's rows and whose columns are summed over (K-major, eight rows
// 1024 bytes apart) or the other way round (MN-major: eight rows are again
// 1024 bytes apart, and the chunks are the leading dimension's step).
// Probabilities and their gradients never leave TMEM: the warps that compute
// them write them back as bf16 pairs, lane = row, and the next product takes
// them from there as its first operand.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>

#include "hlq_attn.cuh"
#include "hlq_tma.cuh"

namespace hlq {
namespace tc {

constexpr int kRows = 128;        // rows of a tile
constexpr int kChunk = 64;        // columns of a chunk
constexpr uint32_t kChunkBytes = kRows * 128;

__device__ __forceinline__ void prefetch(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Matrix descriptors: the low word holds the tile's address and the leading
// step, the high word is the same for all.  Operands are taken in steps of 16
// columns (rows), which are constants added to the low word: a product of 128 x
// 128 x 16 takes 64 clocks, and the one thread that issues them has no time for
// more (descriptors put together for each of them: 110 to 130 clocks).
constexpr uint32_t kDescHigh = 1024 >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint64_t desc(uint32_t low) { return (uint64_t)kDescHigh << 32 | low; }
// The address of a descriptor is the one within the CTA: in a cluster the higher
// bits of a shared address tell the CTA, and would be read as the leading step.
__device__ __forceinline__ uint32_t desc_address(uint32_t tile) { return (tile & 0x3FFFFu) >> 4; }
// Columns summed over (the leading step is not used), or rows.
__device__ __forceinline__ uint32_t by_columns(uint32_t tile) {
  return desc_address(tile) | 1u << 16;
}
__device__ __forceinline__ uint32_t by_rows(uint32_t tile, int rows = kRows) {
  return desc_address(tile) | (uint32_t)rows * 128 >> 4 << 16;
}
__host__ __device__ constexpr uint32_t column_step(int k, int rows = kRows) {
  return ((uint32_t)(k >> 2) * (rows * 128) + (uint32_t)(k & 3) * 32) >> 4;
}
__host__ __device__ constexpr uint32_t row_step(int k) { return (uint32_t)k * 16 * 128 >> 4; }

// 16 more columns summed over, of which the first three hold a number for each
// row (see hlq_attn_bwd_tc.cu): [128 x 16] without swizzle, 8 rows x 16 bytes
// together, the two halves of a row 128 bytes and eight rows 256 bytes apart.
constexpr uint32_t kMoreBytes = kRows * 32;
__device__ __forceinline__ uint64_t more_columns(uint32_t tile) {
  return (uint64_t)(256 >> 4 | 1u << 14) << 32 | (desc_address(tile) | (128u >> 4) << 16);
}
__device__ __forceinline__ uint32_t more_at(int row) { return (row >> 3) * 256 + (row & 7) * 16; }

// One thread of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      :
      : "memory");
  return r != 0;
}

// Bounded wait, as mbar_wait, for waits that a product or a softmax hangs on: the
// time and the abort flag are looked at every 64th try only (reading the timer
// takes long enough to be missed on every wait).
__device__ __forceinline__ bool gives_up(uint32_t& t0, volatile int* abort_flag,
                                         unsigned int* status, int steps = 1) {
  if (*abort_flag) return true;
  const uint32_t t = (uint32_t)(now_ns() >> 16);  // in 32 bits: one register less in each wait
  if (t0 == 0) t0 = t;
  const unsigned long long limit = (kWaitNs >> 16) * steps;
  if (t - t0 <= (uint32_t)(limit < 1u << 31 ? limit : 1u << 31)) return false;
  if (atomicExch((int*)abort_flag, 1) == 0) atomicOr(status, HLQ_DEV_TIMEOUT);
  return true;
}
// By one thread.
__device__ __forceinline__ bool wait_lane(uint64_t* b, uint32_t phase, volatile int* abort_flag,
                                          unsigned int* status) {
  uint32_t t0 = 0;
  for (uint32_t i = 1; !mbar_test(b, phase & 1); ++i)
    if (i % 64 == 0 && gives_up(t0, abort_flag, status)) return false;
  return true;
}
// By a whole warp: one lane may see the phase where another would give up, so the
// lanes vote on both, and the result is the warp's.  `steps`: what is waited for
// comes after so many steps of the CTA's, each of which has the limit (where one of
// them takes longer, the warp that waits for it gives up, and all others with it).
template <typename F>
__device__ __forceinline__ bool wait_warp(volatile int* abort_flag, unsigned int* status,
                                          F&& test, int steps = 1) {
  uint32_t t0 = 0;
  for (uint32_t i = 1; !__all_sync(0xffffffffu, test()); ++i)
    if (i % 64 == 0 && __any_sync(0xffffffffu, gives_up(t0, abort_flag, status, steps))) return false;
  return true;
}

// bf16 x bf16 -> fp32, 128 x n; b_by_rows: the second operand's rows are summed over.
__host__ __device__ constexpr uint32_t idesc(int n, bool b_by_rows) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_by_rows ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
         (uint32_t)(kRows >> 4) << 24;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(add ? 1u : 0u)
      : "memory");
}
// The first operand from TMEM: lane = row, a column holds two of the 16 summed over.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(add ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          saddr(bar))
      : "memory");
}

// d [128 x kN] = A B^T over the first `steps` x 16 columns of both tiles (of
// kSteps at most).  B has kN rows.
template <int kSteps, int kN = kRows>
__device__ __forceinline__ void product_of_rows(uint32_t d, uint32_t a, uint32_t b, int steps) {
  constexpr uint32_t id = idesc(kN, false);
#pragma unroll
  for (int k = 0; k < kSteps; ++k)
    if (k < steps)
      mma_ss(d, desc(a + column_step(k)), desc(b + column_step(k, kN)), id, k > 0);
}
// d [128 x n] (+)= P B over rows 64 half .. of B; these columns of P are in TMEM
// from p on.
__device__ __forceinline__ void product_of_p(uint32_t d, uint32_t p, uint32_t b, uint32_t id,
                                             int half, bool add) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    mma_ts(d, p + 8 * k, desc(b + row_step(4 * half + k)), id, add || k > 0);
}

// 32 columns of this thread's TMEM lane; the values are there after ld_wait.
__device__ __forceinline__ void ld32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
      "[%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
// The registers pass through the wait, so that nothing that reads them can go
// before it.
__device__ __forceinline__ void ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
               :
               : "memory");
  asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void alloc(uint32_t* holder, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   saddr(holder)),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc(uint32_t base, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns)
               : "memory");
}

// After a wait gave up: lets the products issued so far come to their end (for
// two seconds at most), before shared memory and TMEM go.
__device__ __forceinline__ void drain(uint64_t* bar) {
  commit(bar);
  const unsigned long long t0 = now_ns();
  while (!mbar_test(bar, 0) && now_ns() - t0 < kWaitNs) {
  }
}

// Registers of the calling warpgroup: together no more than the launch's.
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// 2^x, 0 for -infinity.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 64 columns (from c0 on) of the 32 rows that a warp has in TMEM, lane = row, to
// rows row0 .. row0 + n - 1 of x, times the lane's factor; zeros where the lane's
// `zero` says so (`none`: in all lanes, and TMEM is not read).
// With `wide` (rows of whole 16 bytes) they pass through shared memory, 8 KB of
// the warp's own, so that a store covers whole rows: a lane's own row piece by
// piece is 32 sectors for each store, which took 4000 clocks for 128 x 256 bf16.
__device__ __forceinline__ void store_64(uint8_t* stage, const Heads& x, bool bf16, int wide,
                                         int64_t row0, int n, int h, int c0, int D, uint32_t at,
                                         bool none, bool zero, float factor) {
  const int lane = threadIdx.x & 31;
  const int64_t to = row0 * x.token + (int64_t)h * x.head + c0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t o[32];
    __syncwarp();
    if (none) {
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = 0;
    } else {
      ld32(at + c0 + 32 * half, o);
      ld_wait(o);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(zero ? 0.f : factor * __uint_as_float(o[i]));
    if (!wide) {
      if (lane < n)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c0 + 32 * half + i < D) {
            const int64_t e = to + lane * x.token + 32 * half + i;
            if (bf16)
              static_cast<__nv_bfloat16*>(x.p)[e] = __float2bfloat16_rn(__uint_as_float(o[i]));
            else
              static_cast<float*>(x.p)[e] = __uint_as_float(o[i]);
          }
    } else if (bf16) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * half + c) ^ (lane & 7)) << 4)) =
            make_uint4(bf16x2(__uint_as_float(o[8 * c]), __uint_as_float(o[8 * c + 1])),
                       bf16x2(__uint_as_float(o[8 * c + 2]), __uint_as_float(o[8 * c + 3])),
                       bf16x2(__uint_as_float(o[8 * c + 4]), __uint_as_float(o[8 * c + 5])),
                       bf16x2(__uint_as_float(o[8 * c + 6]), __uint_as_float(o[8 * c + 7])));
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(stage + lane * 256 + (((8 * half + c) ^ (lane & 7)) << 4)) =
            make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
    }
  }
  __syncwarp();
  if (!wide) return;
  if (bf16) {
    const int c = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      if (r < n && c0 + 8 * c < D)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(x.p) + to + r * x.token + 8 * c) =
            *reinterpret_cast<const uint4*>(stage + r * 128 + ((c ^ (r & 7)) << 4));
    }
  } else {
    const int c = lane & 15;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 2 * i + (lane >> 4);
      if (r < n && c0 + 4 * c < D)
        *reinterpret_cast<uint4*>(static_cast<float*>(x.p) + to + r * x.token + 4 * c) =
            *reinterpret_cast<const uint4*>(stage + r * 256 + ((c ^ (r & 7)) << 4));
    }
  }
  __syncwarp();
}

// The same columns into 8 KB of shared memory as fp32, laid out as there.
__device__ __forceinline__ void stage_64(uint8_t* stage, int c0, uint32_t at, bool none,
                                         float factor) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t o[32];
    __syncwarp();
    if (none) {
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = 0;
    } else {
      ld32(at + c0 + 32 * half, o);
      ld_wait(o);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = none ? 0.f : factor * __uint_as_float(o[4 * c + k]);
      *reinterpret_cast<float4*>(stage + lane * 256 + (((8 * half + c) ^ (lane & 7)) << 4)) =
          make_float4(v[0], v[1], v[2], v[3]);
    }
  }
}

// Tile of kN rows of head h, chunk by chunk; `bar` expects its bytes.
template <int kChunks, int kN = kRows>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar,
                                          int h, int row) {
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(saddr(dst) + c * kN * 128),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c * kChunk), "r"(h), "r"(row), "r"(saddr(bar))
        : "memory");
}

// Zeros in rows `first` .. kN - 1 of a tile, by one warp: rows behind a sequence's
// last hold another sequence's values, and 0 times those need not be 0.
template <int kChunks, int kN = kRows>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int first) {
  const int lane = threadIdx.x & 31;
  for (int i = lane; i < (kN - first) * kChunks * 8; i += 32) {
    const int piece = i & 7, rest = i >> 3, c = rest % kChunks, r = first + rest / kChunks;
    *reinterpret_cast<uint4*>(tile + c * kN * 128 + r * 128 + piece * 16) =
        make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace tc

// Whether TMA can read x [T, H, D] of bf16 (a stride of 0 repeats rows, which
// a tensor map does not).
inline bool tma_heads(const Heads& x, int64_t T, int64_t H) {
  const auto stride = [](int64_t s, int64_t n) { return n <= 1 || (s > 0 && s % 8 == 0 && s < (int64_t)1 << 39); };
  return reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && stride(x.token, T) && stride(x.head, H);
}
// Map of x with boxes of `rows` tokens x 1 head x 64 columns, zeros outside.
bool heads_map(CUtensorMap* map, const Heads& x, int64_t T, int64_t H, int64_t D, int rows);

}  // namespace hlq
