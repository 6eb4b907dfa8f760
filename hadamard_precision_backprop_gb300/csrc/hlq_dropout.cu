// hlq_dropout.cu -- dropout whose mask is drawn again wherever it is needed.
//
//   y[t, c] = kept(e) ? x[t, c] 65536 / (65536 - drop) : 0   (+ residual[t, c])
//
// with e = t C + c, drop = round(65536 p), kept(e) = u16(e) >= drop, and u16(e)
// the e-th of the 16-bit halves of the Philox4x32-10 words of the blocks 0, 1,
// 2, ..: a block serves eight elements, i.e. one 16-byte piece of bf16.
//
// Four bytes (six with the residual) an element in bf16 leave about 22 (32)
// issue slots for it at the copy rate.  Philox takes some 160 for a block: a
// 32-bit word for each element would cost as much as the copy allows, 16 bits
// cost half of that.  Without a residual the drawing still bounds it: 16384 x
// 4096 in bf16 50 us against 39 with p = 0.
#include "hlq_kernels.h"
#include "hlq_rows.cuh"

namespace hlq {
namespace {

constexpr int kThreads = 256;
// Blocks of a thread, all loads first: 16384 x 4096 in bf16 with a residual 65 us
// (0.91 of the copy rate) with two, 67 with one, 98 with four.
constexpr int kBlocks = 2;
constexpr uint32_t kStream = 4;  // of the counter; 0 to 3 are the quantizers'

// Where the eight elements of a block are: kDense: one after the other in all
// tensors (16-byte aligned); kEights: in one row (rows of whole blocks, 16-byte
// aligned); kAny: by single elements.
enum Place { kDense, kEights, kAny };

// The bits of block b's element k, as drawn.
__device__ __forceinline__ uint32_t half_of(const U4& w, int k) {
  const uint32_t word = k < 4 ? (k < 2 ? w.x : w.y) : (k < 6 ? w.z : w.w);
  return k & 1 ? word >> 16 : word & 0xffffu;
}

// Without a residual nothing is added: -0 + 0 would be 0.
template <bool kResidual>
__device__ __forceinline__ float scaled(float x, float scale, float other) {
  return kResidual ? fmaf(x, scale, other) : x * scale;
}

template <int kPlace, bool kX, bool kY, bool kResidual>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const Dropout p) {
  pdl_trigger();
  pdl_wait();
  const int64_t n = p.T * p.C, blocks = (n + 7) / 8;
  uint64_t seed = p.seed;
  if (p.d_seed) {
    const uint2 v = ld_dep_u2(p.d_seed);
    seed += (uint64_t)v.y << 32 | v.x;
  }
  const int64_t first = (int64_t)blockIdx.x * kThreads * kBlocks + threadIdx.x;
  F8 x[kBlocks], r[kBlocks];  // all on their way before the first is used
  if (kPlace != kAny) {
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const int64_t e = 8 * (first + i * kThreads);
      if (e + 8 > n) break;
      const int64_t row = kPlace == kDense ? 0 : e / p.C, col = e - row * p.C;
      x[i] = load8(p.x, kX, row * p.ldx + col);
      if (kResidual) r[i] = load8(p.residual, kY, row * p.ldr + col);
    }
  }
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    const int64_t b = first + i * kThreads, e = 8 * b;
    if (b >= blocks) break;
    U4 w = {0, 0, 0, 0};
    if (p.drop > 0) w = philox_block(seed, kStream, (uint64_t)b);
    const int64_t row = kPlace == kDense ? 0 : e / p.C, col = e - row * p.C;
    if (kPlace != kAny && e + 8 <= n) {
      F8 y;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float other = kResidual ? r[i].v[k] : 0.f;
        y.v[k] = half_of(w, k) >= p.drop ? scaled<kResidual>(x[i].v[k], p.scale, other) : other;
      }
      store8(p.y, kY, row * p.ldy + col, y);
    } else {
      int64_t t = row, c = col;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (e + k >= n) break;
        const float other = kResidual ? load_elem(p.residual, kY, t * p.ldr + c) : 0.f;
        store_elem(p.y, kY, t * p.ldy + c,
                   half_of(w, k) >= p.drop
                       ? scaled<kResidual>(load_elem(p.x, kX, t * p.ldx + c), p.scale, other)
                       : other);
        if (++c == p.C && kPlace != kDense) c = 0, ++t;
      }
    }
  }
}

template <int kPlace, bool kX, bool kY, bool kResidual>
cudaError_t launch(const Dropout& p, cudaStream_t st) {
  const int64_t blocks = (p.T * p.C + 7) / 8, per = kThreads * kBlocks;
  const int64_t grid = (blocks + per - 1) / per;
  if (grid >= (int64_t)1 << 31) return cudaErrorInvalidValue;
  return launch_pdl(dropout_kernel<kPlace, kX, kY, kResidual>, dim3((unsigned)grid),
                    dim3(kThreads), 0, st, p);
}

template <int kPlace, bool kX, bool kY>
cudaError_t launch_types(const Dropout& p, cudaStream_t st) {
  return p.residual ? launch<kPlace, kX, kY, true>(p, st) : launch<kPlace, kX, kY, false>(p, st);
}

template <int kPlace>
cudaError_t launch_place(const Dropout& p, cudaStream_t st) {
  if (p.x_bf16)
    return p.y_bf16 ? launch_types<kPlace, true, true>(p, st)
                    : launch_types<kPlace, true, false>(p, st);
  return p.y_bf16 ? launch_types<kPlace, false, true>(p, st)
                  : launch_types<kPlace, false, false>(p, st);
}

bool aligned16_at(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

cudaError_t launch_dropout(const Dropout& p, cudaStream_t st) {
  const bool dense = p.T <= 1 || (p.ldx == p.C && p.ldy == p.C && (!p.residual || p.ldr == p.C));
  if (dense && aligned16_at(p.x) && aligned16_at(p.y) && aligned16_at(p.residual))
    return launch_place<kDense>(p, st);
  if (rows_of_eight(p.x, p.ldx, p.x_bf16, p.T, p.C) &&
      rows_of_eight(p.residual, p.ldr, p.y_bf16, p.T, p.C) &&
      rows_of_eight(p.y, p.ldy, p.y_bf16, p.T, p.C))
    return launch_place<kEights>(p, st);
  return launch_place<kAny>(p, st);
}

}  // namespace hlq
