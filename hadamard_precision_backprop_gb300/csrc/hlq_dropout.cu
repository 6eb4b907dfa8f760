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
// cost half of that.
#include "hlq_kernels.h"
#include "hlq_rows.cuh"

namespace hlq {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kStream = 4;  // of the counter; 0 to 3 are the quantizers'

// Where the eight elements of a block are: kDense: one after the other in all
// tensors (16-byte aligned); kEights: in one row (rows of whole blocks, 16-byte
// aligned); kAny: by single elements.
enum Place { kDense, kEights, kAny };

template <int kPlace, bool kX, bool kY>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const Dropout p, int per_thread) {
  pdl_trigger();
  pdl_wait();
  const int64_t n = p.T * p.C, blocks = (n + 7) / 8;
  uint64_t seed = p.seed;
  if (p.d_seed) {
    const uint2 v = ld_dep_u2(p.d_seed);
    seed += (uint64_t)v.y << 32 | v.x;
  }
  int64_t b = (int64_t)blockIdx.x * kThreads * per_thread + threadIdx.x;
  for (int i = 0; i < per_thread && b < blocks; ++i, b += kThreads) {
    const int64_t e = 8 * b;
    const bool whole = e + 8 <= n;
    const int64_t row = kPlace == kDense ? 0 : e / p.C, col = kPlace == kDense ? e : e - row * p.C;
    F8 x, r;
    if (kPlace != kAny && whole) {
      x = load8(p.x, kX, row * p.ldx + col);
      if (p.residual) r = load8(p.residual, kY, row * p.ldr + col);
    }
    U4 w = {0, 0, 0, 0};
    if (p.drop > 0) w = philox_block(seed, kStream, (uint64_t)b);
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    if (kPlace != kAny && whole) {
      F8 y;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t u = k & 1 ? words[k / 2] >> 16 : words[k / 2] & 0xffffu;
        const float other = p.residual ? r.v[k] : 0.f;
        y.v[k] = u >= p.drop ? fmaf(x.v[k], p.scale, other) : other;
      }
      store8(p.y, kY, row * p.ldy + col, y);
    } else {
      int64_t t = row, c = col;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (e + k < n) {
          const uint32_t u = k & 1 ? words[k / 2] >> 16 : words[k / 2] & 0xffffu;
          const float other = p.residual ? load_elem(p.residual, kY, t * p.ldr + c) : 0.f;
          store_elem(p.y, kY, t * p.ldy + c,
                     u >= p.drop ? fmaf(load_elem(p.x, kX, t * p.ldx + c), p.scale, other) : other);
          if (++c == p.C && kPlace != kDense) c = 0, ++t;
        }
      }
    }
  }
}

template <int kPlace>
cudaError_t launch(const Dropout& p, cudaStream_t st) {
  const auto kernel = p.x_bf16 ? (p.y_bf16 ? dropout_kernel<kPlace, true, true>
                                           : dropout_kernel<kPlace, true, false>)
                               : (p.y_bf16 ? dropout_kernel<kPlace, false, true>
                                           : dropout_kernel<kPlace, false, false>);
  const int64_t blocks = (p.T * p.C + 7) / 8;
  const int per_thread = 1;
  const int64_t grid = (blocks + (int64_t)kThreads * per_thread - 1) / ((int64_t)kThreads * per_thread);
  if (grid >= (int64_t)1 << 31) return cudaErrorInvalidValue;
  return launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), 0, st, p, per_thread);
}

bool aligned16_at(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

cudaError_t launch_dropout(const Dropout& p, cudaStream_t st) {
  const bool dense = p.T <= 1 || (p.ldx == p.C && p.ldy == p.C && (!p.residual || p.ldr == p.C));
  if (dense && aligned16_at(p.x) && aligned16_at(p.y) && aligned16_at(p.residual))
    return launch<kDense>(p, st);
  if (rows_of_eight(p.x, p.ldx, p.x_bf16, p.T, p.C) &&
      rows_of_eight(p.residual, p.ldr, p.y_bf16, p.T, p.C) &&
      rows_of_eight(p.y, p.ldy, p.y_bf16, p.T, p.C))
    return launch<kEights>(p, st);
  return launch<kAny>(p, st);
}

}  // namespace hlq
