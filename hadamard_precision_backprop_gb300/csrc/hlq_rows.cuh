// hlq_rows.cuh -- device and host pieces shared by the kernels that work on
// rows of bf16 / fp32 elements (layer norm, losses, clipping).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "hlq_device.cuh"

namespace hlq {

// Eight consecutive elements as fp32: one 16-byte access of bf16, two of
// fp32 (the address is 16-byte aligned).
struct F8 {
  float v[8];
};

__device__ __forceinline__ F8 widen8(uint4 r) {
  F8 o;
  o.v[0] = bf16_lo(r.x); o.v[1] = bf16_hi(r.x);
  o.v[2] = bf16_lo(r.y); o.v[3] = bf16_hi(r.y);
  o.v[4] = bf16_lo(r.z); o.v[5] = bf16_hi(r.z);
  o.v[6] = bf16_lo(r.w); o.v[7] = bf16_hi(r.w);
  return o;
}
__device__ __forceinline__ F8 join8(float4 a, float4 b) {
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
// Ordinary loads, not the read-only path: under programmatic dependent launch
// an earlier kernel may write the data while this one is already running.
__device__ __forceinline__ F8 load8(const void* p, bool bf16, int64_t i) {
  if (bf16) return widen8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
  const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  return join8(q[0], q[1]);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void store8(void* p, bool bf16, int64_t i, const F8& o) {
  if (bf16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack_bf16(o.v[0], o.v[1]), pack_bf16(o.v[2], o.v[3]),
                   pack_bf16(o.v[4], o.v[5]), pack_bf16(o.v[6], o.v[7]));
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(o.v[0], o.v[1], o.v[2], o.v[3]);
    q[1] = make_float4(o.v[4], o.v[5], o.v[6], o.v[7]);
  }
}

// Two fp32 in one register pair: one instruction for both.
struct F2 {
  unsigned long long b;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.b) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.b));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(a.b), "l"(b.b), "l"(c.b));
  return r;
}
__device__ __forceinline__ F2 widen2(uint32_t pair) { return f2(bf16_lo(pair), bf16_hi(pair)); }
__device__ __forceinline__ uint32_t pack_bf16(F2 a) {
  const float2 v = split(a);
  return pack_bf16(v.x, v.y);
}

// Four consecutive elements (aligned to four): one access of 8 bytes of bf16
// or 16 of fp32.
struct Quad {
  F2 v[2];
};
template <bool kBf16>
__device__ __forceinline__ Quad load4(const void* p, int64_t i) {
  if constexpr (kBf16) {
    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    return {{widen2(r.x), widen2(r.y)}};
  } else {
    const ulonglong2 r = *reinterpret_cast<const ulonglong2*>(static_cast<const float*>(p) + i);
    return {{{r.x}, {r.y}}};
  }
}
template <bool kBf16>
__device__ __forceinline__ void store4(void* p, int64_t i, const Quad& q) {
  if constexpr (kBf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
        make_uint2(pack_bf16(q.v[0]), pack_bf16(q.v[1]));
  else
    *reinterpret_cast<ulonglong2*>(static_cast<float*>(p) + i) =
        make_ulonglong2(q.v[0].b, q.v[1].b);
}

__device__ __forceinline__ float load_elem(const void* p, bool bf16, int64_t i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
              : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_elem(void* p, bool bf16, int64_t i, float v) {
  if (bf16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p)[i] = v;
}

// Rows that all begin on 16-byte boundaries and hold whole groups of eight.
inline bool rows_of_eight(const void* p, int64_t ld, bool bf16, int64_t T, int64_t C) {
  if (!p) return true;
  const uint64_t size = bf16 ? 2 : 4;
  return C % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 &&
         (T <= 1 || (uint64_t)ld * size % 16 == 0);
}

// Raise a kernel's dynamic shared-memory limit once per device (the call is
// not free, and launches come in the microseconds).
template <auto kKernel>
static cudaError_t allow_smem(size_t bytes) {
  static int done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev] >= (int)bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done[dev] = (int)bytes;
  return e;
}

}  // namespace hlq
