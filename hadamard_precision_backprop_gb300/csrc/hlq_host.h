// hlq_host.h -- host helpers shared by the files of the C ABI: the status
// word's address, launch tracing, alignment, the launch macros (internal).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "hlq.h"

namespace hlq {

constexpr int kMaxDevices = 64;

// Address of the status word on the current device (looked up once).
unsigned int* device_status_ptr();

// SMs of the current device (looked up once); 0 on failure.
int device_sm_count();

// Around every kernel launch: two events while tracing is on.
void trace_before(cudaStream_t s);
void trace_after(const char* what, cudaStream_t s);

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

}  // namespace hlq

#define HLQ_TRY(expr)                                  \
  do {                                                 \
    cudaError_t _e = (expr);                           \
    if (_e != cudaSuccess) return HLQ_ERR_CUDA;        \
  } while (0)

// A kernel launch: traced when tracing is on.
#define HLQ_LAUNCH(name, s, expr)                      \
  do {                                                 \
    trace_before(s);                                   \
    cudaError_t _e = (expr);                           \
    if (_e != cudaSuccess) return HLQ_ERR_CUDA;        \
    trace_after(name, s);                              \
  } while (0)
