// hlq_norm_ring_bf16.cu -- hlq_norm_ring.cuh for bf16 x.
#include "hlq_norm_ring_impl.cuh"

namespace hlq {

cudaError_t launch_norm_bwd_ring_bf16(const NormBwd& p, const RingPlan& r, cudaStream_t st) {
  return p.gy_bf16 ? pick_ring<true, true>(p, r, st) : pick_ring<true, false>(p, r, st);
}

}  // namespace hlq
