// hlq_norm_ring_f32.cu -- hlq_norm_ring.cuh for f32 x.
#include "hlq_norm_ring_impl.cuh"

namespace hlq {

cudaError_t launch_norm_bwd_ring_f32(const NormBwd& p, const RingPlan& r, cudaStream_t st) {
  return p.gy_bf16 ? pick_ring<false, true>(p, r, st) : pick_ring<false, false>(p, r, st);
}

}  // namespace hlq
