// hlq_norm_ring.cuh -- the layer norm's backward pass over rows of aligned
// groups of eight elements: the plan that host and kernel share, and the
// launchers, one file for each type of x.
#pragma once

#include "hlq_kernels.h"

namespace hlq {

constexpr int kMostUnits = 8;    // groups of four columns a thread owns
constexpr int kMostSlabs = 640;  // CTAs of the ring, and slabs of partial sums

// Threads of a CTA at most: 16 warps of up to 128 registers, or 24 where two
// groups of columns a thread leave room for that.
constexpr int ring_threads(int team, int units) {
  return team > 32 ? team : units <= 2 ? 768 : 512;
}

struct RingPlan {
  int team, units;  // threads of a team, groups of four columns of each
  int teams, stages, stage_bytes, grid;
  int before;       // bytes of a CTA's shared memory before its rings
  int cluster;      // the CTAs (all of them) are one cluster and join the sums
                    // themselves; 0: they write slabs
  size_t smem, smem_most;
};
bool norm_bwd_ring_plan(const NormBwd& p, int sms, RingPlan* out);
cudaError_t launch_norm_bwd_ring_bf16(const NormBwd& p, const RingPlan& r, cudaStream_t st);
cudaError_t launch_norm_bwd_ring_f32(const NormBwd& p, const RingPlan& r, cudaStream_t st);


// Rows of any length and alignment, up to 8192 elements, whose stages fit a CTA's
// share of shared memory (forward, fp32 with a residual: not those of 1689 to
// 2048 and above 7192): hlq_norm_elem.cu.
bool norm_fwd_elem_plan(const NormFwd& p, int sms, RingPlan* out);
cudaError_t launch_norm_fwd_elem(const NormFwd& p, const RingPlan& r, cudaStream_t st);
bool norm_bwd_elem_plan(const NormBwd& p, int sms, RingPlan* out);
cudaError_t launch_norm_bwd_elem(const NormBwd& p, const RingPlan& r, cudaStream_t st);

}  // namespace hlq
