"""The operators around the layer at the ends of fp32's range, in the kernels
that only some sizes and alignments reach, and beside other threads.  The
bounds are those of test_gpu_step_ops.py; what a test adds to them it states.
"""
import math

import numpy as np
import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
from tests.test_gpu_step_ops import (BF16, EPS, F32, OUT_U, U, _clean_status, _lib,  # noqa: F401
                                     check, check_clip, check_norm, check_norm_bwd, check_policy,
                                     dev, e_logp, f64, logits_case, logsoftmax64, norm64,
                                     policy_inputs, rng)

pytestmark = pytest.mark.gpu

MIN = {dt: float(torch.finfo(dt).min) for dt in (F32, BF16)}


# ---------------------------------------------------------------------------
# the policy loss where logits are huge
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("V", [37, 500, 70001, 300007])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("scale", [1.0, 0.7, 3.0])
def test_policy_gradient_of_huge_logits(V, dt, scale):
    """Rows whose every logit is one huge number (a whole vocabulary masked by
    it) have a uniform distribution; one logit far above the rest has
    probability 1; a few left by a mask share it."""
    T = 8
    z, a, old, adv, w, ref = policy_inputs(T, V, dt, rng(T, V, 61), scale, 0.2, 0.28)
    w[:] = 1.0 / T
    for t, v in enumerate((-1e10, MIN[dt], 1e10, -1e30, 1e30)):
        z[t] = v
    z[5, 3], a[5] = 1e10, 3                    # one token is all there is
    z[6, 5:], a[6] = MIN[dt], 1                # five tokens left
    z[7] = -MIN[dt]
    lp = logsoftmax64(f64(z) * scale)[np.arange(T), f64(a).astype(int)]
    ratio = np.array([1.1, 0.9, 1.0, 0.5, 2.0, 1.05, 0.95, 1.1])
    old, ref = dev(lp - np.log(ratio)), dev(lp + 0.3)
    got = hlq.hlq_policy_loss(z, a, old, adv, w, ref_logp=ref, kl_coef=0.05, clip_high=0.28,
                              scale=scale)
    check_policy(got, z, a, old, adv, w, ref, scale, 0.2, 0.28, 0.05, 1.0)
