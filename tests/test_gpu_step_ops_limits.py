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


# ---------------------------------------------------------------------------
# layer norm where squares leave fp32's range
# ---------------------------------------------------------------------------
def check_norm_range(got, h, w, b, y_dt, eps):
    """check_norm with everything in units of the row's deviation, and half an
    ulp of a subnormal rstd (2^-150) more."""
    C = h.shape[1]
    n = (C / 32 + 32) * U
    y, mean, rstd = norm64(h, w, b, eps)
    unit = 1 / rstd
    e_mean = (n + 2 * U) * np.abs(h).mean(1)
    d = np.abs(h - mean[:, None])
    e_d = U * d + e_mean[:, None] + U * np.abs(h)
    e_var = 2 * (d * e_d).mean(1) + np.square(e_d).mean(1) + (n + 4 * U) * np.square(d).mean(1)
    var = np.square(d).mean(1) + eps
    r_rstd = e_var / (2 * var) * (1 + e_var / var) + 4 * U
    check(f64(got[1]) / unit, mean / unit, e_mean / unit, "mean")
    check(f64(got[2]) * unit, 1.0, r_rstd + 2.0 ** -150 * unit, "rstd")
    e_y = (np.abs(w) * rstd[:, None] * (e_d + d * (r_rstd[:, None] + 4 * U))
           + 2 * U * np.abs(b) + 2 * OUT_U[y_dt] * np.abs(y))
    check(got[0], y, e_y, "y")


# teams of 8, 32, 128 and 512 threads; the element ring's three; 1024 threads; long rows
WIDTHS = [64, 768, 4096, 16384, 77, 1001, 5663, 9001, 16387, 40000]


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dt", [F32, BF16])
def test_layer_norm_range(C, dt):
    """Finite rows of any size, beside ordinary ones: no flag, right results."""
    r = rng(C, 62)
    T = 9
    w, b = dev(1 + 0.2 * r.normal(size=C)), dev(r.normal(size=C))
    x = r.normal(size=(T, C))
    for t, s in enumerate((1.0, 1e17, 3e19, 1e25, 1e37, 1e-10)):
        x[t] *= s
    x[6] = r.uniform(-3.3e38, 3.3e38, C)
    x[7] = 2e38 * (1 + 0.05 * r.normal(size=C))        # the sum itself leaves the range
    x = dev(x, dt)
    check_norm_range(hlq.hlq_layer_norm(x, w, b, eps=EPS), f64(x), f64(w), f64(b), dt, EPS)
    res = dev(f64(x) * 0.25, dt)
    x[6:8] *= 0.5
    got = hlq.hlq_layer_norm(x, w, b, eps=EPS, residual=res, out_dtype=F32)
    check_norm_range(got, f64(x) + f64(res), f64(w), f64(b), F32, EPS)


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dt", [F32, BF16])
def test_layer_norm_range_without_eps(C, dt):
    """Small rows, nothing added to the variance."""
    r = rng(C, 63)
    x = r.normal(size=(6, C))
    for t, s in enumerate((1e-18, 1e-22, 1e-30, 1e-37, 1.0, 1e30)):
        x[t] *= s
    x = dev(x, dt)
    check_norm_range(hlq.hlq_layer_norm(x, eps=0.0), f64(x), 1.0, 0.0, dt, 0.0)


@pytest.mark.parametrize("C", [64, 768, 4096, 16384, 77, 1001, 5663, 9001, 40000])
def test_layer_norm_range_in_place(C):
    """Rows taken once more are read again: what is written over them comes last."""
    r = rng(C, 68)
    x, res = r.normal(size=(6, C)), r.normal(size=(6, C))
    x[1:5] *= 3e30
    res[2:4] *= 1e30
    x, res = dev(x), dev(res)
    want = hlq.hlq_layer_norm(x, residual=res)
    a, c = x.clone(), res.clone()
    got = hlq.hlq_layer_norm(a, residual=c, out=a, h=c)
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    a, c = x.clone(), res.clone()
    got = hlq.hlq_layer_norm(a, residual=c, out=c, h=a)
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    a = x.clone()
    assert torch.equal(hlq.hlq_layer_norm(a, out=a)[0], hlq.hlq_layer_norm(x)[0])


def test_layer_norm_flags_rows_without_statistics():
    """What is still reported: infinity, NaN, no variance at all with eps 0."""
    for C in (64, 1001, 20000):
        for bad in (float("inf"), -float("inf"), float("nan")):
            x = torch.randn(4, C, device="cuda") * 1e30
            x[2, C // 2] = bad
            y, _, rstd = hlq.hlq_layer_norm(x)
            assert hlq.hlq_read_device_status(clear=True) == hlq.DEV_NONFINITE
            assert bool(torch.isnan(y[2]).any()) and bool(torch.isfinite(y[[0, 1, 3]]).all())
        y, _, rstd = hlq.hlq_layer_norm(torch.zeros(4, C, device="cuda"), eps=0.0)
        assert bool(torch.isinf(rstd).all())
        assert hlq.hlq_read_device_status(clear=True) == hlq.DEV_NONFINITE
        y, mean, rstd = hlq.hlq_layer_norm(torch.zeros(4, C, device="cuda"), eps=1e-30)
        assert not y.any() and not mean.any()
        check(rstd, 1e15, 8 * U * 1e15, "rstd of a zero row")


# ---------------------------------------------------------------------------
# its backward pass there
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T", [6, 700])
@pytest.mark.parametrize("C", [264, 768, 1024, 2048, 4096, 14336, 77, 1001, 5663, 20001])
@pytest.mark.parametrize("x_dt,gy_dt", [(F32, F32), (BF16, BF16)])
def test_layer_norm_backward_range(T, C, x_dt, gy_dt):
    """rstd whose square leaves fp32's range (deviations of 1e20 and more, or
    of 1e-20 and less): xhat, and with it g_x, is an ordinary number."""
    r = rng(T, C, 64)
    s = np.resize([1.0, 3e19, 1e30, 1e37, 1e-25, 1e-37], T)
    x = r.normal(size=(T, C)) * s[:, None]
    x[3] = r.uniform(-1.6e38, 1.6e38, C)       # differences up to the end of the range
    x = dev(x, x_dt)
    w = dev(1 + 0.2 * r.normal(size=C))
    _, mean, rstd = norm64(f64(x), 1.0, 0.0, 0.0)
    mean, rstd = dev(mean), dev(rstd)
    gy = dev(r.normal(size=(T, C)) * np.resize([1.0, 1.0, 1.0, 1e6, 1.0, 1e-3], T)[:, None], gy_dt)
    got = hlq.hlq_layer_norm_backward(gy, x, mean, rstd, w, out_dtype=F32)
    check_norm_bwd(got, gy, x, mean, rstd, w, None)


# ---------------------------------------------------------------------------
# softmax temperatures at the end of the range
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("V", [50, 40000, 300007])
@pytest.mark.parametrize("T", [3, 700])
def test_vocabulary_rows_with_a_huge_scale(T, V):
    """scale * log2(e) above fp32's range: equal logits still share the
    probability, and the largest takes it from smaller ones."""
    if T > 3 and V > 100000:
        T = 500
    z = torch.zeros((T, V), device="cuda")
    z[1, 7] = 1e-3
    a = torch.full((T,), 7, device="cuda")
    want = np.full(T, -math.log(V))
    want[1] = 0.0
    tol = e_logp(np.zeros(1), want, V)
    logp, _ = hlq.hlq_token_logprobs(z, a, scale=3e38)
    check(logp, want, tol, "logp")
    ones = torch.ones(T, device="cuda")
    stats, logp, g = hlq.hlq_policy_loss(z, a, logp, ones, ones / T, scale=3e38, grad_scale=1e-38)
    check(logp, want, tol, "logp")
    assert bool(torch.isfinite(stats).all()) and bool(torch.isfinite(g).all())


# ---------------------------------------------------------------------------
# clipping that is switched off
# ---------------------------------------------------------------------------
def test_clip_grad_norm_without_a_limit_keeps_gradients():
    """max_norm = inf clips nothing, an infinite gradient beside it or not."""
    for bad in (float("inf"), -float("inf")):
        g = [torch.randn(300, device="cuda"), torch.randn(9000, device="cuda")]
        g[0][7] = bad
        want = [t.clone() for t in g]
        outs = [torch.empty_like(t) for t in g]
        nc = hlq.hlq_clip_grad_norm(g, float("inf"), outs=outs)
        assert nc.tolist() == [float("inf"), 1.0]
        for o, t in zip(outs, want):
            assert torch.equal(o, t)
        assert hlq.hlq_clip_grad_norm(g, float("inf")).tolist() == [float("inf"), 1.0]
        for o, t in zip(g, want):
            assert torch.equal(o, t)
        only = hlq.hlq_clip_grad_norm(g, float("inf"), norm_only=True)
        assert only.tolist() == [float("inf"), 1.0]
        assert hlq.hlq_read_device_status(clear=True) == hlq.DEV_NONFINITE
    g = [torch.full((300,), float("nan"), device="cuda")]
    assert bool(torch.isnan(hlq.hlq_clip_grad_norm(g, float("inf"))).all())
    assert hlq.hlq_read_device_status(clear=True) == hlq.DEV_NONFINITE


# ---------------------------------------------------------------------------
# other threads
# ---------------------------------------------------------------------------
def test_other_threads_run_while_a_call_waits():
    """A call that waits (its stream's queue of launches is full behind work
    that takes half a second) leaves the interpreter to other threads."""
    import threading
    import time

    from tests.test_gpu_step_ops import _calls

    for call in _calls():
        call()
        torch.cuda.synchronize()
        longest_gap, stop = [0.0], threading.Event()

        def tick():
            last = time.perf_counter()
            while not stop.is_set():
                time.sleep(0.002)
                now = time.perf_counter()
                longest_gap[0] = max(longest_gap[0], now - last)
                last = now

        thread = threading.Thread(target=tick)
        thread.start()
        try:
            torch.cuda._sleep(1_000_000_000)
            longest_call, until = 0.0, time.perf_counter() + 0.7
            while time.perf_counter() < until and longest_call < 0.2:
                t0 = time.perf_counter()
                call()
                longest_call = max(longest_call, time.perf_counter() - t0)
        finally:
            stop.set()
            thread.join()
        torch.cuda.synchronize()
        assert longest_call > 0.2, "no call waited: nothing was tested"
        assert longest_gap[0] < 0.1


# ---------------------------------------------------------------------------
# kernels that few sizes reach
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,C", [(3, 8193), (5, 9001), (2, 12345), (2, 16383), (400, 9001)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_layer_norm_of_odd_rows_above_8192(T, C, dt):
    """One element at a time, 1024 threads a row."""
    r = rng(T, C, 65)
    x, res = (dev(r.normal(size=(T, C)) + 0.5, dt) for _ in range(2))
    w, b = dev(r.normal(size=C), dt), dev(r.normal(size=C), dt)
    check_norm(hlq.hlq_layer_norm(x, w, b, out_dtype=F32), f64(x), f64(w), f64(b), F32)
    got = hlq.hlq_layer_norm(x, w, b, residual=res)
    h = f64(x) + f64(res)
    check(got[3], h, 2 * OUT_U[dt] * np.abs(h), "h")
    check_norm(got, h, f64(w), f64(b), dt)


@pytest.mark.parametrize("C", [1687, 1689, 2001, 2047, 2049, 7191, 7193, 8190, 8191])
def test_layer_norm_of_odd_fp32_rows_with_a_residual(C):
    """Around the widths whose two slots of a row do not fit a CTA's share of
    shared memory; rows enough to fill every stage again."""
    T = 5000 if C < 4000 else 1500
    r = rng(C, 66)
    x, res = dev(r.normal(size=(T, C))), dev(r.normal(size=(T, C)))
    w, b = dev(r.normal(size=C)), dev(r.normal(size=C))
    got = hlq.hlq_layer_norm(x, w, b, residual=res)
    h = f64(x) + f64(res)
    check(got[3], h, 2 * U * np.abs(h), "h")
    check_norm(got, h, f64(w), f64(b), F32)


@pytest.mark.parametrize("V,ld,off,ldg,offg", [(131073, 131073, 0, 131080, 3),
                                               (151671, 151680, 8, 151671, 1),
                                               (300007, 300010, 2, 300008, 0)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_policy_loss_of_long_rows_at_other_offsets(V, ld, off, ldg, offg, dt):
    """Rows that are read twice, the gradient's at another offset from 16 bytes."""
    T = 5
    z, a, old, adv, w, ref = policy_inputs(T, V, dt, rng(V, ldg), 1.0, 0.2, 0.2, ld, off)
    buf = torch.full((offg + T * ldg + 8,), 7.0, dtype=dt, device="cuda")
    out = buf[offg:].as_strided((T, V), (ldg, 1))
    got = hlq.hlq_policy_loss(z, a, old, adv, w, ref_logp=ref, kl_coef=0.1, out=out)
    check_policy(got, z, a, old, adv, w, ref, 1.0, 0.2, 0.2, 0.1, 1.0)
    touched = torch.zeros_like(buf, dtype=torch.bool)
    touched[offg:].as_strided((T, V), (ldg, 1)).fill_(True)
    assert bool((buf[~touched] == 7).all())


# ---------------------------------------------------------------------------
# log-probabilities of rows that lie elsewhere
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("V", [1001, 32003, 151671])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_logprobs_of_moved_rows(V, dt):
    """The same bits wherever a row lies at the same offset from a 16-byte
    boundary; at another offset its terms are added in another order, and both
    results stay within the bound of a log-probability."""
    T, step = 7, 16 // torch.empty(0, dtype=dt).element_size()
    z, a = logits_case(T, V, dt, rng(V, 67))
    at = torch.from_numpy(a).cuda()
    want = logsoftmax64(f64(z))[np.arange(T), a]
    here = hlq.hlq_token_logprobs(z, at)
    for off in range(step + 1):
        for t in range(T):
            buf = torch.zeros(off + V, dtype=dt, device="cuda")
            row = buf[off:].view(1, V)
            row.copy_(z[t:t + 1])
            got = hlq.hlq_token_logprobs(row, at[t:t + 1])
            if (t * V - off) % step == 0:
                assert torch.equal(got[0], here[0][t:t + 1])
                assert torch.equal(got[1], here[1][t:t + 1])
            check(got[0], want[t:t + 1], e_logp(f64(z), want[t:t + 1], V), "logp")
    check(here[0], want, e_logp(f64(z), want, V), "logp")
