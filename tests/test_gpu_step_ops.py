"""The operators around the layer in a training step against their formulas
in 64 bits: layer norm and its backward pass, token log-probabilities, the
policy loss with the gradient of the logits, the gradient norm and clipping.

Bounds.  u = 2^-24 is half an ulp of fp32; a sum of n terms in any order is
within n u times the sum of their magnitudes, and in the kernels' order (at
least 32 partial sums, joined by a tree) within (n / 32 + 32) u.  An output
rounded to bf16 adds 2^-9 of its value.  exp and log are taken to be within 4
ulp, and the argument of an exp adds its own rounding.
"""
import math

import numpy as np
import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
from hadamard_precision_backprop_gb300 import build as hbuild

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
OUT_U = {F32: U, BF16: 2.0 ** -9}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    hbuild.build()
    hlq.lib()


@pytest.fixture(autouse=True)
def _clean_status():
    hlq.hlq_read_device_status(clear=True)
    yield
    assert hlq.hlq_read_device_status(clear=True) == 0, "a device flag was raised"


def rng(*key):
    return np.random.default_rng([7, *key])


def dev(a, dtype=F32, ld=None, offset=0):
    """A host array on the GPU; ld, offset: as rows `ld` apart that begin
    `offset` elements into a buffer of NaN."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float64)).to(dtype)
    if ld is None and offset == 0:
        return t.cuda()
    rows, cols = t.shape
    ld = cols if ld is None else ld
    buf = torch.full((offset + rows * ld + 8,), float("nan"), dtype=dtype, device="cuda")
    v = buf[offset:].as_strided((rows, cols), (ld, 1))
    v.copy_(t)
    return v


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, want, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    want, tol = np.broadcast_to(want, got.shape), np.broadcast_to(tol, got.shape)
    assert got.shape == want.shape
    assert not np.isnan(got).any(), what
    bad = np.abs(got - want) > tol + 1e-37
    if bad.any():
        i = np.argmax((np.abs(got - want) / (tol + 1e-37)).ravel())
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.size} off; worst at {i}: "
                             f"{got.ravel()[i]} for {want.ravel()[i]}, tol {tol.ravel()[i]}")


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
EPS = 1e-5


def norm64(h, w, b, eps=EPS):
    mean = h.mean(1)
    var = np.square(h - mean[:, None]).mean(1)
    rstd = 1 / np.sqrt(var + eps)
    return (h - mean[:, None]) * rstd[:, None] * w + b, mean, rstd


def check_norm(got, h, w, b, y_dt):
    """y, mean and rstd of the rows h (as the kernel sees them, in 64 bits)."""
    C = h.shape[1]
    n = (C / 32 + 32) * U
    y, mean, rstd = norm64(h, w, b)
    e_mean = (n + 2 * U) * np.abs(h).mean(1)
    d = np.abs(h - mean[:, None])
    e_d = U * d + e_mean[:, None] + U * np.abs(h)          # h itself may be a rounded sum
    e_var = 2 * (d * e_d).mean(1) + np.square(e_d).mean(1) + (n + 4 * U) * np.square(d).mean(1)
    var = np.square(d).mean(1) + EPS
    r_rstd = e_var / (2 * var) * (1 + e_var / var) + 4 * U
    check(got[1], mean, e_mean, "mean")
    check(got[2], rstd, r_rstd * rstd, "rstd")
    e_y = (np.abs(w) * rstd[:, None] * (e_d + d * (r_rstd[:, None] + 4 * U))
           + 2 * U * np.abs(b) + 2 * OUT_U[y_dt] * np.abs(y))
    check(got[0], y, e_y, "y")


SHAPES = [(1, 1), (5, 1), (3, 2), (9, 7), (33, 16), (2100, 64), (40, 77), (31, 128), (17, 513),
          (700, 768), (3, 1000), (401, 1001), (9, 1024), (5, 2056), (7, 4096), (3, 4099), (2, 8192),
          (3, 14336), (2, 16384), (2, 16387), (1, 20000), (2, 40000), (1, 70001)]


@pytest.mark.parametrize("T,C", SHAPES)
@pytest.mark.parametrize("x_dt,y_dt,w_dt", [(BF16, BF16, BF16), (F32, F32, F32), (BF16, F32, F32),
                                            (F32, BF16, BF16)])
def test_layer_norm(T, C, x_dt, y_dt, w_dt):
    r = rng(T, C)
    x = dev(r.normal(size=(T, C)) * 2 + r.normal(size=C), x_dt)
    w, b = dev(1 + 0.2 * r.normal(size=C), w_dt), dev(r.normal(size=C), w_dt)
    got = hlq.hlq_layer_norm(x, w, b, eps=EPS, out_dtype=y_dt)
    assert got[0].dtype == y_dt and got[1].dtype == got[2].dtype == F32
    check_norm(got, f64(x), f64(w), f64(b), y_dt)
    res = dev(r.normal(size=(T, C)), x_dt)
    got = hlq.hlq_layer_norm(x, w, b, eps=EPS, residual=res, out_dtype=y_dt)
    h = f64(x) + f64(res)
    check(got[3], h, 2 * OUT_U[x_dt] * np.abs(h), "h")
    check_norm(got, h, f64(w), f64(b), y_dt)


def test_layer_norm_without_affine_and_statistics():
    x = dev(rng(1).normal(size=(6, 200)))
    y, mean, rstd = hlq.hlq_layer_norm(x, eps=EPS)
    check_norm((y, mean, rstd), f64(x), 1.0, 0.0, F32)
    w = dev(rng(2).normal(size=200))
    check_norm(hlq.hlq_layer_norm(x, w, eps=EPS), f64(x), f64(w), 0.0, F32)
    check_norm(hlq.hlq_layer_norm(x, None, w, eps=EPS), f64(x), 1.0, f64(w), F32)
    y2, m2, r2 = hlq.hlq_layer_norm(x, eps=EPS, with_stats=False)
    assert m2 is None and r2 is None and torch.equal(y2, y)


@pytest.mark.parametrize("C,ld,off", [(64, 80, 8), (64, 67, 0), (64, 64, 3), (77, 77, 1),
                                      (513, 520, 5), (1024, 1030, 2), (4096, 4104, 4)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_layer_norm_strides_and_offsets(C, ld, off, dt):
    T = 11
    r = rng(C, ld, off)
    x, res = dev(r.normal(size=(T, C)), dt, ld, off), dev(r.normal(size=(T, C)), dt, ld + 1, 1)
    w, b = dev(r.normal(size=C)), dev(r.normal(size=C))
    out = torch.full((T, 2 * ld), 7.0, dtype=dt, device="cuda")
    y, mean, rstd, h = hlq.hlq_layer_norm(x, w, b, residual=res, out=out[:, off:off + C])
    check_norm((y, mean, rstd), f64(x) + f64(res), f64(w), f64(b), dt)
    assert bool((out[:, :off] == 7).all()) and bool((out[:, off + C:] == 7).all())
    whole = hlq.hlq_layer_norm(x.contiguous(), w, b, residual=res.contiguous())
    assert torch.equal(h, whole[3])
    # backward, every matrix with a stride of its own
    gy, gr = dev(r.normal(size=(T, C)), F32, ld + 3, 2), dev(r.normal(size=(T, C)), dt, ld + 8, 8)
    out = torch.full((T, 2 * ld), 7.0, dtype=dt, device="cuda")
    got = hlq.hlq_layer_norm_backward(gy, h, mean, rstd, w, g_residual=gr,
                                      out=out[:, off:off + C])
    assert bool((out[:, :off] == 7).all()) and bool((out[:, off + C:] == 7).all())
    check_norm_bwd(got, gy, h, mean, rstd, w, gr)


def test_layer_norm_repeated_rows_and_in_place():
    r = rng(5)
    row, w, b = dev(r.normal(size=(1, 96))), dev(r.normal(size=96)), dev(r.normal(size=96))
    y, mean, rstd = hlq.hlq_layer_norm(row.expand(9, 96), w, b)
    one = hlq.hlq_layer_norm(row, w, b)
    assert torch.equal(y, one[0].expand(9, 96)) and torch.equal(mean, one[1].expand(9))
    g = dev(r.normal(size=(1, 96)))
    back = hlq.hlq_layer_norm_backward(g.expand(9, 96), row.expand(9, 96), mean, rstd, w)
    check_norm_bwd(back, g.expand(9, 96), row.expand(9, 96), mean, rstd, w, None)
    for C in (96, 101, 3000, 40000):
        x, res = dev(r.normal(size=(4, C))), dev(r.normal(size=(4, C)))
        want = hlq.hlq_layer_norm(x, residual=res)
        a, c = x.clone(), res.clone()
        got = hlq.hlq_layer_norm(a, residual=c, out=a, h=c)
        assert got[0] is a and got[3] is c
        for p, q in zip(got, want):
            assert torch.equal(p, q)
        gy, gr = dev(r.normal(size=(4, C))), dev(r.normal(size=(4, C)))
        args = (x, want[1], want[2])
        want_b = hlq.hlq_layer_norm_backward(gy, *args, g_residual=gr)
        for over in (0, 1):                        # over g_y, over the residual's gradient
            g2, r2 = gy.clone(), gr.clone()
            got_b = hlq.hlq_layer_norm_backward(g2, *args, g_residual=r2, out=(g2, r2)[over])
            for p, q in zip(got_b, want_b):
                assert torch.equal(p, q)


def test_layer_norm_constant_and_large_rows():
    """A row without variance gives the bias; values near 1e17 (squares that
    sum below fp32 overflow) and rows of a large offset stay right."""
    b = dev(rng(6).normal(size=300))
    y, mean, rstd = hlq.hlq_layer_norm(dev(np.full((2, 300), 3.0)), None, b, eps=EPS)
    check(y, f64(b), 1e-3 * np.ones(300), "constant rows")
    check(rstd, 1 / math.sqrt(EPS), 4 * U / math.sqrt(EPS), "rstd of a constant row")
    x = rng(7).normal(size=(3, 300)) * np.array([[1e17], [1e-3], [1.0]]) + [[0], [0], [1000.0]]
    x = dev(x)
    check_norm(hlq.hlq_layer_norm(x, eps=EPS), f64(x), 1.0, 0.0, F32)


def check_norm_bwd(got, gy, x, mean, rstd, w, gres):
    gx_dt = got[0].dtype
    g, x64, mu, rs = f64(gy), f64(x), f64(mean)[:, None], f64(rstd)[:, None]
    w64 = np.ones(g.shape[1]) if w is None else f64(w)
    T, C = g.shape
    n = (C / 32 + 32) * U
    xhat, a = (x64 - mu) * rs, g * w64
    e_x = 2 * U * np.abs(xhat) + U * rs * (np.abs(x64) + np.abs(mu))
    sa, sx = a.mean(1, keepdims=True), (a * xhat).mean(1, keepdims=True)
    e_sa = (n + 3 * U) * np.abs(a).mean(1, keepdims=True)
    e_sx = ((n + 4 * U) * np.abs(a * xhat) + np.abs(a) * e_x).mean(1, keepdims=True)
    want = rs * (a - sa - xhat * sx)
    tol = rs * (5 * U * (np.abs(a) + np.abs(sa) + np.abs(xhat * sx)) + e_sa + np.abs(xhat) * e_sx
                + e_x * (np.abs(sx) + e_sx))
    if gres is not None:
        want = want + f64(gres)
    check(got[0], want, tol + 2 * OUT_U[gx_dt] * np.abs(want), "g_x")
    if got[1] is not None:
        nt = (T + 8) * U
        check(got[1], (g * xhat).sum(0),
              nt * np.abs(g * xhat).sum(0) + (np.abs(g) * e_x).sum(0), "g_weight")
        check(got[2], g.sum(0), nt * np.abs(g).sum(0), "g_bias")


@pytest.mark.parametrize("T,C", SHAPES)
@pytest.mark.parametrize("x_dt,gy_dt,gx_dt,w_dt", [(BF16, F32, BF16, BF16), (F32, F32, F32, F32),
                                                   (BF16, BF16, BF16, F32), (F32, BF16, F32, BF16),
                                                   (BF16, BF16, F32, F32), (F32, F32, BF16, F32),
                                                   (BF16, F32, F32, F32), (F32, BF16, BF16, F32)])
def test_layer_norm_backward(T, C, x_dt, gy_dt, gx_dt, w_dt):
    r = rng(T, C, 1)
    x = dev(r.normal(size=(T, C)) * 2 + r.normal(size=C), x_dt)
    w = dev(1 + 0.2 * r.normal(size=C), w_dt)
    _, mean, rstd = norm64(f64(x), 1.0, 0.0)
    mean, rstd = dev(mean), dev(rstd)
    gy = dev(r.normal(size=(T, C)), gy_dt)
    got = hlq.hlq_layer_norm_backward(gy, x, mean, rstd, w, out_dtype=gx_dt)
    assert got[0].dtype == gx_dt and got[1].dtype == got[2].dtype == F32
    check_norm_bwd(got, gy, x, mean, rstd, w, None)
    gr = dev(r.normal(size=(T, C)), gx_dt)
    with_r = hlq.hlq_layer_norm_backward(gy, x, mean, rstd, w, g_residual=gr, out_dtype=gx_dt)
    check_norm_bwd(with_r, gy, x, mean, rstd, w, gr)
    # frozen weights, and a norm without weights
    only = hlq.hlq_layer_norm_backward(gy, x, mean, rstd, w, out_dtype=gx_dt,
                                       with_weight_grads=False)
    assert torch.equal(only[0], got[0]) and only[1] is None and only[2] is None
    bare = hlq.hlq_layer_norm_backward(gy, x, mean, rstd, None, out_dtype=gx_dt)
    check_norm_bwd(bare, gy, x, mean, rstd, None, None)


def test_layer_norm_gradient_against_differences():
    """Directional differences of sum(y g) in 64 bits, in x, weight and bias.
    The forward pass is smooth: a central difference with h = 1e-5 is within
    1e-8 of the directional derivative here; the kernel adds fp32 rounding."""
    T, C = 12, 91
    r = rng(9)
    x, w, b, g = (r.normal(size=s) for s in ((T, C), C, C, (T, C)))
    x, w, b, g = (f64(dev(v)) for v in (x, w, b, g))
    y, mean, rstd = hlq.hlq_layer_norm(dev(x), dev(w), dev(b))
    gx, gw, gb = (f64(t) for t in hlq.hlq_layer_norm_backward(dev(g), dev(x), mean, rstd, dev(w)))
    f = lambda x, w, b: (norm64(x, w, b)[0] * g).sum()  # noqa: E731
    for k in range(5):
        dx, dw, db = (r.normal(size=s) for s in ((T, C), C, C))
        h = 1e-5
        diff = (f(x + h * dx, w + h * dw, b + h * db) - f(x - h * dx, w - h * dw, b - h * db)) / (2 * h)
        along = (gx * dx).sum() + (gw * dw).sum() + (gb * db).sum()
        size = (np.abs(gx * dx)).sum() + np.abs(gw * dw).sum() + np.abs(gb * db).sum()
        assert abs(diff - along) <= 1e-6 * size


def test_layer_norm_empty_batch():
    x = torch.empty((0, 32), device="cuda")
    y, mean, rstd = hlq.hlq_layer_norm(x)
    assert y.shape == (0, 32) and mean.shape == (0,)
    gx, gw, gb = hlq.hlq_layer_norm_backward(x, x, mean, rstd)
    assert gx.shape == (0, 32) and not gw.any() and not gb.any()


@pytest.mark.parametrize("C", [64, 1001, 20000])
def test_layer_norm_flags_nonfinite_rows(C):
    x = torch.randn(4, C, device="cuda")
    x[2, C // 2] = float("inf")
    y, mean, rstd = hlq.hlq_layer_norm(x)
    assert hlq.hlq_read_device_status(clear=True) == hlq.DEV_NONFINITE
    assert bool(torch.isfinite(y[[0, 1, 3]]).all())
    gy = torch.randn(4, C, device="cuda")
    gy[1, 3] = float("nan")
    x[2] = 1.0
    gx, _, gb = hlq.hlq_layer_norm_backward(gy, x, torch.zeros(4, device="cuda"),
                                            torch.ones(4, device="cuda"))
    assert hlq.hlq_read_device_status(clear=True) == hlq.DEV_NONFINITE
    assert bool(torch.isfinite(gx[[0, 2, 3]]).all()) and bool(torch.isnan(gb[3]))


# ---------------------------------------------------------------------------
# log-probabilities and the policy loss
# ---------------------------------------------------------------------------
def logits_case(T, V, dt, r, ld=None, off=0):
    z = r.normal(size=(T, V)) * 3
    a = r.integers(0, V, T)
    z[np.arange(T), a] += 5
    return dev(z, dt, ld, off), a


def logsoftmax64(z):
    top = z.max(1, keepdims=True)
    with np.errstate(divide="ignore"):
        return z - top - np.log(np.exp(z - top).sum(1, keepdims=True))


def e_logp(z, lp, V):
    """Error of a log-probability: rounding of z - max and of the result, and
    the relative error of the sum of exps (the argument's rounding, 4 ulp, the
    sum), with the products by scale and log2(e)."""
    span = np.minimum(np.abs(z).max() * 2, 60.0)
    return 4 * U * (np.abs(lp) + span + 8) + (V / 32 + 32) * U


ROWS = [(1, 1), (3, 2), (1, 7), (5, 33), (64, 100), (2, 513), (7, 1000), (333, 1001), (2, 4096),
        (6, 8191), (1, 32000), (3, 50021), (2, 65537), (1, 128256), (4, 128256), (1, 151671),
        (2, 300007)]


@pytest.mark.parametrize("T,V", ROWS)
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_token_logprobs(T, V, dt, scale):
    z, a = logits_case(T, V, dt, rng(T, V))
    logp, lse = hlq.hlq_token_logprobs(z, torch.from_numpy(a).cuda(), scale=scale)
    z64 = f64(z) * scale
    ls = logsoftmax64(z64)
    want = ls[np.arange(T), a]
    check(logp, want, e_logp(z64, want, V), "logp")
    want_lse = z64[:, 0] - ls[:, 0]
    check(lse, want_lse, e_logp(z64, want_lse, V), "lse")


@pytest.mark.parametrize("V,ld,off", [(100, 104, 0), (1001, 1003, 1), (4096, 4100, 3),
                                      (50021, 50021, 5), (65537, 65600, 7), (131072, 131080, 8)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_token_logprobs_strides(V, ld, off, dt):
    T = 3
    z, a = logits_case(T, V, dt, rng(V, ld), ld, off)
    a = torch.from_numpy(a).cuda()
    got = hlq.hlq_token_logprobs(z, a)
    z64 = f64(z)
    want = logsoftmax64(z64)[np.arange(T), f64(a).astype(int)]
    check(got[0], want, e_logp(z64, want, V), "logp")


def test_token_logprobs_masked_vocabulary_and_bad_tokens():
    z = torch.randn(5, 300, device="cuda")
    z[0, 10:] = -float("inf")            # few tokens allowed
    z[1, :] = -float("inf")
    z[1, 7] = 2.0                        # one token allowed
    a = torch.tensor([3, 7, 299, 0, 5], device="cuda")
    logp, lse = hlq.hlq_token_logprobs(z, a)
    want = logsoftmax64(f64(z))[np.arange(5), f64(a).astype(int)]
    assert float(logp[1]) == 0.0
    check(logp, want, 1e-5, "logp")
    logp, _ = hlq.hlq_token_logprobs(z, torch.tensor([20, 7, 1, 1, 1], device="cuda"))
    assert float(logp[0]) == -float("inf")        # a token of probability 0
    assert hlq.hlq_read_device_status(clear=True) == 0
    for bad in (-1, -100, 300, 1 << 40):
        logp, lse = hlq.hlq_token_logprobs(z, torch.tensor([3, bad, 1, 1, 1], device="cuda"))
        assert bool(torch.isnan(logp[1])) and bool(torch.isfinite(lse).all())
        assert bool(torch.isfinite(logp[[0, 2, 3, 4]]).all())
        assert hlq.hlq_read_device_status(clear=True) == hlq.DEV_BADCODE
    z[2] = -float("inf")                          # no token allowed: no distribution
    logp, _ = hlq.hlq_token_logprobs(z, a)
    assert bool(torch.isnan(logp[2]))
    assert hlq.hlq_read_device_status(clear=True) == hlq.DEV_NONFINITE
    z[2] = 0.0
    z[3, 299] = float("nan")
    logp, _ = hlq.hlq_token_logprobs(z, a)
    assert bool(torch.isnan(logp[3])) and bool(torch.isfinite(logp[[0, 1, 2, 4]]).all())
    assert hlq.hlq_read_device_status(clear=True) == hlq.DEV_NONFINITE


def policy64(z, a, old, ref, adv, w, scale, lo, hi, beta):
    """Loss terms and d loss / d logits, from the definition."""
    T = len(a)
    ls = logsoftmax64(z * scale)
    lp = ls[np.arange(T), a]
    r = np.exp(lp - old)
    inner, outer = r * adv, np.clip(r, 1 - lo, 1 + hi) * adv
    clipped = outer < inner
    pg = -np.minimum(inner, outer)
    c = np.where(clipped, 0.0, -inner)
    kl = np.zeros(T)
    if ref is not None:
        d = ref - lp
        kl = np.expm1(d) - d
        c = c - beta * np.expm1(d)
    g = -np.exp(ls)
    g[np.arange(T), a] = -np.expm1(lp)
    stats = [(w * (pg + beta * kl)).sum(), (w * pg).sum(), (w * kl).sum(), w[clipped].sum()]
    return np.array(stats), lp, g * (w * c * scale)[:, None], c


def policy_inputs(T, V, dt, r, scale, lo, hi, ld=None, off=0):
    z, a = logits_case(T, V, dt, r, ld, off)
    lp = logsoftmax64(f64(z) * scale)[np.arange(T), a]
    ratio = np.exp(0.3 * r.normal(size=T))
    for edge in (1 - lo, 1 + hi):                # a ratio at the edge itself may fall either way
        ratio = np.where(np.abs(ratio - edge) < 1e-2, edge + 2e-2, ratio)
    old, ref, adv = lp - np.log(ratio), lp + 0.5 * r.normal(size=T), r.normal(size=T)
    w = (r.random(T) < 0.75) / T
    return (z, torch.from_numpy(a).cuda()) + tuple(dev(v) for v in (old, adv, w, ref))


def check_policy(got, z, a, old, adv, w, ref, scale, lo, hi, beta, grad_scale):
    T, V = z.shape
    z64, a, w = np.nan_to_num(f64(z)), f64(a).astype(int), f64(w)
    on = w != 0
    n = lambda t: None if t is None else f64(t)  # noqa: E731
    stats, lp, g, c = policy64(z64, a, n(old), n(ref), n(adv), w, scale, lo, hi, beta)
    e_lp = np.where(on, e_logp(z64 * scale, lp, V), 0.0)
    check(got[1], np.where(on, lp, 0.0), e_lp, "logp")
    # r, exp(d) and all that follows carry the error of lp (and exp's own)
    e_r = e_lp + 8 * U
    r = np.exp(lp - n(old))
    ed = np.exp(n(ref) - lp) if ref is not None else np.zeros(T)
    e_pg = (1 + lo + hi + r) * np.abs(n(adv)) * (e_r + 4 * U)
    e_kl = (ed + 1) * e_r + 4 * U * (ed + np.abs(np.log(np.maximum(ed, 1e-30))))
    s = [w * (e_pg + abs(beta) * e_kl), w * e_pg, w * e_kl, w * 0]
    tol = np.array([v.sum() for v in s]) + 4 * U * (np.abs(stats) + 1)
    check(got[0], stats, tol, "stats")
    if got[2] is None:
        return
    g = g * grad_scale
    e_c = r * np.abs(n(adv)) * (e_r + 4 * U) + abs(beta) * (ed * e_r + 4 * U * (ed + 1))
    p = np.exp(logsoftmax64(z64 * scale))
    hot = np.zeros_like(p)
    hot[np.arange(T), a] = 1
    size = np.abs(hot - p)
    tol = (abs(grad_scale) * scale * w * (e_c + np.abs(c) * 8 * U))[:, None] * size
    tol = tol + np.abs(grad_scale * scale * w * c)[:, None] * (p * (e_lp + 8 * U)[:, None])
    check(got[2], g, tol + 2 * OUT_U[got[2].dtype] * np.abs(g), "g")
    assert not got[2][torch.from_numpy(~on).cuda()].any()


@pytest.mark.parametrize("T,V", ROWS)
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("ref,scale,lo,hi,beta,gs", [(True, 1.0, 0.2, 0.28, 0.05, 1.0),
                                                     (False, 0.7, 0.1, 0.1, 0.0, 512.0)])
def test_policy_loss(T, V, dt, ref, scale, lo, hi, beta, gs):
    z, a, old, adv, w, rf = policy_inputs(T, V, dt, rng(T, V, 3), scale, lo, hi)
    rf = rf if ref else None
    kw = dict(ref_logp=rf, clip_low=lo, clip_high=hi, kl_coef=beta, scale=scale, grad_scale=gs)
    got = hlq.hlq_policy_loss(z, a, old, adv, w, **kw)
    assert got[2].dtype == dt
    check_policy(got, z, a, old, adv, w, rf, scale, lo, hi, beta, gs)
    # the loss alone: the same bits
    alone = hlq.hlq_policy_loss(z, a, old, adv, w, with_grad=False, **kw)
    assert alone[2] is None and torch.equal(alone[0], got[0]) and torch.equal(alone[1], got[1])
    # over the logits
    over = z.clone()
    got2 = hlq.hlq_policy_loss(over, a, old, adv, w, out=over, **kw)
    assert got2[2] is over
    for p, q in zip(got2, got):
        assert torch.equal(p, q)


@pytest.mark.parametrize("V,ld,off,ldg,offg", [(100, 104, 0, 100, 0), (1001, 1003, 1, 1001, 1),
                                               (4096, 4100, 3, 4096, 0), (50021, 50021, 5, 50024, 8),
                                               (65537, 65600, 7, 65537, 2),
                                               (131072, 131080, 8, 131072, 0)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_policy_loss_strides(V, ld, off, ldg, offg, dt):
    T = 5
    z, a, old, adv, w, ref = policy_inputs(T, V, dt, rng(V, ldg), 1.0, 0.2, 0.2, ld, off)
    buf = torch.full((offg + T * ldg + 8,), 7.0, dtype=dt, device="cuda")
    out = buf[offg:].as_strided((T, V), (ldg, 1))
    got = hlq.hlq_policy_loss(z, a, old, adv, w, ref_logp=ref, kl_coef=0.1, out=out)
    check_policy(got, z, a, old, adv, w, ref, 1.0, 0.2, 0.2, 0.1, 1.0)
    touched = torch.zeros_like(buf, dtype=torch.bool)
    touched[offg:].as_strided((T, V), (ldg, 1)).fill_(True)
    assert bool((buf[~touched] == 7).all())


@pytest.mark.parametrize("V", [50, 33000])
def test_policy_loss_masked_rows_are_not_read(V):
    T = 6
    z, a, old, adv, w, ref = policy_inputs(T, V, F32, rng(11, V), 1.0, 0.2, 0.2)
    w[:] = 0.25
    w[1] = w[4] = 0
    want = hlq.hlq_policy_loss(z, a, old, adv, w, ref_logp=ref, kl_coef=0.1)
    for t in (z, old, adv, ref):
        t[1] = float("nan")
        t[4] = -float("inf")
    a[1], a[4] = -100, V
    got = hlq.hlq_policy_loss(z, a, old, adv, w, ref_logp=ref, kl_coef=0.1)
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    assert not got[2][[1, 4]].any() and not got[1][[1, 4]].any()
    # nothing left at all
    got = hlq.hlq_policy_loss(z, a, old, adv, torch.zeros_like(w), ref_logp=ref, kl_coef=0.1)
    assert not got[0].any() and not got[1].any() and not got[2].any()


def test_policy_loss_masked_vocabulary_and_bad_tokens():
    T, V = 4, 500
    z, a, old, adv, w, ref = policy_inputs(T, V, F32, rng(12), 1.0, 0.2, 0.2)
    w[:] = 0.25
    a[:] = torch.arange(T, device="cuda")
    z[0, 30:] = -float("inf")
    lp, _ = hlq.hlq_token_logprobs(z, a)
    got = hlq.hlq_policy_loss(z, a, lp, adv, w, ref_logp=lp, kl_coef=0.1)
    assert torch.equal(got[1], lp) and not got[2][0, 30:].any()
    assert bool(torch.isfinite(got[2]).all()) and float(got[0][3]) == 0.0
    assert abs(float(got[0][2])) <= 1e-6
    assert hlq.hlq_read_device_status(clear=True) == 0
    a[2] = V
    got = hlq.hlq_policy_loss(z, a, lp, adv, w, ref_logp=lp, kl_coef=0.1)
    assert bool(torch.isnan(got[1][2])) and bool(torch.isfinite(got[2][[0, 1, 3]]).all())
    assert hlq.hlq_read_device_status(clear=True) == hlq.DEV_BADCODE | hlq.DEV_NONFINITE


def test_policy_gradient_against_differences():
    """Central differences of the loss in 64 bits along random directions."""
    T, V = 9, 37
    r = rng(13)
    z, a, old, adv, w, ref = policy_inputs(T, V, F32, r, 0.8, 0.2, 0.3)
    w[:] = 1.0 / T
    _, _, g = hlq.hlq_policy_loss(z, a, old, adv, w, ref_logp=ref, kl_coef=0.3, scale=0.8,
                                  clip_low=0.2, clip_high=0.3)
    g, z64, ai = f64(g), f64(z), f64(a).astype(int)
    f = lambda x: policy64(x, ai, f64(old), f64(ref), f64(adv), f64(w), 0.8, 0.2, 0.3, 0.3)[0][0]  # noqa: E731
    for k in range(5):
        d = r.normal(size=z64.shape)
        h = 1e-5
        diff = (f(z64 + h * d) - f(z64 - h * d)) / (2 * h)
        assert abs(diff - (g * d).sum()) <= 2e-6 * np.abs(g * d).sum()


def test_policy_loss_empty_batch():
    z = torch.empty((0, 10), device="cuda")
    e = torch.empty(0, device="cuda")
    stats, logp, g = hlq.hlq_policy_loss(z, torch.empty(0, dtype=torch.int64, device="cuda"), e, e,
                                         e)
    assert not stats.any() and logp.shape == (0,) and g.shape == (0, 10)
    logp, lse = hlq.hlq_token_logprobs(z, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert logp.shape == (0,)


# ---------------------------------------------------------------------------
# gradient norm and clipping
# ---------------------------------------------------------------------------
def clip64(gs, max_norm):
    norm = math.sqrt(math.fsum(float(np.square(g).sum()) for g in gs))
    return norm, min(1.0, max_norm / (norm + 1e-6))


def check_clip(grads64, outs, norm_coef, max_norm):
    """Squares in fp32 (or wider), summed over at most 2^16 elements a thread."""
    norm, coef = clip64(grads64, max_norm)
    n = max((g.size for g in grads64), default=0)
    rel = min(n / 256 + 64, 4096) * U
    got = f64(norm_coef)
    check(got[:1], norm, rel * norm, "norm")
    check(got[1:], coef, (rel + 4 * U) * coef, "coef")
    for g, o in zip(grads64, outs or []):
        want = g * coef
        check(o, want.reshape(tuple(o.shape)),
              ((rel + 6 * U + 2 * OUT_U[o.dtype]) * np.abs(want)).reshape(tuple(o.shape)), "out")


SIZES = [[(1,)], [(5,), (3, 7)], [(64, 128), (128,), (0,), (64,)], [(8192,), (8193,), (1,), (16384,)],
         [(257, 129), (4, 5, 6), (100003,)], [(1,)] * 600, [(17 + i,) for i in range(1100)],
         [(1 << 21,), (3,)]]


@pytest.mark.parametrize("k", range(len(SIZES)))
@pytest.mark.parametrize("g_dt,o_dt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_clip_grad_norm(k, g_dt, o_dt, max_norm):
    r = rng(k)
    grads = [dev(r.normal(size=s), g_dt) for s in SIZES[k]]
    g64 = [f64(g) for g in grads]
    outs = [torch.empty(g.shape, dtype=o_dt, device="cuda") for g in grads]
    nc = hlq.hlq_clip_grad_norm(grads, max_norm, outs=outs)
    check_clip(g64, outs, nc, max_norm)
    only = hlq.hlq_clip_grad_norm(grads, max_norm, norm_only=True)
    assert torch.equal(only, nc)
    for g, v in zip(grads, g64):
        assert np.array_equal(f64(g), v)
    nc = hlq.hlq_clip_grad_norm(grads, max_norm)          # in place
    check_clip(g64, grads, nc, max_norm)
    if max_norm > 1e8:
        for g, v in zip(grads, g64):
            assert np.array_equal(f64(g), v)


def test_clip_grad_norm_views_and_mixed_types():
    """Gradients and outputs at any element offset of flat buffers."""
    r = rng(21)
    sizes = [5, 4096, 3, 8191, 1, 30011, 8, 640]
    flat_in = dev(r.normal(size=sum(sizes)))
    flat_out = torch.full((sum(sizes) + 1,), 7.0, dtype=BF16, device="cuda")
    grads, outs, g64, at = [], [], [], 0
    for n in sizes:
        grads.append(flat_in[at:at + n])
        outs.append(flat_out[at + 1:at + 1 + n])
        at += n
    grads[3] = grads[3].to(BF16)
    grads[5] = dev(r.normal(size=30012), BF16)[1:]
    outs[2], outs[6] = torch.empty(3, device="cuda"), torch.empty(9, device="cuda")[1:]
    g64 = [f64(g) for g in grads]
    nc = hlq.hlq_clip_grad_norm(grads, 1.0, outs=outs)
    check_clip(g64, outs, nc, 1.0)
    assert float(flat_out[0]) == 7.0


@pytest.mark.parametrize("scale", [1e-30, 3e-20, 1e15, 1e19, 3e30])
def test_clip_grad_norm_range(scale):
    """Squares beyond fp32's range, above and below."""
    r = rng(22)
    grads = [dev(r.normal(size=n) * scale) for n in (7, 5000, 20000)]
    nc = hlq.hlq_clip_grad_norm(grads, scale, norm_only=True)
    norm, _ = clip64([f64(g) for g in grads], scale)
    check(f64(nc)[:1], norm, 512 * U * norm, "norm")


def test_clip_grad_norm_zero_nonfinite_and_empty():
    z = [torch.zeros(1000, device="cuda"), torch.zeros(3, device="cuda")]
    nc = hlq.hlq_clip_grad_norm(z, 1.0)
    assert nc.tolist() == [0.0, 1.0] and not z[0].any()
    assert hlq.hlq_clip_grad_norm([], 1.0).tolist() == [0.0, 1.0]
    assert hlq.hlq_clip_grad_norm([torch.empty(0, device="cuda")], 1.0).tolist() == [0.0, 1.0]
    g = torch.ones(300, device="cuda")
    assert hlq.hlq_clip_grad_norm([g], 0.0)[1].item() == 0.0 and not g.any()
    g = torch.ones(300, device="cuda")
    assert hlq.hlq_clip_grad_norm([g], float("inf"))[1].item() == 1.0 and bool((g == 1).all())
    assert hlq.hlq_read_device_status(clear=True) == 0
    g[7] = float("inf")
    nc = hlq.hlq_clip_grad_norm([g], 1.0)
    assert nc.tolist() == [float("inf"), 0.0]
    assert bool(torch.isnan(g[7])) and not g[:7].any() and not g[8:].any()
    assert hlq.hlq_read_device_status(clear=True) == hlq.DEV_NONFINITE
    g = torch.ones(300, device="cuda")
    g[299] = float("nan")
    nc = hlq.hlq_clip_grad_norm([g], 1.0)
    assert bool(torch.isnan(nc).all()) and bool(torch.isnan(g).all())
    assert hlq.hlq_read_device_status(clear=True) == hlq.DEV_NONFINITE


# ---------------------------------------------------------------------------
# streams, repetition, capture
# ---------------------------------------------------------------------------
def _calls():
    r = rng(31)
    x, res = dev(r.normal(size=(600, 768)), BF16), dev(r.normal(size=(600, 768)), BF16)
    w, b = dev(r.normal(size=768)), dev(r.normal(size=768))
    gy = dev(r.normal(size=(600, 768)))
    mean, rstd = hlq.hlq_layer_norm(x)[1:]
    z, a, old, adv, wt, ref = policy_inputs(40, 9001, BF16, r, 1.0, 0.2, 0.2)
    grads = [dev(r.normal(size=n)) for n in (100, 70000, 8192)]
    outs = [torch.empty_like(g) for g in grads]
    return [lambda **k: hlq.hlq_layer_norm(x, w, b, residual=res, **k),
            lambda **k: hlq.hlq_layer_norm_backward(gy, x, mean, rstd, w, **k),
            lambda **k: hlq.hlq_token_logprobs(z, a, **k),
            lambda **k: hlq.hlq_policy_loss(z, a, old, adv, wt, ref_logp=ref, kl_coef=0.1, **k),
            lambda **k: (hlq.hlq_clip_grad_norm(grads, 1.0, outs=outs, **k), *outs)]


def test_equal_calls_give_equal_bits_on_any_stream():
    calls = _calls()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for f in calls:
        first = [t.clone() for t in f()]
        for p, q in zip(f(), first):
            assert torch.equal(p, q)
        torch.cuda.synchronize()
        got = f(stream=other)
        other.synchronize()
        for p, q in zip(got, first):
            assert torch.equal(p, q)


def test_calls_replay_in_a_graph():
    calls = _calls()
    first = [[t.clone() for t in f()] for f in calls]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [f() for f in calls]
    for k in range(2):
        for ts in got:
            for t in ts:
                t.fill_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        for ps, qs in zip(got, first):
            for p, q in zip(ps, qs):
                assert torch.equal(p, q)


def test_rows_past_32_bit_offsets():
    """Elements past 2^31: the last rows of a matrix of 2.2e9 elements."""
    C, T = 4096, (1 << 19) + 5
    x = torch.zeros((T, C), dtype=BF16, device="cuda")
    x[-3:] = torch.randn(3, C, device="cuda").to(BF16)
    y, mean, rstd = hlq.hlq_layer_norm(x, eps=EPS)
    check_norm((y[-3:], mean[-3:], rstd[-3:]), f64(x[-3:]), 1.0, 0.0, BF16)
    gx, _, gb = hlq.hlq_layer_norm_backward(y, x, mean, rstd)
    check_norm_bwd((gx[-3:], None, None), y[-3:], x[-3:], mean[-3:], rstd[-3:], None, None)
    z = x.view(-1)[:(T * C) // 65600 * 65600].view(-1, 65600)
    a = torch.zeros(z.shape[0], dtype=torch.int64, device="cuda")
    logp, _ = hlq.hlq_token_logprobs(z, a)
    z64 = f64(z[-1:])
    want = logsoftmax64(z64)[:, 0]
    check(logp[-1:], want, e_logp(z64, want, 65600), "logp")
    nc = hlq.hlq_clip_grad_norm([x], 1.0, norm_only=True)
    norm, _ = clip64([f64(x[-3:])], 1.0)
    check(f64(nc)[:1], norm, 512 * U * norm, "norm")


@pytest.mark.parametrize("T,C", [(2500, 768), (5000, 2048), (2000, 4096), (700, 8192), (500, 14336),
                                 (4000, 24), (3000, 77), (2500, 1001), (900, 5663)])
@pytest.mark.parametrize("x_dt,gy_dt", [(BF16, F32), (F32, BF16)])
def test_layer_norm_backward_many_rows_a_cta(T, C, x_dt, gy_dt):
    """More rows than fit a CTA's stages, several calls on their way at once:
    every stage is filled and read many times over."""
    r = rng(T, C, 5)
    x, gr = dev(r.normal(size=(T, C)), x_dt), dev(r.normal(size=(T, C)), x_dt)
    w, gy = dev(1 + 0.2 * r.normal(size=C)), dev(r.normal(size=(T, C)), gy_dt)
    torch.cuda.synchronize()
    for _ in range(3):
        y, mean, rstd = hlq.hlq_layer_norm(x, w)
        got = [hlq.hlq_layer_norm_backward(gy, x, mean, rstd, w, g_residual=gr) for _ in range(3)]
    check_norm((y, mean, rstd), f64(x), f64(w), 0.0, x_dt)
    check_norm_bwd(got[0], gy, x, mean, rstd, w, gr)
    for other in got[1:]:
        for p, q in zip(other, got[0]):
            assert torch.equal(p, q)


@pytest.mark.parametrize("T,V,dt", [(700, 3000, BF16), (700, 40000, BF16), (500, 70001, F32)])
def test_logprobs_do_not_depend_on_the_number_of_rows(T, V, dt):
    """The same bits for a row alone, in a few rows, in many, and from the
    policy loss: the ratio of an unchanged policy is exactly 1.  (Rows of one
    tensor begin at different offsets from 16 bytes, so a row alone is compared
    where it lies.)"""
    z, a = logits_case(T, V, dt, rng(T, V, 6))
    a = torch.from_numpy(a).cuda()
    many, lse = hlq.hlq_token_logprobs(z, a)
    for lo, hi in ((0, 1), (3, 4), (T - 5, T), (100, 300)):
        few = hlq.hlq_token_logprobs(z[lo:hi], a[lo:hi])
        assert torch.equal(few[0], many[lo:hi]) and torch.equal(few[1], lse[lo:hi])
    ones = torch.ones(T, device="cuda")
    stats, logp, _ = hlq.hlq_policy_loss(z, a, many, ones, ones / T, ref_logp=many, kl_coef=0.1)
    assert torch.equal(logp, many)
    assert float(stats[2]) == 0.0 and float(stats[3]) == 0.0
    assert abs(float(stats[0]) + 1.0) <= 1e-5


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("C", [8, 264, 768, 1024, 2048, 9000])
def test_layer_norm_backward_few_rows(T, C):
    """Where the column sums are joined by one cluster, and just beyond."""
    if C > 1024 and T > 17:
        T -= 100 if T > 100 else 0
    r = rng(T, C, 8)
    x, gy, w = dev(r.normal(size=(T, C)), BF16), dev(r.normal(size=(T, C))), dev(r.normal(size=C))
    _, mean, rstd = hlq.hlq_layer_norm(x)
    got = hlq.hlq_layer_norm_backward(gy, x, mean, rstd, w)
    check_norm_bwd(got, gy, x, mean, rstd, w, None)


def test_outputs_given_or_made_are_the_same_bits():
    """A call that makes its outputs (in one step of the extension) and one that
    is given them (through Python)."""
    r = rng(41)
    x, w, b = dev(r.normal(size=(50, 264)), BF16), dev(r.normal(size=264)), dev(r.normal(size=264))
    made = hlq.hlq_layer_norm(x, w, b)
    given = hlq.hlq_layer_norm(x, w, b, out=torch.empty_like(x))
    gy = dev(r.normal(size=(50, 264)))
    made += hlq.hlq_layer_norm_backward(gy, x, *made[1:3], w)
    given += hlq.hlq_layer_norm_backward(gy, x, *given[1:3], w, out=torch.empty_like(x))
    z, a, old, adv, wt, ref = policy_inputs(9, 700, BF16, r, 1.0, 0.2, 0.2)
    made += hlq.hlq_token_logprobs(z, a)
    given += hlq.hlq_token_logprobs(z, a, logp=torch.empty(9, device="cuda"))
    made += hlq.hlq_policy_loss(z, a, old, adv, wt, ref_logp=ref, kl_coef=0.1)
    given += hlq.hlq_policy_loss(z, a, old, adv, wt, ref_logp=ref, kl_coef=0.1,
                                 out=torch.empty_like(z))
    g = [dev(r.normal(size=n)) for n in (5, 9000)]
    made += (hlq.hlq_clip_grad_norm(g, 1.0, norm_only=True),)
    given += (hlq.hlq_clip_grad_norm(g, 1.0, norm_only=True,
                                     norm_coef=torch.empty(2, device="cuda")),)
    assert len(made) == len(given) == 12
    for p, q in zip(made, given):
        assert torch.equal(p, q)


@pytest.mark.parametrize("o_off", [0, 1, 2, 3])
@pytest.mark.parametrize("g_off", [0, 1, 2, 3])
@pytest.mark.parametrize("g_dt,o_dt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
def test_clip_grad_norm_offsets(g_off, o_off, g_dt, o_dt):
    """Every pair of offsets from a group of four, lengths around the ends of
    groups, warps' runs and chunks; nothing beside the outputs is written."""
    r = rng(51, g_off, o_off)
    grads, outs, bufs = [], [], []
    for n in (1, 2, 3, 4, 5, 127, 128, 131, 1023, 8191, 8192, 8195, 20000):
        grads.append(dev(r.normal(size=n + g_off), g_dt)[g_off:])
        bufs.append(torch.full((n + o_off + 4,), 7.0, dtype=o_dt, device="cuda"))
        outs.append(bufs[-1][o_off:o_off + n])
    g64 = [f64(g) for g in grads]
    check_clip(g64, outs, hlq.hlq_clip_grad_norm(grads, 1.0, outs=outs), 1.0)
    for b, o in zip(bufs, outs):
        assert bool((b[:o_off] == 7).all()) and bool((b[o_off + o.numel():] == 7).all())
    check_clip(g64, grads, hlq.hlq_clip_grad_norm(grads, 1.0), 1.0)
