"""Attention's backward pass in bf16 with an fp32 g_out: p and ds enter the products as two bf16 numbers,
lse and delta as three.  Cases whose g_out is exact in bf16 and whose gradients are fp32, so that only these
roundings and those of fp32 are left; how far they may put a result off; and the same arithmetic in 64 bits
with as many numbers as it is told, to see that one fewer does not pass.

The bounds, in units of d = 2^-24.  A tensor core adds 16 products to a sum at a time and may cut each of the
17 addends off (2 d of the largest, hence at most of the sum of magnitudes): 34 d for 16 terms, 2.2 d a term.
  a score, in units of log: 2.2 D size (its products), 2 for the factor scale log2(e), 1 for its product, and 8 for
      its sum with lse's three numbers; lse: 2 roundings to units of log 2, 2 for 1 / (scale log2(e)) and its
      product, 1 for what the third number leaves, 8 for the sum, 1 for the product: 14; the power of two: 4
  ds / p: 2.2 D of |g| |v|; delta: the sum of D products, 12 (8 in a lane, 4 shuffles), and 1 + 8 as lse
  p and ds: 2^-16 for two numbers (half a step of 2^-8 each), and one product
  the sums: 2.2 d a term, for each of the two numbers."""
import math

import torch

from tests import attention_ref as ref

D24 = 2.0 ** -24


class Inputs:
    """q, k, v, g, out, lse on `device`; values of q, k, v, g and out are exact in bf16."""

    def __init__(self, lens_q, lens_k, Hq, Hk, D, causal, kind="plain", seed=0, device="cpu"):
        gen = torch.Generator().manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        Tq, Tk = sum(lens_q), sum(lens_k)
        q, k, v, g = 0.15 * randn(Tq, Hq, D), randn(Tk, Hk, D), randn(Tk, Hk, D), randn(Tq, Hq, D)
        if kind == "lse":              # hardly any score: lse is the logarithm of the number of keys
            q = 0.1 * q
        elif kind == "delta":            # g . v and g . out are large and nearly alike
            v, g = 1 + 0.1 * v, 0.5 + g.abs()
        elif kind == "large scores":   # about 100 each, but for 1 or so
            c = torch.zeros(D)
            c[:2] = 4.0
            q = 0.05 * randn(Tq, Hq, D)
            q[..., :2] = 12.5 * math.sqrt(D) * (1 + 0.1 * torch.rand(Tq, Hq, 1, generator=gen))
            k = c + 0.02 * k
        self.q, self.k, self.v, g = (x.bfloat16().to(device) for x in (q, k, v, g))
        self.g = g.float()
        self.where = (lens_q, lens_k, 0, 0, causal, D ** -0.5)
        self.causal = causal
        out, lse, _, _ = ref.forward(self.q, self.k, self.v, *self.where, 0.0)
        self.out, self.lse = out.bfloat16(), lse.float()

    def offsets(self):
        return tuple(torch.tensor([0] + [sum(n[:i + 1]) for i in range(len(n))], dtype=torch.int32, device=self.q.device)
                     for n in self.where[:2])


def numbers(x, n, sign=1):
    """x as a sum of n bf16 numbers, all but the first times `sign`."""
    first = x.bfloat16().double()
    rest = x - first
    total = first
    for _ in range(n - 1):
        part = rest.bfloat16().double()
        rest = rest - part
        total = total + sign * part
    return total


def gradients(x, n_p=None, n_ds=None, n_lse=None, n_delta=None, sign=1):
    """g_q, g_k, g_v in 64 bits, and their bounds; with numbers given, p, ds and the keys' side's lse and
    delta are sums of so many bf16 numbers."""
    lens_q, lens_k, _, _, causal, scale = x.where
    g, q, k, v, out, lse = (t.double() for t in (x.g, x.q, x.k, x.v, x.out, x.lse))
    Hk, group, D = k.shape[1], q.shape[1] // k.shape[1], q.shape[2]
    cut = lambda t, n, sign=1: t if n is None else numbers(t, n, sign)  # noqa: E731
    res, tol = ([torch.zeros_like(t) for t in (q, k, v)] for _ in range(2))
    shared = lambda t: t.view(t.shape[0], Hk, group, D).sum(2)  # noqa: E731
    q0 = k0 = 0
    for nq, nk in zip(lens_q, lens_k):
        a, b = slice(q0, q0 + nq), slice(k0, k0 + nk)
        q0, k0 = q0 + nq, k0 + nk
        mask = ref.masks(nq, nk, causal, q.device)
        kk, vv = k[b].repeat_interleave(group, 1), v[b].repeat_interleave(group, 1)
        s = scale * torch.einsum("ihd,jhd->hij", q[a], kk)
        size = scale * torch.einsum("ihd,jhd->hij", q[a].abs(), kk.abs())
        l = lse[a].t()[..., None]
        delta = (g[a] * out[a]).sum(-1).t()[..., None]
        delta_size = (g[a] * out[a]).abs().sum(-1).t()[..., None]
        dp = torch.einsum("ihd,jhd->hij", g[a], vv)
        dp_size = torch.einsum("ihd,jhd->hij", g[a].abs(), vv.abs())
        p = torch.where(mask, (s - l).exp(), 0.0)
        p_keys = torch.where(mask, (s - scale * cut(l / scale, n_lse)).exp(), 0.0)
        ds, ds_keys = p * (dp - delta), p_keys * (dp - cut(delta, n_delta))
        res[0][a] = scale * torch.einsum("hij,jhd->ihd", cut(ds, n_ds, sign), kk)
        res[1][b] = scale * shared(torch.einsum("hij,ihd->jhd", cut(ds_keys, n_ds, sign), q[a]))
        res[2][b] = shared(torch.einsum("hij,ihd->jhd", cut(p_keys, n_p, sign), g[a]))
        off = D24 * ((2.2 * D + 11) * size + 14 * l.abs().nan_to_num(posinf=0.0) + 4)
        ds_off = ds.abs() * (2.0 ** -16 + D24 + off) + p * D24 * (2.2 * D * dp_size + 8 * dp_size + 21 * delta_size)
        n = nq * group
        tol[0][a] = scale * torch.einsum("hij,jhd->ihd", ds_off + 4.4 * (nk + 16) * D24 * ds.abs(), kk.abs())
        tol[1][b] = scale * shared(torch.einsum("hij,ihd->jhd", ds_off + 4.4 * (n + 16) * D24 * ds.abs(), q[a].abs()))
        tol[2][b] = shared(torch.einsum("hij,ihd->jhd", (2.0 ** -16 + off + 4.4 * (n + 16) * D24) * p, g[a].abs()))
    return res, [1.02 * t for t in tol]


def excess(got, want, tol):
    """The largest error in units of its bound (with the fp32 result's own rounding)."""
    room = tol + D24 * (want.abs() + tol) + 1e-37
    return float(((got.double() - want).abs() / room).max())


# name: (lens_q, lens_k, Hq, Hk, D, causal, kind), and the mistakes that it tells
ONE_P, ONE_DS = dict(n_p=1), dict(n_ds=1)
WRONG_SIGN, TWO_LSE, TWO_DELTA = dict(sign=-1), dict(n_lse=2), dict(n_delta=2)
CASES = {
    "64": (([40, 33], [150, 60], 4, 2, 64, False, "plain"), (ONE_P, ONE_DS, WRONG_SIGN)),
    "64 causal": (([70, 33], [90, 33], 4, 4, 64, True, "plain"), (ONE_P, ONE_DS, WRONG_SIGN)),
    "128": (([40, 33], [150, 60], 4, 2, 128, False, "plain"), (ONE_P, ONE_DS, WRONG_SIGN)),
    "80 causal": (([70, 33], [90, 33], 4, 4, 80, True, "plain"), (ONE_P, ONE_DS, WRONG_SIGN)),
    "a cluster, 64": (([64, 64], [70, 64], 8, 1, 64, False, "plain"), (ONE_P, ONE_DS, WRONG_SIGN)),
    "a cluster, 128": (([64, 64], [70, 64], 8, 1, 128, True, "plain"), (ONE_P, ONE_DS, WRONG_SIGN)),
    "lse": (([1] * 30, [8000 + 997 * i for i in range(30)], 2, 1, 16, False, "lse"), (TWO_LSE,)),
    "lse, 128": (([1] * 30, [8000 + 997 * i for i in range(30)], 2, 1, 72, False, "lse"), (TWO_LSE,)),
    "large lse": (([1] * 60, [40 + 5 * i for i in range(60)], 4, 4, 8, False, "large scores"), (TWO_LSE,)),
    "delta": (([1] * 30, [20 + 7 * i for i in range(30)], 4, 4, 8, False, "delta"), (TWO_DELTA,)),
    "delta, 128": (([1] * 30, [20 + 7 * i for i in range(30)], 4, 4, 72, False, "delta"), ()),
}
