"""Attention and its backward pass in 64 bits, with how far a result may be off.

The bounds count, to first order and with 2 % for the rest: `u` for each rounding
of a factor of a product (2^-8 where the tensor cores take bf16, 0 in fp32), the
rounding of the result, and fp32 sums of n terms as n 2^-24 of the sum of their
magnitudes.  A score's error of d changes its probability by the factor 1 + d."""
import torch

F32 = 2.0 ** -24
SLACK = 1.02


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def masks(nq, nk, causal, device):
    i, j = torch.arange(nq, device=device)[:, None], torch.arange(nk, device=device)[None]
    return (j <= i + nk - nq) if causal else torch.ones(nq, nk, dtype=torch.bool, device=device)


def _scores(q, k, scale, group, mask):
    """Scores [Hq, nq, nk], and how far fp32 sums may put them off."""
    kk = k.repeat_interleave(group, 1)
    s = scale * torch.einsum("ihd,jhd->hij", q, kk)
    size = scale * torch.einsum("ihd,jhd->hij", q.abs(), kk.abs())
    return s.masked_fill(~mask, -torch.inf), (q.shape[2] + 4) * F32 * size


def forward(q, k, v, lens_q, lens_k, first_q, first_k, causal, scale, u):
    """out, lse and their bounds (without the rounding of out)."""
    q, k, v = q.double(), k.double(), v.double()
    group = q.shape[1] // k.shape[1]
    out, out_tol = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -torch.inf, dtype=torch.float64, device=q.device)
    lse_tol = torch.zeros_like(lse)
    q0, k0 = first_q, first_k
    for nq, nk in zip(lens_q, lens_k):
        rq, rk = slice(q0, q0 + nq), slice(k0, k0 + nk)
        q0, k0 = q0 + nq, k0 + nk
        if nq == 0 or nk == 0:
            continue
        mask = masks(nq, nk, causal, q.device)
        s, off = _scores(q[rq], k[rk], scale, group, mask)
        some = mask.any(1)
        top = s.amax(-1, keepdim=True).masked_fill(~some[None, :, None], 0.0)
        e = (s - top).exp()
        total = e.sum(-1, keepdim=True)
        p = torch.where(some[None, :, None], e / total, 0.0)
        lse[rq] = torch.where(some[None, :, None], top + total.log(), -torch.inf)[..., 0].t()
        worst = (off * mask).amax(-1) + (nk + 16) * F32        # of a probability, relative
        lse_tol[rq] = (worst + 4 * F32 * lse[rq].t().abs().nan_to_num(posinf=0.0)).t()
        vv = v[rk].repeat_interleave(group, 1)
        out[rq] = torch.einsum("hij,jhd->ihd", p, vv)
        size = torch.einsum("hij,jhd->ihd", p, vv.abs())
        out_tol[rq] = (u + 2 * worst.t()[..., None] + (nk + 16) * F32) * size
    return out, lse, SLACK * out_tol, SLACK * lse_tol


def backward(g, q, k, v, out, lse, lens_q, lens_k, first_q, first_k, causal, scale, u, u_g):
    """g_q, g_k, g_v and their bounds (without the rounding of the results).
    u_g: the rounding of g_out for its products."""
    g, q, k, v, out, lse = (x.double() for x in (g, q, k, v, out, lse))
    Hk, group = k.shape[1], q.shape[1] // k.shape[1]
    res = [torch.zeros_like(x) for x in (q, k, v)]
    tol = [torch.zeros_like(x) for x in (q, k, v)]
    shared = lambda x: x.view(x.shape[0], Hk, group, x.shape[2]).sum(2)  # noqa: E731
    q0, k0 = first_q, first_k
    for nq, nk in zip(lens_q, lens_k):
        rq, rk = slice(q0, q0 + nq), slice(k0, k0 + nk)
        q0, k0 = q0 + nq, k0 + nk
        if nq == 0 or nk == 0:
            continue
        mask = masks(nq, nk, causal, q.device)
        s, off = _scores(q[rq], k[rk], scale, group, mask)
        l = lse[rq].t()[..., None]
        p = torch.where(mask, (s - l).exp(), 0.0)
        off = off + 4 * F32 * l.abs().nan_to_num(posinf=0.0) + 16 * F32
        gg, vv, kk = g[rq], v[rk].repeat_interleave(group, 1), k[rk].repeat_interleave(group, 1)
        D = q.shape[2]
        dp = torch.einsum("ihd,jhd->hij", gg, vv)
        dp_size = torch.einsum("ihd,jhd->hij", gg.abs(), vv.abs())
        delta = (gg * out[rq]).sum(-1).t()[..., None]
        delta_size = (gg * out[rq]).abs().sum(-1).t()[..., None]
        ds = p * (dp - delta)
        # a rounded g_out meets v - out: sum |g| |v - out| <= sum |g| |v| + sum |g| |out|
        ds_off = (u + off) * ds.abs() + p * ((u_g + (D + 4) * F32) * (dp_size + delta_size))
        res[2][rk] = shared(torch.einsum("hij,ihd->jhd", p, gg))
        n = (nq * group + 8) * F32
        tol[2][rk] = shared(torch.einsum("hij,ihd->jhd", (u + u_g + off + n) * p, gg.abs()))
        res[0][rq] = scale * torch.einsum("hij,jhd->ihd", ds, kk)
        tol[0][rq] = scale * torch.einsum("hij,jhd->ihd", ds_off + (nk + 8) * F32 * ds.abs(), kk.abs())
        res[1][rk] = scale * shared(torch.einsum("hij,ihd->jhd", ds, q[rq]))
        tol[1][rk] = scale * shared(torch.einsum("hij,ihd->jhd", ds_off + n * ds.abs(), q[rq].abs()))
    return res, [SLACK * t for t in tol]


def assert_within(got, ref, tol, what):
    """Each value within its bound and the rounding of its type; NaN nowhere."""
    got64 = got.double()
    room = tol + half_step(got.dtype) * (ref.abs() + tol) + 1e-37
    bad = ~((got64 - ref).abs() <= room) & ~(got64 == ref)
    if bad.any():
        at = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: "
                             f"{float(got64[at])} for {float(ref[at])}, allowed {float(room[at])}")
