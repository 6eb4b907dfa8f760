"""Attention, its backward pass and dropout as a block's training step uses them,
with the layer norm before and the linear layers between: against 64-bit
autograd of the same network, against differences, and with the layers' HLQ
backward pass in its place."""
import math

import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
from hadamard_precision_backprop_gb300 import build as hbuild
from tests.test_gpu_dropout import halves

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
LENS, HQ, HK, D, C, P, SEED = [40, 1, 129, 86], 4, 2, 32, 96, 0.25, 77
T = sum(LENS)                                            # 256


@pytest.fixture(scope="module", autouse=True)
def _built():
    hbuild.build()
    hlq.hlq_read_device_status(clear=True)
    yield
    assert hlq.hlq_read_device_status(clear=True) == 0


def inputs():
    gen = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return dict(x=randn(T, C), norm_w=1 + 0.1 * randn(C), norm_b=0.1 * randn(C),
                qkv_w=randn((HQ + 2 * HK) * D, C) / math.sqrt(C), proj_w=randn(C, HQ * D) / math.sqrt(HQ * D)), randn(T, C)


def offsets():
    return torch.tensor([0] + [sum(LENS[:i + 1]) for i in range(len(LENS))], dtype=torch.int32, device="cuda")


def reference(p, keep):
    """The block in 64 bits: x + dropout(proj(attention(qkv(norm(x)))))."""
    x = p["x"]
    d = x - x.mean(1, keepdim=True)
    y = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * p["norm_w"] + p["norm_b"]
    q, k, v = (y @ p["qkv_w"].t()).view(T, HQ + 2 * HK, D).split([HQ, HK, HK], 1)
    outs, at = [], 0
    for n in LENS:
        rows = slice(at, at + n)
        at += n
        kk, vv = (z[rows].repeat_interleave(HQ // HK, 1) for z in (k, v))
        s = torch.einsum("ihd,jhd->hij", q[rows], kk) / math.sqrt(D)
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1), -torch.inf)
        outs.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), vv))
    z = torch.cat(outs).reshape(T, HQ * D) @ p["proj_w"].t()
    return x + torch.where(keep, z * (65536 / (65536 - round(P * 65536))), 0.0)


def step(p, g):
    """Output and gradients through the package (the linear layers by torch)."""
    seqs = offsets()
    y, mean, rstd = hlq.hlq_layer_norm(p["x"], p["norm_w"], p["norm_b"])
    qkv = (y @ p["qkv_w"].t()).view(T, HQ + 2 * HK, D)
    q, k, v = qkv.split([HQ, HK, HK], 1)
    a, lse = hlq.hlq_attention(q, k, v, seqs=seqs, causal=True)
    out = hlq.hlq_dropout(a.view(T, HQ * D) @ p["proj_w"].t(), P, SEED, residual=p["x"])
    g_z = hlq.hlq_dropout(g, P, SEED)
    g_a = (g_z @ p["proj_w"]).view(T, HQ, D)
    g_qkv = hlq.hlq_attention_backward(g_a, q, k, v, a, lse, seqs=seqs, causal=True, packed=True).view(T, -1)
    g_x, g_nw, g_nb = hlq.hlq_layer_norm_backward(g_qkv @ p["qkv_w"], p["x"], mean, rstd, p["norm_w"], g_residual=g)
    return out, dict(x=g_x, norm_w=g_nw, norm_b=g_nb, qkv_w=g_qkv.t() @ y, proj_w=g_z.t() @ a.view(T, -1))


def test_a_block_against_autograd_in_64_bits():
    """Six stages, each with sums of at most 512 terms in fp32: relative to the result's norm
    6 x 512 x 2^-24 < 2e-4 if every rounding went the same way."""
    p, g = inputs()
    keep = torch.from_numpy(halves(T * C, SEED) >= round(P * 65536)).view(T, C).cuda()
    leaves = {n: t.double().requires_grad_() for n, t in p.items()}
    want = reference(leaves, keep)
    want.backward(g.double())
    out, grads = step(p, g)
    assert (out.double() - want.detach()).norm() <= 2e-4 * want.norm()
    for n, leaf in leaves.items():
        off = (grads[n].double() - leaf.grad).norm() / leaf.grad.norm()
        assert off <= 2e-4, (n, float(off))


def test_a_block_against_differences():
    """Central differences in 64 bits along random directions: their own error is of third order in
    the step (1e-4), 1e-7 of the slope or so."""
    p, g = inputs()
    keep = torch.from_numpy(halves(T * C, SEED) >= round(P * 65536)).view(T, C).cuda()
    _, grads = step(p, g)
    gen = torch.Generator(device="cuda").manual_seed(9)
    p64 = {n: t.double() for n, t in p.items()}
    for n in p:
        d = torch.randn(p[n].shape, generator=gen, device="cuda", dtype=torch.float64)
        up, down = ({**p64, n: p64[n] + s * 1e-4 * d} for s in (1, -1))
        slope = float(((reference(up, keep) - reference(down, keep)) * g.double()).sum()) / 2e-4
        got = float((grads[n].double() * d).sum())
        assert abs(got - slope) <= 3e-4 * float((grads[n].double() * d).norm()) * math.sqrt(d.numel()), n


def test_packed_gradients_are_the_layers_g_y():
    """bf16, the HLQ backward pass of the qkv layer and of the projection around the attention's:
    what it takes is the attention's own tensor, and its result that of a copy."""
    p, g = inputs()
    p = {n: t.to(BF16) if n != "x" else t for n, t in p.items()}
    seqs = offsets()
    y, mean, rstd = hlq.hlq_layer_norm(p["x"].to(BF16), p["norm_w"], p["norm_b"])
    xbar, sx = hlq.hlq_compress_activation(y)
    q, k, v = (y @ p["qkv_w"].t()).view(T, HQ + 2 * HK, D).split([HQ, HK, HK], 1)
    a, lse = hlq.hlq_attention(q, k, v, seqs=seqs, causal=True)
    abar, sa = hlq.hlq_compress_activation(a.view(T, -1))
    g_z = hlq.hlq_dropout(g, P, SEED, out_dtype=BF16)
    g_a, g_proj = hlq.hlq_linear_backward(g_z, p["proj_w"], abar, sa, seed=1)
    assert g_a.dtype == F32
    g_qkv = hlq.hlq_attention_backward(g_a.view(T, HQ, D), q, k, v, a, lse, seqs=seqs, causal=True, packed=True)
    parts = hlq.hlq_attention_backward(g_a.view(T, HQ, D), q, k, v, a, lse, seqs=seqs, causal=True)
    assert torch.equal(g_qkv, torch.cat(parts, 1))
    g_y, g_w = hlq.hlq_linear_backward(g_qkv.view(T, -1), p["qkv_w"], xbar, sx, seed=2)
    again = hlq.hlq_linear_backward(g_qkv.clone().view(T, -1), p["qkv_w"], xbar, sx, seed=2)
    assert torch.equal(g_y, again[0]) and torch.equal(g_w, again[1])
    g_x, *_ = hlq.hlq_layer_norm_backward(g_y, p["x"].to(BF16), mean, rstd, p["norm_w"], g_residual=g, out_dtype=F32)
    for t in (g_x, g_w, g_proj):
        assert torch.isfinite(t).all() and t.any()


def test_calls_on_two_streams_at_once():
    """Different shapes and passes side by side, many times, give what they give alone."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    calls = []
    for B, L, Hq, Hk, Dh, causal in ((3, 300, 8, 2, 64, True), (2, 700, 4, 1, 128, False), (1, 130, 6, 6, 80, True)):
        q = torch.randn(B * L, Hq, Dh, generator=gen, device="cuda").to(BF16)
        k, v = (torch.randn(B * L, Hk, Dh, generator=gen, device="cuda").to(BF16) for _ in range(2))
        g = torch.randn(B * L, Hq, Dh, generator=gen, device="cuda")

        def call(q=q, k=k, v=v, g=g, kw=dict(batch=B, causal=causal)):
            out, lse = hlq.hlq_attention(q, k, v, **kw)
            return (out, lse, *hlq.hlq_attention_backward(g, q, k, v, out, lse, **kw))

        calls.append(call)
    alone = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(20):
        for call, stream, to in zip(calls, streams, got):
            with torch.cuda.stream(stream):
                to.append(call())
    torch.cuda.synchronize()
    for want, runs in zip(alone, got):
        for run in runs:
            assert all(torch.equal(x, y) for x, y in zip(want, run))
