"""Attention on the tensor cores with heads that are not whole eights (TMA reads them where their room is
one) and results in rows that begin anywhere: stores by single elements, sums of a cluster by single
elements, and the rows' pass by single elements that rounds g_out."""
import math

import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
from hadamard_precision_backprop_gb300 import build as hbuild
from tests import attention_ref as ref
from tests.test_gpu_attention import U, Case, placed

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    hbuild.build()
    hlq.hlq_read_device_status(clear=True)
    yield
    assert hlq.hlq_read_device_status(clear=True) == 0


def in_room(x, room):
    """x [T, H, D] in heads of `room` elements, of which the last hold NaN."""
    wide = torch.full((*x.shape[:2], room), math.nan, dtype=x.dtype, device=x.device)
    wide[..., :x.shape[2]] = x
    return wide[..., :x.shape[2]]


def traced(call, names):
    hlq.hlq_trace_begin(8)
    got = call()
    torch.cuda.synchronize()
    assert [n for n, _ in hlq.hlq_trace_end()] == names
    return got


SIZES = [(1, 8), (20, 24), (60, 64), (64, 64), (71, 72), (100, 104), (124, 128), (128, 128)]


@pytest.mark.parametrize("results", ["dense", "odd"])
@pytest.mark.parametrize("lens,Hq,Hk,causal", [([70, 150], 4, 2, True), ([600, 70], 8, 1, False), ([600, 70], 7, 1, True)], ids=str)
@pytest.mark.parametrize("D,room", SIZES)
def test_heads_in_more_room(D, room, lens, Hq, Hk, causal, results):
    """`results`: dense heads of D, or rows that begin at odd elements.  Eight (seven) heads that share
    one go to a cluster."""
    c = Case(BF16, lens, lens, Hq, Hk, D, causal, front=2, back=67)
    c.q, c.k, c.v = (in_room(x, room) for x in (c.q, c.k, c.v))
    clean = [c.clean(x) for x in (c.q, c.k, c.v)]
    want, want_lse, tol, lse_tol = ref.forward(*clean, *c.where, U[BF16])
    place = lambda shape, dt: placed(torch.zeros(shape, dtype=dt, device="cuda"), results)  # noqa: E731
    mine = place(c.q.shape, BF16)
    out, lse = traced(lambda: hlq.hlq_attention(c.q, c.k, c.v, out=mine, **c.kw), ["attn_fwd_tc"])
    assert out is mine
    ref.assert_within(out, want, tol, "out")
    none = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, none)
    ref.assert_within(lse.masked_fill(none, 0.0), want_lse.masked_fill(none, 0.0), lse_tol, "lse")
    out, lse = want.to(BF16), want_lse.float()
    for gout_dtype in (BF16, F32):
        g = (1e-2 * torch.randn(c.q.shape, generator=c.gen, device="cuda")).to(gout_dtype)
        grads, tols = ref.backward(g, *clean, out, lse, *c.where, U[BF16], U[BF16] if gout_dtype == F32 else 0.0)
        g[~c.inside_q] = math.nan
        for g_dtype in (BF16, F32):
            outs = [place(x.shape, g_dtype) for x in (c.q, c.k, c.v)]
            got = traced(lambda: hlq.hlq_attention_backward(
                in_room(g, room), c.q, c.k, c.v, in_room(out, room), lse, g_q=outs[0], g_k=outs[1], g_v=outs[2], **c.kw),
                ["attn_bwd_rows", "attn_bwd_tc"])
            for x, r, t, what in zip(got, grads, tols, ("g_q", "g_k", "g_v")):
                ref.assert_within(x, r, t, what)
