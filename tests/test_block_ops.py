"""Attention, its backward pass and dropout refuse bad arguments on the host (no
device needed): through the C ABI and through the binding."""
import ctypes
import importlib.util
import os
import random

import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
from hadamard_precision_backprop_gb300 import build as hbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# A non-null address, never touched: every call below has one invalid argument.
FAKE = 1 << 20
FAKE_WS = 1 << 24
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    hbuild.build()
    return hlq.lib()


def heads(ptr=FAKE, token=256, head=64):
    return ctypes.byref(hlq._Heads(ptr, token, head))


def attention(L, **kw):
    a = dict(q=heads(), k=heads(), v=heads(), dt=1, Tq=32, Tk=32, Hq=4, Hk=4, D=64, seqs=None, seqs_k=None,
             batch=2, causal=1, scale=0.125, out=heads(), lse=FAKE)
    a.update(kw)
    return L.hlq_attention(*a.values(), None)


def backward(L, **kw):
    a = dict(g=heads(), g_out_dt=0, q=heads(), k=heads(), v=heads(), out=heads(), dt=1, lse=FAKE, Tq=32, Tk=32, Hq=4,
             Hk=4, D=64, seqs=None, seqs_k=None, batch=2, causal=1, scale=0.125, g_q=heads(), g_k=heads(), g_v=heads(),
             g_dt=1, ws=FAKE_WS, ws_bytes=1 << 30)
    a.update(kw)
    return L.hlq_attention_backward(*a.values(), None)


@pytest.mark.parametrize("call", [attention, backward])
def test_attention_validation(L, call):
    assert call(L, dt=2) == 1
    assert call(L, q=None) == 1
    assert call(L, v=heads(None)) == 1
    assert call(L, lse=None) == 1
    assert call(L, scale=0.0) == 1
    assert call(L, scale=-1.0) == 1
    assert call(L, scale=NAN) == 1
    assert call(L, scale=INF) == 1
    assert call(L, scale=2.0 ** -65) == 1
    assert call(L, scale=2.0 ** 65) == 1
    assert call(L, seqs_k=FAKE) == 1                    # offsets of the keys alone
    assert call(L, Tq=-1) == 2
    assert call(L, Hk=3) == 2
    assert call(L, Hq=0) == 2
    assert call(L, D=0) == 2
    assert call(L, batch=0) == 2
    assert call(L, batch=3) == 2                        # 32 rows are not three sequences
    assert call(L, seqs=FAKE, Tk=16) == 2               # other keys need offsets of their own
    assert call(L, q=heads(token=-1)) == 2
    assert call(L, k=heads(head=(1 << 40) + 1)) == 2
    assert call(L, D=257) == 4
    assert call(L, Tq=1 << 31, batch=1) == 4
    assert call(L, Tq=1 << 30, Tk=1 << 30) == 4         # Tq Hq
    assert call(L, q=heads(FAKE + 1)) == 3
    assert call(L, lse=FAKE + 2) == 3
    assert call(L, seqs=FAKE + 2) == 3


def test_attention_outputs_do_not_overlap(L):
    assert attention(L, out=heads(token=255)) == 2
    assert attention(L, out=heads(token=0)) == 2
    assert attention(L, out=heads(head=63)) == 2
    assert attention(L, out=heads(token=64, head=32 * 64 - 1)) == 2
    assert attention(L, out=heads(None)) == 1
    assert attention(L, Tq=0, Tk=0, q=heads(None), k=heads(None), v=heads(None), out=heads(None), lse=None) == 0


def test_attention_backward_validation(L):
    assert backward(L, g_out_dt=3) == 1
    assert backward(L, g_dt=-1) == 1
    assert backward(L, g_q=heads(token=0)) == 2
    assert backward(L, g_k=heads(head=1)) == 2
    assert backward(L, g_v=heads(None)) == 1
    assert backward(L, g_v=heads(FAKE + 2), g_dt=0) == 3
    assert backward(L, ws=None) == 5
    need = L.hlq_attention_backward_workspace_bytes(32, 4, 64, 1, 0)
    assert need >= 2 * 32 * 4 * 4 + 32 * 4 * 64 * 2
    assert L.hlq_attention_backward_workspace_bytes(32, 4, 64, 1, 1) < need
    assert L.hlq_attention_backward_workspace_bytes(32, 4, 257, 1, 1) == 0
    assert L.hlq_attention_backward_workspace_bytes(-1, 4, 64, 1, 1) == 0
    assert backward(L, ws_bytes=need - 1) == 5
    assert backward(L, ws=FAKE_WS + 16) == 3


def dropout(L, **kw):
    a = dict(x=FAKE, ldx=64, x_dt=1, r=None, ldr=0, T=8, C=64, p=0.1, seed=1, d_seed=None, y=FAKE, ldy=64, y_dt=1)
    a.update(kw)
    return L.hlq_dropout(*a.values(), None)


def test_dropout_validation(L):
    for p in (-0.1, 1.1, NAN, INF):
        assert dropout(L, p=p) == 1
    assert dropout(L, x=None) == 1
    assert dropout(L, y=None) == 1
    assert dropout(L, x_dt=5) == 1
    assert dropout(L, y_dt=2) == 1
    assert dropout(L, T=-1) == 2
    assert dropout(L, C=0) == 2
    assert dropout(L, ldx=63) == 2
    assert dropout(L, ldy=0) == 2
    assert dropout(L, r=FAKE, ldr=1) == 2
    assert dropout(L, T=1 << 31) == 4
    assert dropout(L, y=FAKE + 2, y_dt=0) == 3
    assert dropout(L, d_seed=FAKE + 4) == 3
    assert dropout(L, T=0, x=None, y=None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(8, 2, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        hlq.hlq_attention(x, x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        hlq.hlq_attention_backward(x, x, x, x, x, x[..., 0])
    with pytest.raises(ValueError, match="CUDA tensor"):
        hlq.hlq_dropout(x[0], 0.1, 1)


@pytest.mark.gpu
def test_binding_refuses_what_does_not_fit():
    q = torch.zeros(8, 4, 64, device="cuda")
    k = torch.zeros(8, 2, 64, device="cuda")
    seqs = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    bad = [
        (dict(k=k[:, :1].expand(8, 3, 64)), "divide"), (dict(k=k.bfloat16()), "dtype"), (dict(v=k[:4]), "shape"),
        (dict(k=k[..., :32], v=k[..., :32]), "heads of"), (dict(q=q[0]), "shape"), (dict(q=q.transpose(0, 2)), "contiguous"),
        (dict(seqs=seqs.long()), "dtype"), (dict(seqs=seqs[:1]), "shape"), (dict(seqs=seqs, batch=3), "batch is 3"),
        (dict(seqs_k=seqs), "needs seqs"), (dict(seqs=seqs.cpu()), "CUDA"), (dict(out=q.bfloat16()), "dtype"),
        (dict(lse=torch.zeros(4, 8, device="cuda")), "shape"),
    ]
    for kw, match in bad:
        with pytest.raises(ValueError, match=match):
            hlq.hlq_attention(**{**dict(q=q, k=k, v=k), **kw})
    with pytest.raises(TypeError):
        hlq.hlq_attention(q.half(), k.half(), k.half())
    with pytest.raises(hlq.HLQError, match="SHAPE"):
        hlq.hlq_attention(q, k, k, batch=3)
    with pytest.raises(hlq.HLQError, match="SHAPE"):
        hlq.hlq_attention(q[..., :0], k[..., :0], k[..., :0])
    with pytest.raises(hlq.HLQError, match="UNSUPPORTED"):
        hlq.hlq_attention(*[torch.zeros(8, 2, 257, device="cuda")] * 3)
    lse = torch.zeros(8, 4, device="cuda")
    ok = dict(g_out=q, q=q, k=k, v=k, out=q, lse=lse)
    bad = [(dict(lse=lse[:, :2]), "contiguous|shape"), (dict(g_out=q[:4]), "shape"), (dict(out=q.bfloat16()), "dtype"),
           (dict(k=k[:4], v=k[:4], packed=True), "as many keys"), (dict(packed=True, g_q=q), "packed"),
           (dict(g_k=q), "shape"), (dict(g_q=q.clone(), g_k=k.bfloat16()), "dtype")]
    for kw, match in bad:
        with pytest.raises(ValueError, match=match):
            hlq.hlq_attention_backward(**{**ok, **kw})
    with pytest.raises(ValueError, match="seed"):
        hlq.hlq_dropout(lse, 0.1, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        hlq.hlq_dropout(lse, 0.1, 1, residual=lse[:4])
    with pytest.raises(hlq.HLQError, match="INVALID"):
        hlq.hlq_dropout(lse, 1.5, 1)


def _cases():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_performance_cases_are_well_formed():
    m = _cases()
    listed = m.listed()
    assert len({c["name"] for c in listed}) == len(listed)
    rng = random.Random(5)
    most = max(m.work(c)["flops"] for c in listed)
    for c in listed + [m.draw(rng) for _ in range(200)]:
        w = m.work(c)
        assert w["bytes"] > 0 and 0 < w["flops"] <= most
