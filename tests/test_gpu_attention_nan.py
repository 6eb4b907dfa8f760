"""NaN within a sequence: no gradient that the formulas make NaN comes out as a number."""
import math

import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
from hadamard_precision_backprop_gb300 import build as hbuild
from tests.test_gpu_attention import Case

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    hbuild.build()
    hlq.hlq_read_device_status(clear=True)
    yield
    assert hlq.hlq_read_device_status(clear=True) == 0


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("gout", [BF16, F32])
@pytest.mark.parametrize("dtype,Hq,Hk,D", [(BF16, 4, 2, 64), (BF16, 4, 4, 128), (BF16, 8, 1, 64), (BF16, 2, 1, 136), (F32, 4, 2, 64)])
def test_one_key_of_nan(dtype, Hq, Hk, D, gout, causal):
    """One key of the second sequence is NaN: so is the log-sum-exp of each query that sees it, and
    with it that query's probabilities of all keys.  The last query sees all of them, so every g_k
    and g_v of the sequence is NaN; the other sequences' gradients are not."""
    lens = [130, 600, 40]
    at = 130 + 300
    c = Case(dtype, lens, lens, Hq, Hk, D, causal)
    c.k[at] = math.nan
    out, lse = hlq.hlq_attention(c.q, c.k, c.v, **c.kw)
    sees = slice(at if causal else 130, 730)
    assert out[sees].isnan().all() and lse[sees].isnan().all()
    g = (0.01 * torch.randn(c.q.shape, generator=c.gen, device="cuda")).to(gout)
    g_q, g_k, g_v = hlq.hlq_attention_backward(g, c.q, c.k, c.v, out, lse, **c.kw)
    assert g_q[sees].isnan().all()
    assert g_k[130:730].isnan().all() and g_v[130:730].isnan().all()
    for x in (out, lse, g_q, g_k, g_v):
        assert torch.isfinite(x[:130]).all() and torch.isfinite(x[730:]).all()
