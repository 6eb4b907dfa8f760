"""Attention at the ends of its range: the most queries, and so many keys that one CTA works for
seconds."""
import math

import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
from hadamard_precision_backprop_gb300 import build as hbuild

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    hbuild.build()
    hlq.hlq_read_device_status(clear=True)
    yield
    torch.cuda.empty_cache()
    assert hlq.hlq_read_device_status(clear=True) == 0


def need(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes * 2 ** 30:
        pytest.skip(f"needs {gigabytes} GB of device memory")


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,D", [(BF16, 8), (F32, 1)])
def test_the_most_queries(dtype, D, causal):
    """2^31 - 1024 queries of 16 keys: the same 1024 again and again, whose results are alike wherever
    they stand.  Causal: all but the last 16 see nothing."""
    need(90)
    T, n = 2 ** 31 - 1024, 1024
    gen = torch.Generator(device="cuda").manual_seed(1)
    part = torch.randn(n, 1, D, generator=gen, device="cuda").to(dtype)
    k, v = (torch.randn(16, 1, D, generator=gen, device="cuda").to(dtype) for _ in range(2))
    q = torch.empty(T, 1, D, dtype=dtype, device="cuda")
    q.view(-1, n, D)[:] = part.view(1, n, D)
    out, lse = hlq.hlq_attention(q, k, v, causal=causal)
    del q
    want, want_lse = hlq.hlq_attention(part, k, v, causal=causal)
    blocks, block_lses = out.view(-1, n * D), lse.view(-1, n)
    if causal:
        assert torch.equal(blocks[-1], want.view(-1)) and torch.equal(block_lses[-1], want_lse.view(-1))
        blocks, block_lses = blocks[:-1], block_lses[:-1]
        want, want_lse = torch.zeros_like(want), torch.full_like(want_lse, -torch.inf)
    for i in range(0, blocks.shape[0], 2 ** 18):
        assert (blocks[i:i + 2 ** 18] == want.view(1, -1)).all()
        assert (block_lses[i:i + 2 ** 18] == want_lse.view(1, -1)).all()


def test_keys_for_seconds():
    """One query of 400 million keys, the last tile of them not full: one CTA goes over them for longer
    than any single wait may take.  All scores are 0, and only the last five keys and values are not:
    lse is log n, out 5 / n, g_v is g / n and ds = (g . v - g . out) / n.  What rounds: the sum of
    ones, by whole multiples of 128 that fp32 holds up to 2^31; log n (19.8: two roundings of 2^-20);
    p, ds and the results to bf16 (2^-8 each); p by the error of its exponent, below 2^-16."""
    need(40)
    n, D, last = 400_000_005, 8, 5
    q = torch.zeros(1, 1, D, dtype=BF16, device="cuda")
    k = torch.zeros(n, 1, D, dtype=BF16, device="cuda")
    k[-last:] = 1
    out, lse = hlq.hlq_attention(q, k, k)
    assert hlq.hlq_read_device_status() == 0
    assert abs(float(lse) - math.log(n)) <= 2.0 ** -18
    assert ((out.double() * n / last - 1).abs() <= 2.0 ** -7).all()
    g = torch.ones(1, 1, D, dtype=BF16, device="cuda")
    g_q, g_k, g_v = hlq.hlq_attention_backward(g, q, k, k, out, lse)
    assert hlq.hlq_read_device_status() == 0
    ds = D / n * (1 - last / n)
    assert ((g_q.double() / (D ** -0.5 * ds * last) - 1).abs() <= 2.0 ** -6).all()
    assert not g_k.any()
    for part in g_v.split(10 ** 8):
        assert ((part.float() * n - 1).abs() <= 2.0 ** -6).all()
