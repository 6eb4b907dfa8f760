"""The bounds of tests/attention_two_numbers.py tell two bf16 numbers from one, three from two, and a
second number of the wrong sign (mistakes planted in 64-bit arithmetic on the CPU); the kernels keep them."""
import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
from hadamard_precision_backprop_gb300 import build as hbuild
from tests import attention_two_numbers as two


@pytest.mark.parametrize("name", two.CASES)
def test_the_bounds_tell_a_number_less(name):
    args, mistakes = two.CASES[name]
    x = two.Inputs(*args)
    want, tol = two.gradients(x)
    right, _ = two.gradients(x, n_p=2, n_ds=2, n_lse=3, n_delta=3)
    for r, w, t in zip(right, want, tol):
        assert two.excess(r, w, t) <= 1
    for mistake in mistakes:
        wrong, _ = two.gradients(x, **{**dict(n_p=2, n_ds=2, n_lse=3, n_delta=3), **mistake})
        assert max(two.excess(r, w, t) for r, w, t in zip(wrong, want, tol)) > 1.5, mistake


@pytest.mark.gpu
@pytest.mark.parametrize("name", two.CASES)
def test_the_kernels_keep_them(name):
    hbuild.build()
    hlq.hlq_read_device_status(clear=True)
    x = two.Inputs(*two.CASES[name][0], device="cuda")
    want, tol = two.gradients(x)
    seqs, seqs_k = x.offsets()
    hlq.hlq_trace_begin(8)
    got = hlq.hlq_attention_backward(x.g, x.q, x.k, x.v, x.out, x.lse, seqs=seqs, seqs_k=seqs_k, causal=x.causal,
                                     out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert [n for n, _ in hlq.hlq_trace_end()] == ["attn_bwd_rows", "attn_bwd_tc"]
    for r, w, t, what in zip(got, want, tol, ("g_q", "g_k", "g_v")):
        assert two.excess(r, w, t) <= 1, (what, two.excess(r, w, t))
    assert hlq.hlq_read_device_status() == 0
