"""Dropout against numpy's integers and 64-bit arithmetic: which elements are
kept, bit for bit, and their values; strides, alignments, in place, seeds."""
import math

import numpy as np
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
    assert hlq.hlq_read_device_status(clear=True) == 0


def halves(n, seed, first=0):
    """The 16-bit numbers of n elements from `first` (a multiple of 8): Philox4x32-10, eight for each block."""
    with np.errstate(over="ignore"):
        c = [np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64), None, None, None]
        c = [c[0] & np.uint64(0xFFFFFFFF), c[0] >> np.uint64(32), np.full_like(c[0], 4), np.zeros_like(c[0])]
        k0, k1 = seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF
        for _ in range(10):
            a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
            hi, lo = np.uint64(32), np.uint64(0xFFFFFFFF)
            c = [(b >> hi) ^ c[1] ^ np.uint64(k0), b & lo, (a >> hi) ^ c[3] ^ np.uint64(k1), a & lo]
            k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    out = np.empty((c[0].size, 8), np.int64)
    for i in range(8):
        out[:, i] = (c[i // 2] >> np.uint64(16 * (i % 2))) & np.uint64(0xFFFF)
    return out.reshape(-1)[:n]


def check(y, x, p, seed, residual):
    drop = int(np.rint(p * 65536))
    kept = torch.from_numpy(halves(x.numel(), seed) >= drop).view(x.shape).to(x.device)
    factor = 65536 / (65536 - drop) if drop < 65536 else 0.0
    want = torch.where(kept, x.double() * factor, 0.0)
    size = want.abs()
    if residual is not None:
        want, size = want + residual.double(), size + residual.double().abs()
    # the factor's rounding and (fp32) that of the product and sum, then the result's
    room = 2.0 ** -24 * 2 * size + torch.finfo(y.dtype).eps / 2 * want.abs() * 1.01 + 1e-40
    assert ((y.double() - want).abs() <= room).all()
    other = torch.zeros_like(y) if residual is None else residual
    assert torch.equal(y[~kept], other[~kept])
    return kept


@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (3, 8), (5, 13), (64, 768), (33, 1001), (2003, 65)])
@pytest.mark.parametrize("x_dt,y_dt", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("residual", [False, True])
def test_values(shape, x_dt, y_dt, residual):
    x = torch.randn(shape, device="cuda").to(x_dt)
    r = torch.randn(shape, device="cuda").to(y_dt) if residual else None
    for p, seed in ((0.0, 1), (0.1, 2 ** 63 + 12345), (0.5, 0), (1.0, 7), (1e-6, 3), (2.0 ** -17 * 3, 2 ** 64 - 1)):
        y = hlq.hlq_dropout(x, p, seed, residual=r, out_dtype=y_dt)
        assert y.dtype == y_dt
        check(y, x, p, seed, r)


@pytest.mark.parametrize("T,C", [(2 ** 23 + 1, 4096), (33, 2 ** 30)])
def test_elements_past_32_bits(T, C):
    """Above 2^35 elements: the blocks' numbers pass 32 bits too."""
    if torch.cuda.mem_get_info()[0] < 2 * T * C + 2 ** 30:
        pytest.skip("needs 70 GB of device memory")
    x = torch.ones(T, C, dtype=BF16, device="cuda")
    y = hlq.hlq_dropout(x, 0.5, 11, out=x).view(-1)
    for first in (0, 2 ** 31 - 800, 2 ** 32 - 800, 2 ** 35 - 800, T * C - 4096):
        n = min(4096, T * C - first)
        want = 2.0 * torch.from_numpy(halves(n, 11, first) >= 32768).to("cuda")
        assert torch.equal(y[first:first + n].float(), want)


def test_share_kept_and_other_seeds():
    x = torch.ones(4096, 4096, device="cuda")
    a, b = (hlq.hlq_dropout(x, 0.25, seed) for seed in (1, 2))
    n = x.numel()
    sigma = math.sqrt(0.25 * 0.75 / n)
    for y in (a, b):
        assert abs(float((y == 0).double().mean()) - 0.25) < 6 * sigma
    assert abs(float(((a == 0) & (b == 0)).double().mean()) - 0.0625) < 6 * math.sqrt(0.0625 * 0.9375 / n)


@pytest.mark.parametrize("C", [16, 24, 61])
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_strides_and_alignments(C, pad, shift):
    """The mask depends on an element's row and column alone."""
    T = 37

    def placed(v):
        flat = torch.full((T * (C + pad) + shift,), math.nan, dtype=v.dtype, device="cuda")
        view = flat[shift:].view(T, C + pad)[:, :C]
        view.copy_(v)
        return flat, view

    x, r = torch.randn(T, C, device="cuda").to(BF16), torch.randn(T, C, device="cuda")
    want = hlq.hlq_dropout(x, 0.3, 99, residual=r)
    check(want, x, 0.3, 99, r)
    (_, xs), (_, rs), (flat, out) = placed(x), placed(r), placed(torch.zeros_like(r))
    got = hlq.hlq_dropout(xs, 0.3, 99, residual=rs, out=out)
    assert got is out and torch.equal(out, want)
    assert flat.isnan().sum() == flat.numel() - T * C          # nothing between the rows
    assert torch.equal(hlq.hlq_dropout(x, 0.3, 99, residual=rs), want)


def test_broadcast_rows_and_in_place():
    row, x = torch.randn(1, 40, device="cuda"), torch.randn(9, 40, device="cuda")
    want = hlq.hlq_dropout(row.expand(9, 40).contiguous(), 0.4, 5, residual=x)
    assert torch.equal(hlq.hlq_dropout(row.expand(9, 40), 0.4, 5, residual=x), want)
    y = x.clone()
    assert hlq.hlq_dropout(row.expand(9, 40), 0.4, 5, residual=y, out=y) is y and torch.equal(y, want)
    y = x.clone()
    assert torch.equal(hlq.hlq_dropout(y, 0.4, 5, out=y), hlq.hlq_dropout(x, 0.4, 5))


def test_what_is_dropped_is_no_number():
    x = torch.full((64, 64), math.nan, device="cuda")
    y = hlq.hlq_dropout(x, 0.5, 11)
    kept = torch.from_numpy(halves(4096, 11) >= 32768).view(64, 64).cuda()
    assert torch.equal(y.isnan(), kept) and not y[~kept].any()


def test_the_gradient_is_the_same_call():
    """y is linear in x, so differences of y give the gradient exactly where they are representable."""
    x = torch.randint(-64, 64, (50, 30), device="cuda").float()
    step = torch.randint(-64, 64, (50, 30), device="cuda").float()
    y0, y1 = (hlq.hlq_dropout(v, 0.5, 21, residual=x) for v in (x, x + step))
    g = hlq.hlq_dropout(torch.ones_like(x), 0.5, 21)
    assert torch.equal(y1 - y0, g * step)


def test_seed_on_the_device_and_a_captured_graph():
    x = torch.randn(100, 33, device="cuda")
    seed = torch.tensor([-3], dtype=torch.int64, device="cuda")
    assert torch.equal(hlq.hlq_dropout(x, 0.2, seed), hlq.hlq_dropout(x, 0.2, 2 ** 64 - 3))
    assert torch.equal(hlq.hlq_dropout(x, 0.2, -3), hlq.hlq_dropout(x, 0.2, 2 ** 64 - 3))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        y = hlq.hlq_dropout(x, 0.2, seed)
        g = hlq.hlq_dropout(y, 0.2, seed)
    for s in (5, 6):
        seed.fill_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, hlq.hlq_dropout(x, 0.2, s)) and torch.equal(g, hlq.hlq_dropout(y, 0.2, s))


def test_python_and_extension_give_the_same(monkeypatch):
    x, r = torch.randn(70, 50, device="cuda"), torch.randn(70, 50, device="cuda").to(BF16)
    seed = torch.tensor(77, device="cuda")
    got = []
    for ext in (hlq._load_ext(), hlq._NoExt()):
        monkeypatch.setattr(hlq, "_ext", ext)
        got.append([hlq.hlq_dropout(x, 0.3, 77, residual=r), hlq.hlq_dropout(x, 0.3, seed, residual=r),
                    hlq.hlq_dropout(x, 0, 2 ** 64 - 1, out_dtype=BF16)])
        assert torch.equal(got[-1][0], got[-1][1])
    for a, b in zip(*got):
        assert a.dtype == b.dtype and torch.equal(a, b)
