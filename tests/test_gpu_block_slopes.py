"""A block's gradients against differences, along directions in which a gradient's error cannot hide."""
import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
from hadamard_precision_backprop_gb300 import build as hbuild
from tests.test_gpu_block_step import C, P, SEED, T, inputs, reference, step
from tests.test_gpu_dropout import halves

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    hbuild.build()
    hlq.hlq_read_device_status(clear=True)
    yield
    assert hlq.hlq_read_device_status(clear=True) == 0


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_slopes_along_the_gradients(seed):
    """Directions are the gradient itself, each element times a factor between 1/2 and 3/2: the slope is
    then a sum of squares.  Gradients are within 2e-4 of their norm (sums of at most 512 terms in fp32 in
    six stages), so a slope is off by 2e-4 times the gradient's and the direction's norms at most; the
    central differences' own error, of third order in steps of 1e-4, is 1e-6 of that or so."""
    p, g = inputs()
    keep = torch.from_numpy(halves(T * C, SEED) >= round(P * 65536)).view(T, C).cuda()
    _, grads = step(p, g)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    p64 = {n: t.double() for n, t in p.items()}
    for n in p:
        got = grads[n].double()
        d = got * (0.5 + torch.rand(got.shape, generator=gen, device="cuda", dtype=torch.float64))
        d /= d.abs().max()
        up, down = ({**p64, n: p64[n] + s * 1e-4 * d} for s in (1, -1))
        slope = float(((reference(up, keep) - reference(down, keep)) * g.double()).sum()) / 2e-4
        assert abs(float((got * d).sum()) - slope) <= 2.1e-4 * float(got.norm() * d.norm()), n
