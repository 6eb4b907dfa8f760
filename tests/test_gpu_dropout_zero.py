"""Dropout without a residual is a product: zeros that are kept keep their sign."""
import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
from hadamard_precision_backprop_gb300 import build as hbuild
from tests.test_gpu_dropout import halves

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    hbuild.build()


@pytest.mark.parametrize("x_dt,y_dt", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("T,C,ld", [(33, 40, 40), (33, 40, 48), (33, 41, 43), (5, 13, 13)])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_the_sign_of_a_kept_zero(p, T, C, ld, x_dt, y_dt):
    """Dense, rows of whole eights, single elements.  Dropped elements are +0."""
    wide = torch.zeros(T, ld, dtype=x_dt, device="cuda")
    x = wide[:, :C]
    x[::2] = -0.0
    y = hlq.hlq_dropout(x, p, 9, out_dtype=y_dt)
    kept = torch.from_numpy(halves(T * C, 9) >= round(p * 65536)).view(T, C).cuda()
    assert not y.any()
    assert torch.equal(torch.signbit(y), torch.signbit(x) & kept)
