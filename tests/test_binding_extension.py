"""The binding's extension module belongs to one torch: what is built, and what
is loaded, where torch is another."""
import os

import pytest
import torch

from hadamard_precision_backprop_gb300 import build as hbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    hbuild.build()


def test_another_torch_has_a_module_of_its_own(monkeypatch):
    path = hbuild.ext_path()
    assert os.path.exists(path) and hbuild.is_current(True)
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert hbuild.ext_path() != path
    assert not hbuild.is_current(True) and hbuild.is_current(False)
