"""The binding's extension module belongs to one torch: what is built, and what
is loaded, where torch is another."""
import os

import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
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


def test_a_module_built_for_another_torch_is_not_loaded(monkeypatch):
    """The Python path does the call (here: refuses its argument)."""
    monkeypatch.setattr(hlq, "_ext", None)
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    with pytest.warns(RuntimeWarning, match="not built for this torch"):
        with pytest.raises(ValueError, match="CUDA tensor"):
            hlq.hlq_layer_norm(torch.zeros(8, 64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        hlq.hlq_token_logprobs(torch.zeros(8, 64), torch.zeros(8, dtype=torch.int64))


def test_a_torch_without_cuda_gets_the_library_alone(monkeypatch, tmp_path):
    commands = []

    def run(cmd, what):
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(hbuild, "_run", run)
    monkeypatch.setattr(hbuild, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(hbuild, "LIB", str(tmp_path / "libhlq.so"))
    monkeypatch.setattr(torch.version, "cuda", None)
    assert hbuild.build(force=True) == str(tmp_path / "libhlq.so")
    assert not any("hlq_torch.cpp" in a for cmd in commands for a in cmd)
    monkeypatch.undo()
    assert hbuild.can_bind()
