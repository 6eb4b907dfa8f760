"""The example of a whole policy step runs and learns."""
import os
import runpy

import pytest

import hadamard_precision_backprop_gb300 as hlq
from hadamard_precision_backprop_gb300 import build as hbuild

pytestmark = pytest.mark.gpu

EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                       "policy_step.py")


def test_policy_example_learns():
    """64 questions, 512 answers: chance is 1 in 512; an untrained policy stays
    below 2 %, and one whose gradients point the right way is far above it."""
    hbuild.build()
    hlq.hlq_read_device_status(clear=True)
    rewards = runpy.run_path(EXAMPLE)["main"](say=lambda *_: None)
    assert max(rewards[:2]) < 0.02
    assert sum(rewards[-5:]) / 5 > 0.2
    assert hlq.hlq_read_device_status(clear=True) == 0
