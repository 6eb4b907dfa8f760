"""Rules of the tensor-core kernels that no run can show without a hang, read from their sources
(no device needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hadamard_precision_backprop_gb300", "csrc")
TMEM = ["hlq_gemm_tc.cu", "hlq_attn_fwd_tc.cu", "hlq_attn_bwd_tc.cu"]


def code(name):
    """A source without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", TMEM)
def test_the_next_kernel_is_let_in_after_tmem_is_held(name):
    """A CTA of the next kernel takes TMEM before it waits for this one.  If it came to an SM whose
    CTA of this kernel has none yet, each could wait for the other.  One thread's trigger counts for
    its CTA, so a trigger stands behind the CTA's barrier that follows the allocation, or behind the
    allocation in the allocating warp's own block."""
    text = code(name)
    triggers = [m.start() for m in re.finditer(r"pdl_trigger\(\)", text)]
    assert triggers
    for at in triggers:
        held = [m.start() for m in re.finditer(r"tcgen05\.alloc|\balloc\(&bar\.tmem", text[:at])]
        assert held, "a trigger without an allocation before it"
        between = text[held[-1]:at]
        opened = text[:held[-1]].rstrip().endswith("{")
        assert "__syncthreads();" in between or (opened and "}" not in between), between
