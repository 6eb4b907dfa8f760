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


@pytest.mark.parametrize("name", ["hlq_attn_fwd_tc.cu", "hlq_attn_bwd_tc.cu"])
def test_a_warp_votes_on_a_wait(name):
    """A bounded wait may end for one lane and give up for another.  Where a whole warp waits, the
    lanes vote before the instructions that need all of them (elections, products, TMEM accesses);
    only the one thread that loads waits alone."""
    warp = code("hlq_attn_tc.cuh")
    warp = warp[warp.index("bool wait_warp("):]
    warp = warp[:warp.index("\n}")]
    assert "while" not in warp and "!__all_sync(0xffffffffu, test())" in warp
    assert re.findall(r"return ([^;]*);", warp) == ["false", "true"]
    assert "__any_sync(0xffffffffu, gives_up(t0, abort_flag, status, steps))) return false;" in warp
    text = code(name)
    kernels = len(re.findall(r"AttnTile t;", text))
    assert text.count("return wait_warp(abort_flag, p.status, [&] { return mbar_test(b, phase & 1); });") == kernels
    lane = r"const auto wait_alone = \[&\]\(uint64_t\* b, uint32_t phase\) \{\s*return wait_lane\(b, phase, abort_flag, p\.status\);\s*\};"
    text, n = re.subn(lane, "", text)
    assert n == kernels
    text = re.sub(r"const auto load_\w+ = \[&\]\(.*?\n *\};", "", text, flags=re.S)  # one thread's
    text = text.replace("__all_sync(0xffffffffu, wait_alone(", "")
    assert "wait_lane(" not in text and "wait_alone(" not in text and "mbar_wait" not in text
