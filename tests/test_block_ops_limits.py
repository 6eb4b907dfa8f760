"""Sizes and strides at the ends of what attention and its backward pass take: refused on the
host (no device needed)."""
import pytest

from tests.test_block_ops import L, attention, backward, heads  # noqa: F401


@pytest.mark.parametrize("call", [attention, backward])
def test_lengths_whose_tiles_leave_32_bits(L, call):  # noqa: F811
    """A tile of up to 256 rows may reach past a sequence's end: positions are counted in 32 bits."""
    for T in (2 ** 31 - 1, 2 ** 31 - 128, 2 ** 31 - 1023):
        assert call(L, Tq=T, Hq=1, Hk=1, D=8, batch=1) == 4
        assert call(L, Tq=32, Tk=T, Hq=1, Hk=1, D=8, batch=1) == 4
    # the longest are taken: refused here for what is checked after the sizes
    T = 2 ** 31 - 1024
    assert call(L, Tq=T, Hq=1, Hk=1, D=8, batch=1, scale=0.0) == 1
    assert call(L, Tk=T, Hq=1, Hk=1, D=8, batch=1, scale=0.0) == 1
