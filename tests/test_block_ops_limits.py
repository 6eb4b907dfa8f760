"""Sizes and strides at the ends of what attention and its backward pass take: refused on the
host (no device needed)."""
import pytest

from tests.test_block_ops import FAKE, L, attention, backward, heads  # noqa: F401


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


@pytest.mark.parametrize("call,out", [(attention, "out"), (backward, "g_q")])
def test_output_strides_whose_product_leaves_64_bits(L, call, out):  # noqa: F811
    """2^24 heads 2^40 apart are 2^64 elements of a token, and not the few (less than none) that the low
    bits of the product say: with tokens 8 apart they overlap.  Tokens and heads the other way round alike."""
    for T, H, token, head in ((2, 2 ** 24, 8, 2 ** 40), (2 ** 24, 2, 2 ** 40, 8)):
        assert call(L, Tq=T, Tk=T, Hq=H, Hk=1, D=64, batch=1, **{out: heads(token=token, head=head)}) == 2


@pytest.mark.parametrize("call,out", [(attention, "out"), (backward, "g_q")])
def test_output_strides_at_their_limits(L, call, out):  # noqa: F811
    """One step less overlaps; exactly enough is taken (refused here for a later argument)."""
    for T, H, token, head in ((2, 4, 3 * 70 + 64, 70), (5, 3, 70, 4 * 70 + 64), (2, 1, 64, 0), (1, 2, 0, 64)):
        late = dict(lse=None)
        args = dict(Tq=T, Tk=T, Hq=H, Hk=1, D=64, batch=1, **late)
        assert call(L, **args, **{out: heads(token=token, head=head)}) == 1
        less = heads(token=token - 1, head=head) if token > head else heads(token=token, head=head - 1)
        assert call(L, **args, **{out: less}) == 2


def test_backward_passes_of_more_ctas_than_a_grid(L):  # noqa: F811
    """Both sides' CTAs are one grid, of less than 2^31: a size like any other, not a failed launch."""
    B = 2 ** 29
    for kw in (dict(batch=B, Hq=1, Hk=1, Tq=64, Tk=64, seqs=FAKE), dict(batch=1, Hq=2 ** 29 - 1, Hk=2 ** 29 - 1, Tq=1, Tk=1, seqs=FAKE),
               dict(batch=2 ** 30 - 2, Hq=1, Hk=1, Tq=64, Tk=64, seqs=FAKE)):
        n = (kw["Tq"] // 32 + kw["batch"] + 2) * kw["Hq"] + (kw["Tk"] // 32 + kw["batch"] + 2) * kw["Hk"]
        late = dict(scale=0.0)                          # is looked at after the sizes
        assert backward(L, D=8, **kw, **late) == (4 if n >= 2 ** 31 else 1)
        assert attention(L, D=8, **kw, **late) == 1     # its own grid is half of that
