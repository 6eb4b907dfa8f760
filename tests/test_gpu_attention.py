"""Attention and its backward pass against the formulas in 64 bits: lengths from
none to several tiles, masks that leave rows empty, shared heads, head sizes,
strides and alignments, rows of no sequence, NaN beside a sequence, streams and
captured graphs."""
import math

import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
from hadamard_precision_backprop_gb300 import build as hbuild
from tests import attention_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    hbuild.build()
    hlq.hlq_read_device_status(clear=True)
    yield
    assert hlq.hlq_read_device_status(clear=True) == 0


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def placed(x, layout):
    """x [T, H, D] with the same values in another layout."""
    T, H, D = x.shape
    if layout == "dense":
        return x.contiguous()
    if layout == "part":           # of a wider row, as a qkv layer's output
        wide = torch.full((T, H + 5, D), math.nan, dtype=x.dtype, device=x.device)
        view = wide[:, 2:2 + H]
    elif layout == "heads first":
        view = torch.empty((H, T, D), dtype=x.dtype, device=x.device).transpose(0, 1)
    else:                          # "odd": rows begin anywhere
        flat = torch.full((T * (H * D + 3) + 1,), math.nan, dtype=x.dtype, device=x.device)
        view = flat[1:].view(T, H * D + 3)[:, :H * D].view(T, H, D)
    view.copy_(x)
    return view


class Case:
    """Inputs of one call: sequences with `lens_q` queries and `lens_k` keys, `front` rows before
    the first and `back` rows behind the last that hold NaN."""

    def __init__(self, dtype, lens_q, lens_k, Hq, Hk, D, causal, front=0, back=0, layout="dense", seed=0,
                 offsets=None, scale=None, spread=1.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lens_q, self.lens_k, self.causal = lens_q, lens_k, causal
        self.front, self.D = front, D
        Tq, Tk = front + sum(lens_q) + back, front + sum(lens_k) + back
        q, k, v = randn(gen, Tq, Hq, D), randn(gen, Tk, Hk, D), randn(gen, Tk, Hk, D)
        q *= spread * torch.linspace(0.2, 2.0, Hq, device="cuda")[:, None]
        for x in (q, k, v):
            x[:front] = math.nan
            x[x.shape[0] - back:] = math.nan
        self.q, self.k, self.v = (placed(x.to(dtype), layout) for x in (q, k, v))
        self.gen = gen
        self.varied = offsets if offsets is not None else front > 0 or back > 0 or len(set(lens_q)) > 1 \
            or len(set(lens_k)) > 1
        off = lambda lens: torch.tensor([front] + [front + sum(lens[:i + 1]) for i in range(len(lens))],  # noqa: E731
                                        dtype=torch.int32, device="cuda")
        same = lens_q == lens_k
        self.kw = dict(causal=causal)
        if scale is not None:
            self.kw["scale"] = scale
        self.scale = D ** -0.5 if scale is None else scale
        if self.varied:
            self.kw.update(seqs=off(lens_q), seqs_k=None if same else off(lens_k))
        else:
            self.kw.update(batch=len(lens_q))
        self.inside_q = torch.zeros(Tq, dtype=torch.bool, device="cuda")
        self.inside_q[front:front + sum(lens_q)] = True
        self.where = (lens_q, lens_k, front, front, causal, self.scale)

    def clean(self, x):
        return torch.nan_to_num(x, nan=0.0)

    def check_forward(self, u):
        out, lse = hlq.hlq_attention(self.q, self.k, self.v, **self.kw)
        want, want_lse, tol, lse_tol = ref.forward(self.clean(self.q), self.clean(self.k), self.clean(self.v),
                                                   *self.where, u)
        ref.assert_within(out, want, tol, "out")
        none = want_lse == -math.inf
        assert torch.equal(lse == -math.inf, none)
        ref.assert_within(lse.masked_fill(none, 0.0), want_lse.masked_fill(none, 0.0), lse_tol, "lse")
        assert not out[~self.inside_q].any()
        return out, lse, want, want_lse

    def check_backward(self, u, gout_dtype, g_dtype=None, layout="dense", packed=False):
        want, want_lse, _, _ = ref.forward(self.clean(self.q), self.clean(self.k), self.clean(self.v), *self.where, u)
        out, lse = want.to(self.q.dtype), want_lse.float()
        g = (1e-2 * randn(self.gen, *self.q.shape)).to(gout_dtype)
        u_g = u if gout_dtype == F32 else 0.0
        grads, tols = ref.backward(g, self.clean(self.q), self.clean(self.k), self.clean(self.v), out, lse,
                                   *self.where, u, u_g)
        g = g.clone()
        g[~self.inside_q] = math.nan
        g, out = placed(g, layout), placed(torch.where(self.inside_q[:, None, None], out, math.nan).to(out.dtype), layout)
        got = hlq.hlq_attention_backward(g, self.q, self.k, self.v, out, lse, out_dtype=g_dtype, packed=packed, **self.kw)
        if packed:
            Hq, Hk = self.q.shape[1], self.k.shape[1]
            assert got.is_contiguous() and got.shape[1] == Hq + 2 * Hk
            got = got.split([Hq, Hk, Hk], 1)
        for x, r, t, what in zip(got, grads, tols, ("g_q", "g_k", "g_v")):
            assert x.dtype == (g_dtype or self.q.dtype)
            ref.assert_within(x, r, t, what)


U = {BF16: 2.0 ** -8, F32: 0.0}
LENGTHS = [[1], [5, 5, 5], [0, 5, 1, 0, 130], [128], [129, 129], [127, 1, 256, 257], [511, 30], [700]]
HEADS = [(1, 1, 64), (4, 2, 128), (3, 1, 80), (2, 2, 8), (6, 2, 40)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_forward(lens, heads, causal, dtype):
    Case(dtype, lens, lens, *heads, causal).check_forward(U[dtype])


@pytest.mark.parametrize("dtype,gout", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_backward(lens, heads, causal, dtype, gout):
    Case(dtype, lens, lens, *heads, causal).check_backward(U[dtype], gout, packed=len(lens) % 2 == 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens_q,lens_k", [([5], [300]), ([300], [5]), ([1, 1, 1], [1000, 0, 129]), ([260, 0, 3], [130, 7, 3]),
                                           ([64, 64], [200, 200]), ([200, 200], [64, 64]), ([0], [40]), ([40], [0])])
def test_other_numbers_of_keys(lens_q, lens_k, causal, dtype):
    """Causal: the last query sees all keys; with fewer keys than queries the first ones see nothing."""
    c = Case(dtype, lens_q, lens_k, 4, 2, 64, causal)
    c.check_forward(U[dtype])
    c.check_backward(U[dtype], F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [1, 20, 100, 136, 256])
@pytest.mark.parametrize("layout", ["dense", "part", "heads first", "odd"])
def test_layouts_and_head_sizes(layout, D, dtype):
    c = Case(dtype, [70, 150], [70, 150], 4, 2, D, True, layout=layout)
    c.check_forward(U[dtype])
    c.check_backward(U[dtype], BF16, layout=layout)
    c.check_backward(U[dtype], F32, F32, layout=layout)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 200])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_of_no_sequence(causal, D, dtype):
    """NaN in rows before the first and behind the last sequence reaches nothing; their results are zeros."""
    c = Case(dtype, [200, 0, 131], [200, 0, 131], 2, 1, D, causal, front=3, back=140)
    c.check_forward(U[dtype])
    c.check_backward(U[dtype], F32)
    c.check_backward(U[dtype], BF16, packed=True)


@pytest.mark.parametrize("D", [64, 128, 72])
@pytest.mark.parametrize("lens_q,lens_k,heads,causal", [
    ([1150], [1150], (32, 8), True), ([1150], [1150], (32, 8), False), ([1024] * 5, [1024] * 5, (8, 4), True),
    ([1280, 0, 130, 2600], [1280, 0, 130, 2600], (16, 2), True), ([300, 1025], [1900, 770], (31, 1), True),
    ([1400], [1025], (26, 13), True), ([1900], [1900], (20, 4), True), ([2000], [1793], (20, 5), True),
    ([700, 900, 4000], [2900, 3000, 1], (9, 9), True), ([200, 0, 1500], [900, 1000, 700], (22, 2), False),
    ([700 + 50 * (i % 5) for i in range(258)],) * 2 + ((2, 1), False)],
    ids=lambda x: str(x[:5]) if isinstance(x, (list, tuple)) else str(x))
def test_long_sequences_of_many_heads(lens_q, lens_k, heads, causal, D):
    """Two tiles of queries a CTA: the last with one or none of them, either of them seeing no key."""
    varied = len(set(lens_q)) > 1
    c = Case(BF16, lens_q, lens_k, *heads, D, causal, front=3 * varied, back=200 * varied)
    c.check_forward(U[BF16])


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,D", [(F32, 32), (F32, 20), (F32, 64), (F32, 50), (F32, 128), (F32, 72), (F32, 160), (BF16, 132)])
def test_many_tiles_in_fp32(dtype, D, causal):
    lens = [70, 1, 130, 0] * 9
    c = Case(dtype, lens, lens, 12, 4, D, causal, front=2, back=67)
    c.check_forward(U[dtype])
    c.check_backward(U[dtype], F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 100])
def test_offsets_past_32_bits(D, dtype):
    """Tokens 2^23 + 8 elements apart: from the 256th on an element's offset passes 2^31."""
    T, step = 300, 2 ** 23 + 8
    gen = torch.Generator(device="cuda").manual_seed(D)
    small = [randn(gen, T, h, D).to(dtype) for h in (4, 2, 2, 4, 4)]
    kw = dict(batch=2, causal=True)

    def far(x, room, at):
        view = room[at:].as_strided((T, x.shape[1], D), (step, D, 1))
        view.copy_(x)
        return view

    room = torch.empty(T * step, dtype=dtype, device="cuda")
    q, k, v, g = (far(x, room, i * 1024) for i, x in enumerate(small[:4]))
    out = far(small[4], room, 4096)
    want, want_lse = hlq.hlq_attention(*small[:3], **kw)
    got, lse = hlq.hlq_attention(q, k, v, out=out, **kw)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    grads = [far(torch.zeros_like(x), room, (5 + i) * 1024) for i, x in enumerate(small[:3])]
    for x, y in zip(hlq.hlq_attention_backward(g, q, k, v, got, lse, g_q=grads[0], g_k=grads[1], g_v=grads[2], **kw),
                    hlq.hlq_attention_backward(small[3], *small[:3], want, want_lse, **kw)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_batch_that_is_mostly_padding(dtype):
    """Two short sequences in 3000 rows; queries and keys with offsets of their own."""
    c = Case(dtype, [5, 64], [130, 9], 4, 2, 64, True, front=700, back=2231)
    c.check_forward(U[dtype])
    c.check_backward(U[dtype], F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("poison", [math.nan, math.inf])
def test_a_sequence_of_nan_reaches_no_other(poison, dtype):
    """The sequence between two others holds NaN or infinities; tiles of 64 and 128 rows reach into it."""
    lens = [150, 90, 170]
    a = Case(dtype, lens, lens, 4, 2, 64, False)
    out, lse = hlq.hlq_attention(a.q, a.k, a.v, **a.kw)
    g = (0.01 * randn(a.gen, *a.q.shape)).to(dtype)
    grads = hlq.hlq_attention_backward(g, a.q, a.k, a.v, out, lse, **a.kw)
    bad = slice(150, 240)
    for x in (a.q, a.k, a.v, g):
        x[bad] = poison
    out2, lse2 = hlq.hlq_attention(a.q, a.k, a.v, **a.kw)
    mixed, mixed_lse = out.clone(), lse.clone()
    mixed[bad], mixed_lse[bad] = poison, poison
    grads2 = hlq.hlq_attention_backward(g, a.q, a.k, a.v, mixed, mixed_lse, **a.kw)
    keep = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
    keep[bad] = False
    for x, y in zip((out, lse, *grads), (out2, lse2, *grads2)):
        assert torch.equal(x[keep], y[keep])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_scores(dtype):
    """Scores of hundreds: the probabilities are nearly one-hot and the maximum rises from tile to tile."""
    c = Case(dtype, [500], [500], 2, 2, 64, False, spread=20.0)
    c.k *= torch.linspace(0.1, 3.0, 500, device="cuda")[:, None, None].to(dtype)
    c.check_forward(U[dtype])
    c.check_backward(U[dtype], dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [2.0 ** -64, 1e-6, 3.0])
def test_scales(scale, dtype):
    c = Case(dtype, [150], [150], 2, 1, 64, True, scale=scale)
    c.check_forward(U[dtype])
    c.check_backward(U[dtype], F32)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads", [(8, 1, 64), (7, 1, 128), (12, 2, 80), (3, 1, 64)], ids=str)
def test_key_heads_that_many_share(heads, causal):
    """Long enough that a tile of keys is shared out over a cluster, evenly or not."""
    c = Case(BF16, [600, 70], [600, 70], *heads, causal)
    c.check_backward(U[BF16], BF16)
    c.check_backward(U[BF16], F32, F32, packed=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scale_and_broadcast_inputs(dtype):
    """A scale of the caller's; one key head expanded to four (strides of 0)."""
    c = Case(dtype, [130, 40], [130, 40], 4, 4, 64, True, scale=0.3)
    c.k, c.v = c.k[:, :1].expand(-1, 4, -1), c.v[:, :1].expand(-1, 4, -1)
    c.check_forward(U[dtype])
    c.check_backward(U[dtype], F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_equal_calls_give_equal_bits_and_offsets_do_not_matter(dtype):
    """The same sequences as `batch` and as offsets; twice."""
    a = Case(dtype, [140] * 3, [140] * 3, 4, 2, 64, True)
    b = Case(dtype, [140] * 3, [140] * 3, 4, 2, 64, True, offsets=True)
    got = []
    for c in (a, b, a):
        out, lse = hlq.hlq_attention(c.q, c.k, c.v, **c.kw)
        g = (out.float() * 0.3).to(dtype)
        got.append((out, lse, *hlq.hlq_attention_backward(g, c.q, c.k, c.v, out, lse, **c.kw)))
    for x, y, z in zip(*got):
        assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("many,front,back", [(40, 0, 0), (128, 300, 1), (129, 0, 0), (256, 5, 0), (257, 130, 515), (1000, 1, 0), (1025, 257, 129)])
def test_many_sequences(many, front, back, causal, dtype):
    """More sequences than a warp looks at in one step, most of them short or empty."""
    lens = [(7 * i * i) % 11 + (150 if i % 97 == 5 else 0) for i in range(many)]
    lens_k = lens if many % 2 else [(5 * i) % 9 + (270 if i % 89 == 3 else 0) for i in range(many)]
    c = Case(dtype, lens, lens_k, 2, 1, 64, causal, front=front, back=back)
    c.check_forward(U[dtype])
    c.check_backward(U[dtype], BF16)


@pytest.mark.parametrize("at", [0, 3, 130, 299])
def test_bad_offsets_among_many(at):
    q = torch.randn(3000, 1, 64, device="cuda").to(BF16)
    off = 10 * torch.arange(301, dtype=torch.int32)
    for bad in (-7, 3001, int(off[at]) + 25):
        seqs = off.clone()
        seqs[at] = bad
        hlq.hlq_read_device_status(clear=True)
        out, lse = hlq.hlq_attention(q, q, q, seqs=seqs.cuda())
        assert hlq.hlq_read_device_status(clear=True) & hlq.DEV_BADCODE
        hlq.hlq_attention_backward(q, q, q, q, out, lse, seqs=seqs.cuda())
        assert hlq.hlq_read_device_status(clear=True) & hlq.DEV_BADCODE


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offsets", [False, True])
def test_no_keys_or_no_queries_at_all(offsets, dtype):
    for lens_q, lens_k in (([130, 5], [0, 0]), ([0, 0], [130, 5]), ([0, 0], [0, 0])):
        if not offsets:
            lens_q, lens_k = [max(lens_q)] * 2, [max(lens_k)] * 2
        c = Case(dtype, lens_q, lens_k, 4, 2, 64, True, offsets=offsets)
        c.check_forward(U[dtype])
        c.check_backward(U[dtype], F32)


def test_bad_offsets_raise_the_flag():
    """Offsets that decrease or leave the tensors: nothing outside is touched."""
    q = torch.randn(300, 2, 64, device="cuda").to(BF16)
    for off in ([0, 200, 100, 300], [0, 100, 400], [-5, 300]):
        hlq.hlq_read_device_status(clear=True)
        seqs = torch.tensor(off, dtype=torch.int32, device="cuda")
        out, lse = hlq.hlq_attention(q, q, q, seqs=seqs)
        assert hlq.hlq_read_device_status(clear=True) & hlq.DEV_BADCODE
        hlq.hlq_attention_backward(q, q, q, q, out, lse, seqs=seqs)
        assert hlq.hlq_read_device_status(clear=True) & hlq.DEV_BADCODE


def test_outputs_of_the_caller():
    c = Case(BF16, [130, 70], [130, 70], 4, 2, 64, True)
    out, lse = hlq.hlq_attention(c.q, c.k, c.v, **c.kw)
    mine, my_lse = torch.zeros(200, 6, 64, dtype=BF16, device="cuda"), torch.empty_like(lse)
    got = hlq.hlq_attention(c.q, c.k, c.v, out=mine[:, 1:5], lse=my_lse, **c.kw)
    assert got[1] is my_lse and torch.equal(my_lse, lse) and torch.equal(mine[:, 1:5], out)
    assert not mine[:, 0].any() and not mine[:, 5].any()
    g = torch.randn_like(out)
    want = hlq.hlq_attention_backward(g, c.q, c.k, c.v, out, lse, **c.kw)
    wide = torch.zeros(200, 10, 64, dtype=BF16, device="cuda")
    hlq.hlq_attention_backward(g, c.q, c.k, c.v, out, lse, g_q=wide[:, 1:5], g_k=wide[:, 5:7], g_v=wide[:, 7:9], **c.kw)
    for x, y in zip(want, (wide[:, 1:5], wide[:, 5:7], wide[:, 7:9])):
        assert torch.equal(x, y)
    assert not wide[:, 0].any() and not wide[:, 9].any()


def test_python_and_extension_give_the_same(monkeypatch):
    c = Case(BF16, [130, 70], [130, 70], 4, 2, 64, True)
    g = torch.randn_like(c.q)
    got = []
    for ext in (hlq._load_ext(), hlq._NoExt()):
        monkeypatch.setattr(hlq, "_ext", ext)
        out, lse = hlq.hlq_attention(c.q, c.k, c.v, **c.kw)
        got.append((out, lse, hlq.hlq_attention_backward(g, c.q, c.k, c.v, out, lse, packed=True, **c.kw),
                    *hlq.hlq_attention_backward(g, c.q, c.k, c.v, out, lse, out_dtype=F32, **c.kw)))
    for x, y in zip(*got):
        assert x.dtype == y.dtype and torch.equal(x, y)


def test_another_stream_and_a_captured_graph():
    """Two graphs of the same calls share no workspace; replays follow their inputs."""
    shapes = [([200, 57], 64), ([129], 128)]
    runs = []
    stream = torch.cuda.Stream()
    for lens, D in shapes:
        c = Case(BF16, lens, lens, 4, 2, D, True, seed=len(lens))
        g = torch.randn_like(c.q)

        def call(c=c, g=g):
            out, lse = hlq.hlq_attention(c.q, c.k, c.v, **c.kw)
            return out, hlq.hlq_attention_backward(g, c.q, c.k, c.v, out, lse, packed=True, **c.kw)

        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            call()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = call()
        runs.append((c, call, graph, got))
    for c, call, _, _ in runs:
        c.q.mul_(0.5)
    for _, _, graph, _ in runs:
        graph.replay()
    for _, call, _, got in runs:
        for x, y in zip(call(), got):
            assert torch.equal(x, y)
