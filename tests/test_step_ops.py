"""The operators around the layer in a training step refuse bad arguments on
the host (no device needed): through the C ABI and through the binding."""
import ctypes

import pytest
import torch

import hadamard_precision_backprop_gb300 as hlq
from hadamard_precision_backprop_gb300 import build as hbuild

# A non-null address, never touched: every call below has one invalid argument.
FAKE = 1 << 20
FAKE_WS = 1 << 24
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    hbuild.build()
    return hlq.lib()


def norm(L, **kw):
    a = dict(x=FAKE, ldx=64, r=None, ldr=0, x_dt=1, w=FAKE, b=FAKE, w_dt=1, T=8, C=64, eps=1e-5,
             y=FAKE, ldy=64, y_dt=1, h=None, ldh=0, mean=FAKE, rstd=FAKE)
    a.update(kw)
    return L.hlq_layer_norm(*a.values(), None)


def test_layer_norm_validation(L):
    assert norm(L, x=None) == 1
    assert norm(L, y=None) == 1
    assert norm(L, x_dt=2) == 1
    assert norm(L, w_dt=-1) == 1
    assert norm(L, y_dt=7) == 1
    assert norm(L, eps=-1e-5) == 1
    assert norm(L, eps=NAN) == 1
    assert norm(L, eps=INF) == 1
    assert norm(L, r=FAKE, ldr=64) == 1               # a residual needs h
    assert norm(L, h=FAKE, ldh=64) == 1
    assert norm(L, mean=None) == 1                    # both statistics or neither
    assert norm(L, T=-1) == 2
    assert norm(L, C=0) == 2
    assert norm(L, ldx=63) == 2
    assert norm(L, ldx=-64) == 2
    assert norm(L, ldy=0) == 2                        # only an input repeats a row
    assert norm(L, r=FAKE, ldr=64, h=FAKE, ldh=0) == 2
    assert norm(L, T=1 << 31) == 4
    assert norm(L, C=1 << 31, ldx=1 << 31, ldy=1 << 31) == 4
    assert norm(L, x=FAKE + 1) == 3
    assert norm(L, y=FAKE + 2, y_dt=0) == 3
    assert norm(L, rstd=FAKE + 2) == 3
    assert norm(L, T=0, x=None, y=None) == 0          # nothing to do


def norm_bwd(L, **kw):
    a = dict(gy=FAKE, ldgy=64, gy_dt=0, x=FAKE, ldx=64, x_dt=1, mean=FAKE, rstd=FAKE, w=FAKE,
             w_dt=1, gr=None, ldgr=0, T=8, C=64, gx=FAKE, ldgx=64, gx_dt=1, gw=FAKE, gb=FAKE,
             ws=FAKE_WS, ws_bytes=1 << 30)
    a.update(kw)
    return L.hlq_layer_norm_backward(*a.values(), None)


def test_layer_norm_backward_validation(L):
    need = L.hlq_layer_norm_backward_workspace_bytes(8, 64)
    assert need > 0 and need % 256 == 0
    assert L.hlq_layer_norm_backward_workspace_bytes(-1, 64) == 0
    assert L.hlq_layer_norm_backward_workspace_bytes(8, 0) == 0
    for name in ("gy", "x", "mean", "rstd", "gx"):
        assert norm_bwd(L, **{name: None}) == 1, name
    for name in ("gy_dt", "x_dt", "w_dt", "gx_dt"):
        assert norm_bwd(L, **{name: 2}) == 1, name
    assert norm_bwd(L, C=0) == 2
    assert norm_bwd(L, ldgy=1) == 2
    assert norm_bwd(L, ldgx=0) == 2
    assert norm_bwd(L, gr=FAKE, ldgr=5) == 2
    assert norm_bwd(L, gy=FAKE + 2) == 3
    assert norm_bwd(L, gw=FAKE + 1) == 3
    assert norm_bwd(L, ws=FAKE_WS + 64) == 3
    assert norm_bwd(L, ws=None) == 5
    assert norm_bwd(L, ws_bytes=need - 256) == 5


def test_token_logprobs_validation(L):
    def call(**kw):
        a = dict(x=FAKE, ld=100, dt=1, tg=FAKE, T=4, V=100, scale=1.0, lp=FAKE, lse=None)
        a.update(kw)
        return L.hlq_token_logprobs(*a.values(), None)

    for name in ("x", "tg", "lp"):
        assert call(**{name: None}) == 1, name
    assert call(dt=3) == 1
    for bad in (0.0, -1.0, NAN, INF):
        assert call(scale=bad) == 1
    assert call(V=0) == 2
    assert call(ld=99) == 2
    assert call(T=-4) == 2
    assert call(V=1 << 31, ld=1 << 31) == 4
    assert call(tg=FAKE + 4) == 3
    assert call(x=FAKE + 1) == 3
    assert call(T=0, x=None, tg=None, lp=None) == 0


def test_policy_loss_validation(L):
    need = L.hlq_policy_loss_workspace_bytes(4, 100)
    assert need > 0 and need % 256 == 0
    assert L.hlq_policy_loss_workspace_bytes(4, 0) == 0

    def call(**kw):
        a = dict(x=FAKE, ld=100, dt=1, act=FAKE, old=FAKE, ref=FAKE, adv=FAKE, w=FAKE, T=4, V=100,
                 scale=1.0, lo=0.2, hi=0.2, kl=0.1, gs=1.0, stats=FAKE, lp=FAKE, g=FAKE, ldg=100,
                 ws=FAKE_WS, ws_bytes=need)
        a.update(kw)
        return L.hlq_policy_loss(*a.values(), None)

    for name in ("x", "act", "old", "adv", "w", "stats"):
        assert call(**{name: None}) == 1, name
    assert call(dt=5) == 1
    for bad in (0.0, NAN, INF):
        assert call(scale=bad) == 1
    assert call(lo=-0.1) == 1
    assert call(hi=NAN) == 1
    assert call(kl=INF) == 1
    assert call(gs=NAN) == 1
    assert call(V=0) == 2
    assert call(ldg=99) == 2
    assert call(ldg=0) == 2
    assert call(g=FAKE + 1) == 3
    assert call(old=FAKE + 2) == 3
    assert call(ws=FAKE_WS + 8) == 3
    assert call(ws=None) == 5
    assert call(ws_bytes=need - 256) == 5


def test_clip_grad_norm_validation(L):
    need = L.hlq_clip_grad_norm_workspace_bytes(2)
    assert need > 0 and need % 256 == 0
    assert L.hlq_clip_grad_norm_workspace_bytes(100000) > need
    assert L.hlq_clip_grad_norm_workspace_bytes(-1) == 0

    def call(n=2, g=(FAKE, FAKE), gdt=(0, 1), o=(FAKE, FAKE), odt=(0, 1), num=(8, 8), m=1.0,
             nc=FAKE, ws=FAKE_WS, ws_bytes=need):
        arr = lambda ct, v: None if v is None else (ct * len(v))(*v)  # noqa: E731
        return L.hlq_clip_grad_norm(n, arr(ctypes.c_void_p, g), arr(ctypes.c_int32, gdt),
                                    arr(ctypes.c_void_p, o), arr(ctypes.c_int32, odt),
                                    arr(ctypes.c_int64, num), m, nc, ws, ws_bytes, None)

    assert call(n=-1) == 1
    assert call(g=None) == 1
    assert call(gdt=None) == 1
    assert call(odt=None) == 1
    assert call(num=None) == 1
    assert call(nc=None) == 1
    assert call(m=-1.0) == 1
    assert call(m=NAN) == 1
    assert call(g=(FAKE, None)) == 1
    assert call(o=(None, FAKE)) == 1
    assert call(gdt=(0, 2)) == 1
    assert call(odt=(3, 0)) == 1
    assert call(num=(8, -8)) == 2
    assert call(num=(8, (1 << 40) + 1)) == 4
    assert call(g=(FAKE + 2, FAKE)) == 3
    assert call(o=(FAKE, FAKE + 1)) == 3
    assert call(nc=FAKE + 2) == 3
    assert call(ws=FAKE_WS + 16) == 3
    assert call(ws_bytes=need - 256) == 5
    assert call(ws=None) == 5


class _Fake:
    """Stands in for a CUDA tensor in the binding's checks."""

    def __init__(self, shape, dtype=torch.float32, stride=None, cuda=True, index=0):
        self.shape, self.dtype, self.is_cuda, self._index = torch.Size(shape), dtype, cuda, index
        self._meta = torch.empty(shape, dtype=dtype, device="meta")
        if stride is not None:
            self._meta = torch.empty_strided(shape, stride, dtype=dtype, device="meta")
        self.device = torch.device("cuda", index)

    def stride(self):
        return self._meta.stride()

    def is_contiguous(self):
        return self._meta.is_contiguous()

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self._index

    def numel(self):
        return self._meta.numel()

    def element_size(self):
        return self._meta.element_size()

    def data_ptr(self):
        return FAKE


@pytest.fixture
def no_call(monkeypatch):
    """The library fails the test if it is called; device 0 is current."""
    class _NoCall:
        def __getattr__(self, name):
            raise AssertionError(f"library called: {name}")

    monkeypatch.setattr(hlq, "lib", lambda: _NoCall())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def test_binding_refuses_rows_it_cannot_read(no_call):
    v = _Fake((64,))
    out = _Fake((8, 64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        hlq.hlq_layer_norm(torch.zeros(8, 64))
    with pytest.raises(ValueError, match="shape"):
        hlq.hlq_layer_norm(_Fake((64,)))
    with pytest.raises(ValueError, match="rows of x must be contiguous"):
        hlq.hlq_layer_norm(_Fake((8, 64), stride=(1, 8)))
    with pytest.raises(TypeError, match="dtype"):
        hlq.hlq_layer_norm(_Fake((8, 64), dtype=torch.float16))
    with pytest.raises(ValueError, match="is current"):
        hlq.hlq_layer_norm(_Fake((8, 64), index=1))
    with pytest.raises(ValueError, match="weight must have shape"):
        hlq.hlq_layer_norm(_Fake((8, 64)), _Fake((63,)))
    with pytest.raises(ValueError, match="one dtype"):
        hlq.hlq_layer_norm(_Fake((8, 64)), v, _Fake((64,), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="out must have shape"):
        hlq.hlq_layer_norm(_Fake((8, 64)), v, v, out=_Fake((8, 63)))
    with pytest.raises(ValueError, match="out is on cuda:1"):
        hlq.hlq_layer_norm(_Fake((8, 64)), v, v, out=_Fake((8, 64), index=1))
    with pytest.raises(ValueError, match="residual must be of dtype"):
        hlq.hlq_layer_norm(_Fake((8, 64)), v, v, out=out,
                           residual=_Fake((8, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="only with a residual"):
        hlq.hlq_layer_norm(_Fake((8, 64)), v, v, out=out, h=out)
    with pytest.raises(ValueError, match="with_stats"):
        hlq.hlq_layer_norm(_Fake((8, 64)), v, v, out=out, mean=_Fake((8,)), with_stats=False)


def test_binding_refuses_wrong_companions(no_call):
    x, v, s = _Fake((8, 64)), _Fake((64,)), _Fake((8,))
    ws = _Fake((1 << 20,), dtype=torch.uint8)
    back = lambda **kw: hlq.hlq_layer_norm_backward(  # noqa: E731
        **{**dict(g_y=x, x=x, mean=s, rstd=s, weight=v, out=x, g_weight=v, g_bias=v, ws=ws), **kw})
    with pytest.raises(ValueError, match="g_y must have shape"):
        back(g_y=_Fake((8, 32)))
    with pytest.raises(ValueError, match="mean must have shape"):
        back(mean=_Fake((7,)))
    with pytest.raises(ValueError, match="rstd must be of dtype"):
        back(rstd=_Fake((8,), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="g_residual must be of dtype"):
        back(g_residual=_Fake((8, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="with_weight_grads"):
        back(with_weight_grads=False)
    tok = _Fake((8,), dtype=torch.int64)
    with pytest.raises(ValueError, match="targets must be of dtype"):
        hlq.hlq_token_logprobs(x, _Fake((8,), dtype=torch.int32), logp=s, lse=s)
    with pytest.raises(ValueError, match="targets must have shape"):
        hlq.hlq_token_logprobs(x, _Fake((9,), dtype=torch.int64), logp=s, lse=s)
    loss = lambda **kw: hlq.hlq_policy_loss(**{**dict(  # noqa: E731
        logits=x, actions=tok, old_logp=s, advantages=s, weights=s, stats=_Fake((4,)), logp=s,
        out=x, ws=ws), **kw})
    with pytest.raises(ValueError, match="old_logp must have shape"):
        loss(old_logp=_Fake((4,)))
    with pytest.raises(ValueError, match="weights must be a contiguous"):
        loss(weights=_Fake((8,), stride=(2,)))
    with pytest.raises(ValueError, match="ref_logp is on cuda:1"):
        loss(ref_logp=_Fake((8,), index=1))
    with pytest.raises(ValueError, match="out must be of dtype"):
        loss(out=_Fake((8, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="with_grad"):
        loss(with_grad=False)


def test_binding_refuses_unclippable_gradients(no_call):
    g, nc, ws = _Fake((8, 4)), _Fake((2,)), _Fake((1 << 16,), dtype=torch.uint8)
    clip = lambda grads, **kw: hlq.hlq_clip_grad_norm(grads, 1.0, norm_coef=nc, ws=ws,  # noqa: E731
                                                      **kw)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        clip([g, _Fake((8, 4), stride=(1, 8))])
    with pytest.raises(ValueError, match="one device"):
        clip([g, _Fake((8, 4), index=1)])
    with pytest.raises(TypeError, match="dtype"):
        clip([_Fake((8,), dtype=torch.float64)])
    with pytest.raises(ValueError, match="1 outs for 2"):
        clip([g, g], outs=[g])
    with pytest.raises(ValueError, match="as many elements"):
        clip([g], outs=[_Fake((8, 3))])
    with pytest.raises(ValueError, match="norm_only"):
        clip([g], outs=[g], norm_only=True)
    with pytest.raises(ValueError, match="is current"):
        clip([_Fake((8,), index=1)])
