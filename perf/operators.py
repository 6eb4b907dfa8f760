"""Cases of the operators that stand around a linear layer's backward pass in one training step: layer norm
(forward and backward), the log-probabilities of the tokens taken, the clipped policy loss with the gradient of
the logits, and the global gradient norm with clipping.

Where ``own`` is false, ``run`` is elementary torch arithmetic in fp32, rounded once at the end; where it is true,
it is the call a user makes of the package."""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.05
MAX_NORM, NORM_EPS = 1.0, 1e-6
GRAD_SCALE = 1024.0


def listed():
    return [
        # the residual stream of a 4096-wide model, 8 sequences of 2048 tokens: the add and the norm in one call
        dict(name="norm 16384x4096 residual", op="norm", T=16384, C=4096, x="bf16", y="bf16", w="bf16", residual=True),
        # an odd width (a pruned layer), fp32 master weights, a batch of some sequences
        dict(name="norm 2003x1001", op="norm", T=2003, C=1001, x="bf16", y="bf16", w="f32", residual=False),
        # backward of the norm before ViT-B's qkv: g_y is the fp32 g_x of the linear layer, the residual's gradient is added
        dict(name="norm bwd 12608x768", op="norm_bwd", T=12608, C=768, x="bf16", gy="f32", gx="bf16", w="bf16", residual=True),
        # the same for one image: latency
        dict(name="norm bwd 197x768", op="norm_bwd", T=197, C=768, x="bf16", gy="f32", gx="bf16", w="bf16", residual=False),
        # the widest layer of the 14336-wide MLP, everything 16 bits
        dict(name="norm bwd 16384x14336", op="norm_bwd", T=16384, C=14336, x="bf16", gy="bf16", gx="bf16", w="f32", residual=False),
        # log-probabilities of one sampled token of each of 4 sequences: rows are few and long
        dict(name="logprobs 4x128256", op="logprobs", T=4, V=128256, x="bf16"),
        # old log-probabilities of a batch of responses, a vocabulary of odd size, fp32 logits
        dict(name="logprobs 2048x32003", op="logprobs", T=2048, V=32003, x="f32"),
        # one short response
        dict(name="policy 17x32000", op="policy", T=17, V=32000, x="f32", ref=False),
        # an odd vocabulary in 16 bits: rows begin at any even address
        dict(name="policy 1000x50021", op="policy", T=1000, V=50021, x="bf16", ref=True),
        # two responses of 2048 tokens, a large vocabulary
        dict(name="policy 4096x128256", op="policy", T=4096, V=128256, x="bf16", ref=True),
        # a small network's gradients: latency
        dict(name="clip 2 layers of 64", op="clip", layers=2, width=64, x="f32", out="f32"),
        # fp32 weight gradients of 16 layers, written as the 16-bit gradients that an optimizer takes
        dict(name="clip 16 layers of 1280", op="clip", layers=16, width=1280, x="f32", out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "logprobs", "policy", "clip"])
    kind = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    if op in ("norm", "norm_bwd"):
        C = _log_int(rng, 17, 16384)
        if rng.random() < 0.6:
            C = max(16, C // 16 * 16)
        T = _log_int(rng, 1, max(1, min(50176, (16384 * 4096) // C)))
        if op == "norm":
            return dict(op=op, T=T, C=C, x=kind(), y=kind(), w=kind(), residual=rng.random() < 0.5)
        return dict(op=op, T=T, C=C, x=kind(), gy=kind(), gx=kind(), w=kind(), residual=rng.random() < 0.5)
    if op in ("logprobs", "policy"):
        V = _log_int(rng, 500, 128256)
        if rng.random() < 0.5:
            V = V // 16 * 16
        T = _log_int(rng, 1, max(1, min(4096, (2048 * 128256) // V)))
        return dict(op=op, T=T, V=V, x=kind(), **({"ref": rng.random() < 0.5} if op == "policy" else {}))
    width = _log_int(rng, 48, 1280)
    if rng.random() < 0.6:
        width = max(16, width // 16 * 16)
    return dict(op=op, layers=_log_int(rng, 1, 16), width=width, x=kind(), out=kind())


def _shapes(case):
    """The gradients of the layers: two norms, qkv and the projection with their biases, and the MLP's two products."""
    w = case["width"]
    m = 5 * w // 2
    return [(w,), (w,), (3 * w, w), (3 * w,), (w, w), (w,), (w,), (w,), (m, w), (m,), (w, m), (w,)] * case["layers"]


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op, dt = case["op"], DTYPES[case["x"]]
    if op in ("norm", "norm_bwd"):
        T, C, wdt = case["T"], case["C"], DTYPES[case["w"]]
        s["weight"] = (1 + 0.1 * _randn(gen, C)).to(wdt)
        s["bias"] = (0.1 * _randn(gen, C)).to(wdt)
        # activations: a scale and an offset of each channel, some channels far larger than the others
        scale = torch.where(torch.rand(C, generator=gen, device="cuda") < 0.01, 20.0, 1.0)
        x = _randn(gen, T, C) * scale + 0.3 * _randn(gen, C)
        s["x"] = x.to(dt)
        if op == "norm":
            s["residual"] = _randn(gen, T, C).to(dt) if case["residual"] else None
        else:
            h = s["x"].double()
            mean = h.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((h - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
            s["g_y"] = (1e-3 * _randn(gen, T, C)).to(DTYPES[case["gy"]])
            s["g_residual"] = (1e-3 * _randn(gen, T, C)).to(DTYPES[case["gx"]]) if case["residual"] else None
    elif op in ("logprobs", "policy"):
        T, V = case["T"], case["V"]
        logits = 2.5 * _randn(gen, T, V)
        s["tokens"] = torch.randint(V, (T,), generator=gen, device="cuda")
        rows = torch.arange(T, device="cuda")
        logits[rows, s["tokens"]] += 10.0  # a token that was sampled is one of the likely ones
        s["logits"] = logits.to(dt)
        if op == "policy":
            z = s["logits"].float()
            lp = z[rows, s["tokens"]].double() - torch.logsumexp(z, 1).double()
            # ratios around 1, as some updates after sampling; none at the very edge of the clipping, where rounding would decide
            ratio = (0.15 * _randn(gen, T)).double().exp()
            for edge in (1 - CLIP_LOW, 1 + CLIP_HIGH):
                ratio = torch.where((ratio - edge).abs() < 2e-3, ratio + 4e-3, ratio)
            s["old"] = (lp - ratio.log()).float()
            s["ref"] = (lp + 0.3 * _randn(gen, T)).float() if case["ref"] else None
            s["advantage"] = _randn(gen, T)
            # prompt and padding positions carry no loss: a quarter of the rows
            keep = torch.randperm(T, generator=gen, device="cuda") >= _masked(case)
            s["weight"] = keep.float() / max(1, T - _masked(case))
    else:
        s["grads"] = [(0.02 * _randn(gen, *shape)).to(dt) for shape in _shapes(case)]
        sizes = [g.numel() for g in s["grads"]]
        s["flat"] = torch.empty(sum(sizes), dtype=DTYPES[case["out"]], device="cuda")  # the optimizer's buffer
        s["outs"] = [v.view(g.shape) for v, g in zip(s["flat"].split(sizes), s["grads"])]
    return s


def _masked(case):
    return case["T"] // 4


def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import hadamard_precision_backprop_gb300 as hlq

    case = s["case"]
    op = case["op"]
    if op == "norm":
        return hlq.hlq_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, residual=s["residual"],
                                  out_dtype=DTYPES[case["y"]])
    if op == "norm_bwd":
        return hlq.hlq_layer_norm_backward(s["g_y"], s["x"], s["mean"], s["rstd"], s["weight"],
                                           g_residual=s["g_residual"], out_dtype=DTYPES[case["gx"]])
    if op == "logprobs":
        return hlq.hlq_token_logprobs(s["logits"], s["tokens"])
    if op == "policy":
        return hlq.hlq_policy_loss(s["logits"], s["tokens"], s["old"], s["advantage"], s["weight"], ref_logp=s["ref"],
                                   clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=KL_COEF, grad_scale=GRAD_SCALE)
    norm = hlq.hlq_clip_grad_norm(s["grads"], MAX_NORM, outs=s["outs"])
    return norm, s["flat"]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        mean = h.mean(1, keepdim=True)
        d = h - mean
        rstd = ((d * d).mean(1, keepdim=True) + EPS).rsqrt()
        y = d * rstd * s["weight"].float() + s["bias"].float()
        got = (y.to(DTYPES[case["y"]]), mean[:, 0], rstd[:, 0])
        return got if s["residual"] is None else got + (h.to(s["x"].dtype),)
    if op == "norm_bwd":
        g_y, rstd = s["g_y"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        a = g_y * s["weight"].float()
        g_x = rstd * (a - a.mean(1, keepdim=True) - xhat * (a * xhat).mean(1, keepdim=True))
        if s["g_residual"] is not None:
            g_x = g_x + s["g_residual"].float()
        return g_x.to(DTYPES[case["gx"]]), (g_y * xhat).sum(0), g_y.sum(0)
    if op == "logprobs":
        z = s["logits"].float()
        top = z.amax(1, keepdim=True)
        lse = (top + (z - top).exp().sum(1, keepdim=True).log())[:, 0]
        return z.gather(1, s["tokens"][:, None])[:, 0] - lse, lse
    if op == "policy":
        w, adv = s["weight"], s["advantage"]
        on = w != 0
        z = torch.where(on[:, None], s["logits"].float(), 0.0)
        e = (z - z.amax(1, keepdim=True)).exp()
        p = e / e.sum(1, keepdim=True)
        at = s["tokens"][:, None]
        lp = (z.gather(1, at) - z.amax(1, keepdim=True) - e.sum(1, keepdim=True).log())[:, 0]
        ratio = (lp - s["old"]).exp()
        inner, outer = ratio * adv, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv
        clipped = outer < inner
        policy = -torch.minimum(inner, outer)
        c = torch.where(clipped, 0.0, -inner)
        kl = torch.zeros_like(policy)
        if s["ref"] is not None:
            d = s["ref"] - lp
            kl = d.exp() - d - 1
            c = c + KL_COEF * (1 - d.exp())
        c = GRAD_SCALE * torch.where(on, w * c, 0.0)
        g = -c[:, None] * p
        g = g.scatter_add(1, at, c[:, None])
        wsum = lambda v: torch.where(on, w * v, 0.0).sum()  # noqa: E731
        stats = torch.stack([wsum(policy + KL_COEF * kl), wsum(policy), wsum(kl), wsum(clipped.float())])
        return stats, torch.where(on, lp, 0.0), g.to(s["logits"].dtype)
    flat = torch.cat([g.reshape(-1).float() for g in s["grads"]])
    norm = (flat * flat).sum().sqrt()
    coef = (MAX_NORM / (norm + NORM_EPS)).clamp(max=1.0)
    return torch.stack([norm, coef]), (flat * coef).to(s["flat"].dtype)


def work(case):
    op, size = case["op"], {"bf16": 2, "f32": 4}
    if op in ("norm", "norm_bwd"):
        n, C, T = case["T"] * case["C"], case["C"], case["T"]
        if op == "norm":
            per = size[case["x"]] * (3 if case["residual"] else 1) + size[case["y"]]
            return {"bytes": n * per + 2 * C * size[case["w"]] + 8 * T, "flops": 8 * n}
        per = size[case["x"]] + size[case["gy"]] + size[case["gx"]] * (2 if case["residual"] else 1)
        return {"bytes": n * per + C * size[case["w"]] + 8 * C + 8 * T, "flops": 14 * n}
    if op == "logprobs":
        return {"bytes": case["T"] * (case["V"] * size[case["x"]] + 16), "flops": 4 * case["T"] * case["V"]}
    if op == "policy":
        read, T, V = case["T"] - _masked(case), case["T"], case["V"]
        return {"bytes": (read + T) * V * size[case["x"]] + T * (28 if case["ref"] else 24) + 16, "flops": 7 * read * V}
    n = sum(math.prod(shape) for shape in _shapes(case))
    return {"bytes": n * (size[case["x"]] + size[case["out"]]) + 8, "flops": 3 * n}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        var, mean = torch.var_mean(h, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        y = torch.addcmul(s["bias"].double(), (h - mean[:, None]) * rstd[:, None], s["weight"].double())
        return (y, mean, rstd) if s["residual"] is None else (y, mean, rstd, h)
    if op == "norm_bwd":
        T, C = case["T"], case["C"]
        a, rstd = s["g_y"].double(), s["rstd"].double()
        xhat = s["x"].double().sub_(s["mean"].double()[:, None]).mul_(rstd[:, None])
        g_weight, g_bias = torch.einsum("tc,tc->c", a, xhat), a.sum(0)
        a.mul_(s["weight"].double())
        along = torch.einsum("tc,tc->t", a, xhat) / C
        a.sub_(a.sum(1)[:, None] / C).addcmul_(xhat, along[:, None], value=-1).mul_(rstd[:, None])
        return a if s["g_residual"] is None else a.add_(s["g_residual"].double()), g_weight, g_bias
    if op == "logprobs":
        z = s["logits"].double()
        lse = torch.logsumexp(z, 1)
        return z[torch.arange(case["T"], device="cuda"), s["tokens"]] - lse, lse
    if op == "policy":
        T = case["T"]
        rows, on = torch.arange(T, device="cuda"), s["weight"] > 0
        lps = torch.log_softmax(s["logits"].double(), 1)
        lp = lps[rows, s["tokens"]]
        adv, w = s["advantage"].double(), s["weight"].double()
        ratio = torch.exp(lp - s["old"].double())
        held = torch.where(adv > 0, ratio > 1 + CLIP_HIGH, ratio < 1 - CLIP_LOW) & (adv != 0)
        bounded = torch.where(adv > 0, ratio.clamp(max=1 + CLIP_HIGH), ratio.clamp(min=1 - CLIP_LOW))
        policy, slope = -bounded * adv, torch.where(held, 0.0, -ratio * adv)
        kl = torch.zeros_like(lp)
        if s["ref"] is not None:
            d = s["ref"].double() - lp
            kl, slope = torch.expm1(d) - d, slope - KL_COEF * torch.expm1(d)
        c = GRAD_SCALE * w * slope
        g = lps.exp_().mul_(-c[:, None])
        g[rows, s["tokens"]] += c
        stats = torch.stack([(w * (policy + KL_COEF * kl)).sum(), (w * policy).sum(), (w * kl).sum(),
                             (w * held.double()).sum()])
        return stats, torch.where(on, lp, 0.0), g
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    coef = torch.clamp(MAX_NORM / (norm + NORM_EPS), max=1.0)
    return torch.stack([norm, coef]), torch.cat([g.double().reshape(-1) for g in s["grads"]]) * coef
