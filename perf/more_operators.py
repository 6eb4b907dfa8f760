"""Cases of the operators between a block's linear layers in one training step: softmax attention over packed
sequences, its backward pass (which recomputes the probabilities), and dropout from a counter-based generator
whose mask is never stored, with the residual added.

Where ``own`` is false, ``run`` is elementary torch arithmetic in fp32, rounded once at the end; where it is true,
it is the call a user makes of the package."""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LARGEST = 8 * 32 * 2048 * 2048  # query-key pairs of the largest listed case, all heads


def listed():
    return [
        # ViT-B: 64 images of 197 tokens, q, k and v are views of the qkv layer's output
        dict(name="attention 64x197", op="attention", B=64, L=197, ragged=False, Hq=12, Hk=12, D=64, x="bf16", causal=False),
        # a Llama layer with 8 key-value heads, 8 sequences of 2048 tokens
        dict(name="attention 8x2048 causal", op="attention", B=8, L=2048, ragged=False, Hq=32, Hk=8, D=128, x="bf16", causal=True),
        # prompts and answers of any length packed one after the other, a head of 80
        dict(name="attention packed 24, up to 1500", op="attention", B=24, L=1500, ragged=True, Hq=16, Hk=4, D=80, x="bf16", causal=True),
        # one short text: latency
        dict(name="attention 1x77", op="attention", B=1, L=77, ragged=False, Hq=8, Hk=8, D=64, x="bf16", causal=True),
        # one long document, queries that share one key-value head
        dict(name="attention 1x16384 causal", op="attention", B=1, L=16384, ragged=False, Hq=4, Hk=1, D=128, x="bf16", causal=True),
        # the backward passes of the first two: the output's gradient is the fp32 g_x of the projection
        dict(name="attention bwd 64x197", op="attention_bwd", B=64, L=197, ragged=False, Hq=12, Hk=12, D=64, x="bf16", gout="f32", causal=False),
        dict(name="attention bwd 8x2048 causal", op="attention_bwd", B=8, L=2048, ragged=False, Hq=32, Hk=8, D=128, x="bf16", gout="bf16", causal=True),
        # packed sequences of any length, a head of 80
        dict(name="attention bwd packed 24, up to 1500", op="attention_bwd", B=24, L=1500, ragged=True, Hq=16, Hk=4, D=80, x="bf16", gout="f32", causal=True),
        # a small network in fp32
        dict(name="attention bwd 5x129 f32", op="attention_bwd", B=5, L=129, ragged=False, Hq=6, Hk=6, D=32, x="f32", gout="f32", causal=False),
        # the residual stream of a 4096-wide model, 8 sequences of 2048 tokens
        dict(name="dropout 16384x4096 residual", op="dropout", T=16384, C=4096, x="bf16", y="bf16", residual=True, p=0.1),
        # an odd width, a gradient in fp32 going back to a 16-bit branch
        dict(name="dropout 2003x1001", op="dropout", T=2003, C=1001, x="f32", y="bf16", residual=False, p=0.25),
        # one image: latency
        dict(name="dropout 197x768 residual", op="dropout", T=197, C=768, x="bf16", y="f32", residual=True, p=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention_bwd", "attention_bwd", "dropout"])
    if op == "dropout":
        C = _log_int(rng, 17, 16384)
        if rng.random() < 0.6:
            C = max(16, C // 16 * 16)
        T = _log_int(rng, 1, max(1, min(50176, (16384 * 4096) // C)))
        return dict(op=op, T=T, C=C, x=rng.choice(["bf16", "f32"]), y=rng.choice(["bf16", "f32"]), residual=rng.random() < 0.5,
                    p=rng.choice([0.0, 0.05, 0.1, 0.25, 0.5]))
    D = rng.choice([32, 48, 64, 64, 72, 80, 96, 128, 128])
    Hk = rng.choice([1, 2, 3, 4, 8, 12])
    Hq = Hk * rng.choice([1, 1, 2, 4, 7])
    L = _log_int(rng, 1, min(16384, int(math.sqrt(LARGEST / Hq))))
    B = _log_int(rng, 1, max(1, min(64, LARGEST // (Hq * L * L), 32768 // L)))
    case = dict(op=op, B=B, L=L, ragged=B > 1 and rng.random() < 0.5, Hq=Hq, Hk=Hk, D=D,
                x="bf16" if rng.random() < 0.85 else "f32", causal=rng.random() < 0.6)
    if op == "attention_bwd":
        case["gout"] = rng.choice(["bf16", "f32"])
    return case


def _lengths(case):
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [L] * B
    rng = random.Random(B * 1000003 + L)  # one sequence is the longest, the others are spread over the logarithm
    return [L] + [_log_int(rng, 1, L) for _ in range(B - 1)]


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    dt = DTYPES[case["x"]]
    if case["op"] == "dropout":
        T, C = case["T"], case["C"]
        s["x"] = _randn(gen, T, C).to(dt)
        s["residual"] = _randn(gen, T, C).to(DTYPES[case["y"]]) if case["residual"] else None
        s["seed"] = random.Random(seed).getrandbits(63)
        return s
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    lengths = _lengths(case)
    T = sum(lengths)
    # what the qkv layer gives: some heads look at few tokens, some at all of them
    qkv = _randn(gen, T, Hq + 2 * Hk, D)
    qkv[:, :Hq] *= 0.5 + 1.5 * torch.rand(Hq, 1, generator=gen, device="cuda")
    qkv[:, Hq + Hk:] += 0.3 * _randn(gen, Hk, D)
    s["qkv"] = qkv.to(dt)
    s["q"], s["k"], s["v"] = s["qkv"].split([Hq, Hk, Hk], 1)
    s["seqs"] = torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32, device="cuda") if case["ragged"] else None
    if case["op"] == "attention_bwd":
        s["out"], s["lse"] = _attention(s)
        s["g_out"] = (1e-3 * _randn(gen, T, Hq, D)).to(DTYPES[case["gout"]])
    return s


def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import hadamard_precision_backprop_gb300 as hlq

    case = s["case"]
    if case["op"] == "dropout":
        return hlq.hlq_dropout(s["x"], case["p"], s["seed"], residual=s["residual"], out_dtype=DTYPES[case["y"]])
    if case["op"] == "attention":
        return hlq.hlq_attention(s["q"], s["k"], s["v"], seqs=s["seqs"], batch=case["B"], causal=case["causal"])
    # one tensor, which is the g_y of the qkv layer
    return hlq.hlq_attention_backward(s["g_out"], s["q"], s["k"], s["v"], s["out"], s["lse"], seqs=s["seqs"],
                                      batch=case["B"], causal=case["causal"], packed=True)


def _plain(s):
    op = s["case"]["op"]
    return _dropout(s) if op == "dropout" else _attention(s) if op == "attention" else _attention_bwd(s)


def _places(s):
    """Token of each place of [B, L], whether it is one, and the place (sequence, position) of each token."""
    case, dev = s["case"], s["q"].device
    T, B, L = s["q"].shape[0], case["B"], case["L"]
    start = torch.arange(B + 1, device=dev) * L if s["seqs"] is None else s["seqs"].long()
    token = start[:-1, None] + torch.arange(L, device=dev)
    there = token < start[1:, None]
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(start, t, right=True) - 1
    return token.clamp(max=T - 1), there, b, t - start[b]


def _padded(x, token, Hk):
    """[T, H, D] as [B, Hk, H / Hk, L, D] in fp32."""
    B, L = token.shape
    _, H, D = x.shape
    return x.float()[token].view(B, L, Hk, H // Hk, D).permute(0, 2, 3, 1, 4)


def _scores(s, token, there):
    case = s["case"]
    q, k = _padded(s["q"], token, case["Hk"]), _padded(s["k"], token, case["Hk"])
    z = (q @ k.transpose(-1, -2)) * (1 / math.sqrt(case["D"]))
    mask = there[:, None, None, None, :]
    if case["causal"]:
        at = torch.arange(case["L"], device=z.device)
        mask = mask & (at[None, :] <= at[:, None])
    return q, k, z.masked_fill_(~mask, -math.inf)


def _attention(s):
    token, there, b, at = _places(s)
    _, _, z = _scores(s, token, there)
    top = z.amax(-1, keepdim=True)
    e = (z - top).exp()
    total = e.sum(-1, keepdim=True)
    out = (e / total) @ _padded(s["v"], token, s["case"]["Hk"])
    lse = (top + total.log())[..., 0]
    T, Hq, D = s["q"].shape
    return out.permute(0, 3, 1, 2, 4)[b, at].reshape(T, Hq, D).to(s["q"].dtype), lse.permute(0, 3, 1, 2)[b, at].reshape(T, Hq)


def _attention_bwd(s):
    case = s["case"]
    T, Hq, D = s["q"].shape
    Hk, scale = case["Hk"], 1 / math.sqrt(case["D"])
    token, there, b, at = _places(s)
    q, k, z = _scores(s, token, there)
    here = there[:, None, None, :, None]
    p = torch.where(here, (z - _padded(s["lse"][..., None], token, Hk)).exp(), 0.0)
    del z
    v = _padded(s["v"], token, Hk)
    g = torch.where(here, _padded(s["g_out"], token, Hk), 0.0)
    delta = (g * _padded(s["out"], token, Hk)).sum(-1, keepdim=True)
    g_v = (p.transpose(-1, -2) @ g).sum(2)
    ds = p * (g @ v.transpose(-1, -2) - delta)
    del p
    g_q = scale * (ds @ k)
    g_k = scale * (ds.transpose(-1, -2) @ q).sum(2)
    g_q = g_q.permute(0, 3, 1, 2, 4)[b, at].reshape(T, Hq, D)
    return torch.cat([g_q] + [x.permute(0, 2, 1, 3)[b, at] for x in (g_k, g_v)], 1).to(s["q"].dtype)


M0, M1, W0, W1, LOW = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85, 0xFFFFFFFF
STREAM = 4  # of the generator's counter: dropout


def _threshold(p):
    return int(round(p * 65536))


def _dropout(s):
    """Philox4x32-10 (its ten rounds are a loop over whole tensors): 16 bits for each element."""
    case, x = s["case"], s["x"].float()
    n = x.numel()
    c0 = torch.arange((n + 7) // 8, device=x.device)
    c1, c2, c3 = torch.zeros_like(c0), torch.full_like(c0, STREAM), torch.zeros_like(c0)
    k0, k1 = s["seed"] & LOW, s["seed"] >> 32
    for r in range(10):
        a, b = c0 * M0, c2 * M1  # mod 2^64
        c0, c1, c2, c3 = (b >> 32 & LOW) ^ c1 ^ k0, b & LOW, (a >> 32 & LOW) ^ c3 ^ k1, a & LOW
        k0, k1 = k0 + W0 & LOW, k1 + W1 & LOW
    words = torch.stack([c0, c1, c2, c3], 1)
    bits = torch.stack([words & 0xFFFF, words >> 16], 2).view(-1)[:n].view(x.shape)
    drop = _threshold(case["p"])
    y = torch.where(bits >= drop, x * (65536 / (65536 - drop)), 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[case["y"]])


def _pairs(case):
    """Query-key pairs that the mask leaves, of one head."""
    return sum(n * (n + 1) // 2 if case["causal"] else n * n for n in _lengths(case))


def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "dropout":
        n = case["T"] * case["C"]
        return {"bytes": n * (size[case["x"]] + size[case["y"]] * (2 if case["residual"] else 1)), "flops": 3 * n}
    T, Hq, Hk, D, x = sum(_lengths(case)), case["Hq"], case["Hk"], case["D"], size[case["x"]]
    if case["op"] == "attention":
        return {"bytes": T * (2 * Hq + 2 * Hk) * D * x + 4 * T * Hq, "flops": 4 * _pairs(case) * Hq * D}
    return {"bytes": T * (3 * Hq + 4 * Hk) * D * x + T * Hq * (D * size[case["gout"]] + 4), "flops": 10 * _pairs(case) * Hq * D}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        return _exact_dropout(s)
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    group, ends = Hq // Hk, np.cumsum(_lengths(case))
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    first, second, third = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    lses = torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    for n, end in zip(_lengths(case), ends):
        rows = slice(int(end) - n, int(end))
        upper = torch.ones(n, n, dtype=torch.bool, device=q.device).triu_(1) if case["causal"] else None
        for h in range(Hk):
            heads = slice(h * group, (h + 1) * group)
            a = torch.einsum("ihd,jd->hij", q[rows, heads], k[rows, h]).mul_(D ** -0.5)
            if upper is not None:
                a.masked_fill_(upper, -torch.inf)
            if case["op"] == "attention":
                lses[rows, heads] = torch.logsumexp(a, -1).t()
                first[rows, heads] = torch.einsum("hij,jd->ihd", torch.softmax(a, -1), v[rows, h])
                continue
            a = a.sub_(s["lse"][rows, heads].double().t()[..., None]).exp_()
            g = s["g_out"][rows, heads].double()
            third[rows, h] = torch.einsum("hij,ihd->jd", a, g)
            lost = torch.einsum("ihd,ihd->hi", g, s["out"][rows, heads].double())
            a.mul_(torch.einsum("ihd,jd->hij", g, v[rows, h]).sub_(lost[..., None])).mul_(D ** -0.5)
            first[rows, heads] = torch.einsum("hij,jd->ihd", a, k[rows, h])
            second[rows, h] = torch.einsum("hij,ihd->jd", a, q[rows, heads])
    return (first, lses) if case["op"] == "attention" else torch.cat([first, second, third], 1)


def _exact_dropout(s):
    case, n = s["case"], s["x"].numel()
    u = np.uint64
    low = u(LOW)
    block = np.arange((n + 7) // 8, dtype=u)
    ctr = [block & low, block >> u(32), np.full_like(block, STREAM), np.zeros_like(block)]
    for r in range(10):
        keys = [u((key + r * step) & LOW) for key, step in ((s["seed"] & LOW, W0), (s["seed"] >> 32, W1))]
        left, right = u(M0) * ctr[0], u(M1) * ctr[2]
        ctr = [(right >> u(32)) ^ ctr[1] ^ keys[0], right & low, (left >> u(32)) ^ ctr[3] ^ keys[1], left & low]
    draws = np.empty((len(block), 8), np.uint16)
    for i in range(8):
        draws[:, i] = (ctr[i // 2] >> u(16 * (i % 2))) & u(0xFFFF)
    kept = torch.from_numpy(draws.reshape(-1)[:n].astype(np.int32) >= _threshold(case["p"])).to(s["x"].device).view(s["x"].shape)
    y = kept * s["x"].double() * 65536 / (65536 - _threshold(case["p"]))
    return y if s["residual"] is None else y + s["residual"].double()
