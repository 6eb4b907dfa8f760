"""A policy trained by reward: its backward pass in libhlq, down to the embedding.

The policy reads one token and answers with another: embedding, layer norm,
vocabulary projection.  It is rewarded for the answer `table[token]`.  Each
step samples answers, takes their log-probabilities, and makes two updates of
the clipped policy loss: logits -> loss and gradient of the logits (over the
logits) -> both gradients of the projection (HLQ: int4 / int8) -> layer norm
backward -> norm and clipping of all gradients -> plain gradient descent.

    python examples/policy_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import hadamard_precision_backprop_gb300 as hlq  # noqa: E402


def main(steps=60, tokens=2048, width=256, vocab=512, kinds=64, lr=1.0, seed=0, say=print):
    """Returns the mean reward of each step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    emb = randn(kinds, width)
    norm_w, norm_b = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
    proj = 0.02 * randn(vocab, width)
    params = [emb, norm_w, norm_b, proj]
    table = torch.randint(vocab, (kinds,), generator=gen, device="cuda") % 16   # 16 right answers
    rewards = []

    def forward(tok):
        x = emb[tok].bfloat16()
        y, mean, rstd = hlq.hlq_layer_norm(x, norm_w, norm_b)
        return x, y, mean, rstd, y @ proj.bfloat16().t()

    for step in range(steps):
        tok = torch.randint(kinds, (tokens,), generator=gen, device="cuda")
        logits = forward(tok)[-1]
        answers = torch.multinomial(torch.softmax(logits.float(), 1), 1, generator=gen)[:, 0]
        old, _ = hlq.hlq_token_logprobs(logits, answers)
        reward = (answers == table[tok]).float()
        advantage = (reward - reward.mean()) / (reward.std() + 1e-3)
        weight = torch.full((tokens,), 1.0 / tokens, device="cuda")
        for _ in range(2):
            x, y, mean, rstd, logits = forward(tok)
            xbar, scale = hlq.hlq_compress_activation(y)
            stats, _, g_logits = hlq.hlq_policy_loss(logits, answers, old, advantage, weight,
                                                     ref_logp=old, kl_coef=0.01, out=logits)
            g_y, g_proj = hlq.hlq_linear_backward(g_logits, proj.bfloat16(), xbar, scale,
                                                  seed=step)
            g_x, g_w, g_b = hlq.hlq_layer_norm_backward(g_y, x, mean, rstd, norm_w,
                                                        out_dtype=torch.float32)
            g_emb = torch.zeros_like(emb).index_add_(0, tok, g_x)
            grads = [g_emb, g_w, g_b, g_proj]
            hlq.hlq_clip_grad_norm(grads, 1.0)
            for p, g in zip(params, grads):
                p.sub_(lr * g)
        rewards.append(float(reward.mean()))
        if step % 10 == 0 or step == steps - 1:
            say(f"step {step}: reward {rewards[-1]:.3f}, loss {float(stats[0]):.4f}, "
                f"clipped {float(stats[3]):.3f}")
    return rewards


if __name__ == "__main__":
    main()
