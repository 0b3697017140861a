"""Trains a small draft head with the library's losses.

A drafter predicts the next K tokens of every context from one hidden state; a
frozen target model supplies labels and its top logits.  Each step runs

* the cross entropy of the head against the target's sampled tokens
  (``linear_cross_entropy_fwd_bwd``: no logits are kept),
* every other step instead the distillation from the target's top logits
  through the head (``linear_topk_distill_fwd_bwd``),

and applies plain gradient steps to the hidden states' producer and to the
head.  Afterwards the draft's logits are formed once, their divergence from the
target is measured with ``topk_distill`` (the target's remaining mass as one
more token) and the expected accepted length with ``overlap``.

    python examples/train_draft_head.py [--steps 200]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sampling_spec_verify_gb300 as ssv  # noqa: E402


def train(steps=200, B=64, K=4, V=8192, H=256, k=32, lr=0.05, seed=0, device="cuda"):
    """Returns (first loss, last loss, divergence before, after, accepted length before, after)."""
    g = torch.Generator(device=device).manual_seed(seed)
    N = B * K
    rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    feats = rand(N, H)                                # what the drafter sees of each position
    target = 2.0 * (feats @ rand(H, V)) / H ** 0.5    # the target's logits
    p = torch.softmax(target, dim=1)
    vals, ids = torch.topk(target, k, dim=1)
    ids = ids.to(torch.int32)
    lse = torch.logsumexp(target, dim=1)
    decay = 0.8 ** (torch.arange(N, device=device) % K).float()   # later positions count less

    body = 0.2 * rand(H, H)
    head = 0.2 * rand(V, H) / H ** 0.5
    status = torch.zeros(1, dtype=torch.int32, device=device)

    def evaluate():
        z = (feats @ body).bfloat16() @ head.bfloat16().t()
        kl = ssv.topk_distill(z, ids, vals, teacher_lse=lse)
        ov = ssv.overlap(target.bfloat16().view(B, K, V), z.view(B, K, V), 1.0)
        return float(kl.loss), float(ov.expected_accepted.mean())

    before = evaluate()
    first = last = None
    for step in range(steps):
        x = (feats @ body).bfloat16()
        w = head.bfloat16()
        if step % 2 == 0:
            labels = torch.multinomial(p, 1, generator=g)[:, 0].to(torch.int32)
            o = ssv.linear_cross_entropy_fwd_bwd(x, w, labels, row_weight=decay, grad_dtype=torch.float32)
        else:
            o = ssv.linear_topk_distill_fwd_bwd(x, w, ids, vals, row_weight=decay, grad_dtype=torch.float32)
            last = float(o.loss)
            first = last if first is None else first
        status |= o.status
        body -= lr * (feats.t() @ o.grad_hidden)
        head -= 10.0 * lr * o.grad_weight
    after = evaluate()
    assert int(status) == 0
    return first, last, before[0], after[0], before[1], after[1]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    first, last, kl0, kl1, tau0, tau1 = train(steps=ap.parse_args().steps)
    print(f"distillation loss {first:.3f} -> {last:.3f}; KL of the target's top tokens {kl0:.3f} -> {kl1:.3f}; "
          f"expected accepted length {tau0:.3f} -> {tau1:.3f} of 4")
