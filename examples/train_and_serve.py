#!/usr/bin/env python3
"""A 2:4-sparse layer under a vocabulary head, from training to 4-bit decoding.

    python examples/train_and_serve.py [--steps 60] [--vocab 2000] [--width 512]

The toy task is a fixed random map from each word to the next.  A word's embedding (fixed) goes
through one layer kept 2:4 by SR-STE and a dense head:

    hidden = prune(W1) x,   loss = cross entropy of the logits W2 hidden at the next word

Training, each step: mask and compress W1 (compress), the sparse product (spmm), loss and gradient
without storing the logits (xent, xent_grad), the sparse-refined gradient (srste_grad), and for
both matrices the orthogonalised momentum as the update (orthogonalize).

Serving: W1's kept values and W2 in 4 bits with a scale for 64 columns (quantize), and one token
at a time through both (matvec), the sparse layer by its 2:4 metadata.
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import masking_sparse_gemm_amd as nm


def train(steps: int, vocab: int, width: int, tokens: int, seed: int = 0, report=print):
    """(W1 pruned, W2, embeddings, next words, losses)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    embed = randn(width, vocab).to(torch.bfloat16)         # a column a word
    follow = torch.randperm(vocab, generator=gen, device="cuda")
    weights = [randn(width, width) / width ** 0.5, randn(vocab, width) / width ** 0.5]
    momentum = [torch.zeros_like(w) for w in weights]
    losses = []
    for step in range(steps):
        words = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
        x = embed[:, words].contiguous()
        w1, w2 = (w.to(torch.bfloat16) for w in weights)
        values, meta = nm.compress(w1, 2, 4, layout="blocked")
        hidden = nm.spmm(values, meta, x, 2, 4, layout="blocked", rows=width)
        target = follow[words]
        loss, lse = nm.xent(w2, hidden, target)
        gout = torch.full((tokens,), 1.0 / tokens, device="cuda")
        g2, dhidden = nm.xent_grad(w2, hidden, target, lse, gout)
        g1 = nm.srste_grad(w1, (dhidden @ x.t()).contiguous(), 2, 4)
        rate = 0.06 * (1 - step / steps)
        for w, m, g in zip(weights, momentum, (g1, g2)):
            m.mul_(0.9).add_(g.float())
            update = nm.orthogonalize(m.to(torch.bfloat16)).float()
            w.sub_(rate * max(1.0, w.shape[0] / w.shape[1]) ** 0.5 * update)
        losses.append(float(loss.mean()))
        if report and (step % 10 == 0 or step + 1 == steps):
            report(f"step {step:3d}  loss {losses[-1]:.3f}")
    w1, w2 = (w.to(torch.bfloat16) for w in weights)
    return nm.prune(w1, 2, 4), w2, embed, follow, losses


def serve(w1: torch.Tensor, w2: torch.Tensor, embed: torch.Tensor, words, group: int = 64):
    """The next word after each of `words`, one token at a time from the 4-bit matrices."""
    width, vocab = w1.shape[0], w2.shape[0]
    values, meta = nm.compress(w1, 2, 4, layout="blocked")
    sparse = nm.quantize(values, group, layout="blocked", rows=width)
    head = nm.quantize(w2, group)
    answers = []
    for word in words:
        x = embed[:, word:word + 1].contiguous()
        hidden = nm.matvec(*sparse, x, group, rows=width, meta=meta)
        logits = nm.matvec(*head, hidden, group, rows=vocab, out_dtype=torch.float32)
        answers.append(int(logits.argmax()))
    return answers


def main(argv=None) -> dict:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--vocab", type=int, default=2000)
    p.add_argument("--width", type=int, default=512)   # a multiple of 64
    p.add_argument("--tokens", type=int, default=1024)
    a = p.parse_args(argv)
    w1, w2, embed, follow, losses = train(a.steps, a.vocab, a.width, a.tokens)
    words = list(range(0, a.vocab, max(1, a.vocab // 100)))
    full = (w2.float() @ (w1.float() @ embed[:, words].float())).argmax(0).tolist()
    four = serve(w1, w2, embed, words)
    truth = follow[words].tolist()
    share = [sum(x == y for x, y in zip(s, truth)) / len(words) for s in (full, four)]
    print(f"next words right: {share[0]:.2f} with the trained weights, {share[1]:.2f} in 4 bits "
          f"({len(words)} words, one token at a time)")
    return dict(losses=losses, right=share[0], right_4bit=share[1])


if __name__ == "__main__":
    main()
