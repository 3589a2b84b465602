#!/usr/bin/env python3
"""A 2:4-sparse layer under a vocabulary head, from training to 4-bit decoding.

    python examples/train_and_serve.py [--steps 60] [--vocab 2000] [--width 512]

The toy task is a fixed random map from each word to the next.  A word's embedding (fixed) goes
through one residual layer kept 2:4 by SR-STE and a dense head:

    hidden = x + gelu(prune(W1) x + b1),   loss = cross entropy of the logits W2 hidden at the next word

Training, each step: mask and compress W1 (compress), the sparse product with its bias, activation
and residual (spmm_act), loss and gradient without storing the logits (xent, xent_grad), the layer's
gradient (spmm_act_grad), refined where the mask prunes (srste_grad), all of them clipped together
(clip_grads), and for both matrices the orthogonalised momentum as the update (orthogonalize).

Serving: W1's kept values and W2 in 4 bits with a scale for 64 columns (quantize), and one token
at a time through both (matvec_act by the layer's 2:4 metadata, matvec), a penalty on the word that was
just said (adjust_logits).
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
    """(W1 pruned, b1, W2, embeddings, next words, losses)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    embed = randn(width, vocab).to(torch.bfloat16)         # a column a word
    follow = torch.randperm(vocab, generator=gen, device="cuda")
    weights = [randn(width, width) / width ** 0.5, randn(vocab, width) / width ** 0.5]
    bias = torch.zeros(width, device="cuda")
    momentum = [torch.zeros_like(w) for w in weights]
    losses = []
    for step in range(steps):
        words = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
        x = embed[:, words].contiguous()
        w1, w2 = (w.to(torch.bfloat16) for w in weights)
        values, meta = nm.compress(w1, 2, 4, layout="blocked")
        hidden, z = nm.spmm_act(values, meta, x, bias=bias, act="gelu", residual=x, keep=True,
                                layout="blocked", rows=width)
        target = follow[words]
        loss, lse = nm.xent(w2, hidden, target)
        gout = torch.full((tokens,), 1.0 / tokens, device="cuda")
        g2, dhidden = nm.xent_grad(w2, hidden, target, lse, gout)
        g1, gb = nm.spmm_act_grad(None, None, x, dhidden, z, act="gelu", want=("dW", "dbias"))
        nm.srste_grad(w1, g1, 2, 4, out=g1)
        nm.clip_grads([g1, g2, gb], 1.0)
        rate = 0.06 * (1 - step / steps)
        for w, m, g in zip(weights, momentum, (g1, g2)):
            m.mul_(0.9).add_(g.float())
            update = nm.orthogonalize(m.to(torch.bfloat16)).float()
            w.sub_(rate * max(1.0, w.shape[0] / w.shape[1]) ** 0.5 * update)
        bias.sub_(rate * gb)
        losses.append(float(loss.mean()))
        if report and (step % 10 == 0 or step + 1 == steps):
            report(f"step {step:3d}  loss {losses[-1]:.3f}")
    w1, w2 = (w.to(torch.bfloat16) for w in weights)
    return nm.prune(w1, 2, 4), bias, w2, embed, follow, losses


def serve(w1: torch.Tensor, bias: torch.Tensor, w2: torch.Tensor, embed: torch.Tensor, words,
          group: int = 64):
    """The next word after each of `words`, one token at a time from the 4-bit matrices."""
    width, vocab = w1.shape[0], w2.shape[0]
    values, meta = nm.compress(w1, 2, 4, layout="blocked")
    sparse = nm.quantize(values, group, layout="blocked", rows=width)
    head = nm.quantize(w2, group)
    starts = torch.tensor([0, 1], device="cuda")
    presence = torch.ones(1, device="cuda")
    said = torch.tensor(words, device="cuda")
    answers = []
    for i, word in enumerate(words):
        x = embed[:, word:word + 1].contiguous()
        hidden = nm.matvec_act(*sparse, x, group, rows=width, meta=meta, bias=bias, act="gelu",
                               residual=x)
        logits = nm.matvec(*head, hidden, group, rows=vocab, out_dtype=torch.float32)
        nm.adjust_logits(logits, said[i:i + 1], starts, presence=presence, out=logits)
        answers.append(int(logits.argmax()))
    return answers


def main(argv=None) -> dict:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--vocab", type=int, default=2000)
    p.add_argument("--width", type=int, default=512)   # a multiple of 64
    p.add_argument("--tokens", type=int, default=1024)
    a = p.parse_args(argv)
    w1, bias, w2, embed, follow, losses = train(a.steps, a.vocab, a.width, a.tokens)
    words = list(range(0, a.vocab, max(1, a.vocab // 100)))
    x = embed[:, words].float()
    hidden = x + torch.nn.functional.gelu(w1.float() @ x + bias[:, None])
    full = (w2.float() @ hidden).argmax(0).tolist()
    four = serve(w1, bias, w2, embed, words)
    truth = follow[words].tolist()
    share = [sum(x == y for x, y in zip(s, truth)) / len(words) for s in (full, four)]
    print(f"next words right: {share[0]:.2f} with the trained weights, {share[1]:.2f} in 4 bits "
          f"({len(words)} words, one token at a time)")
    return dict(losses=losses, right=share[0], right_4bit=share[1])


if __name__ == "__main__":
    main()
