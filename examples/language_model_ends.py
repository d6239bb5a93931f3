"""A training step around the ends of a language model with tied weights: the
matrix W that looks the tokens up also projects on the vocabulary.

    e     = sqrt(C) W[tokens]               embedding
    y     = norm(e)                         root-mean-square norm
    l     = mean over the positions that count of cross entropy(y . W^T, targets)
    dy, dW  from the loss;  de = norm'(dy);  dW += the embedding's gradient of de

What lies between the norm and the embedding in a model is left out.  Positions
whose target is -100 (prompts, padding) do not count; they cost next to nothing.

    python examples/language_model_ends.py --tokens 4096 --hidden 2048 --vocab 32000

prints how far each result is from the same computation in fp32 torch.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matmul_selection_gb300 as mm  # noqa: E402

EPS = 1e-6
BF16, F32, I64 = mm.MM_BF16, mm.MM_F32, mm.MM_I64


def train_step(w, weight, tokens, targets, stream=None):
    """(loss, dW, dweight) of a batch of tokens; w and weight in bf16."""
    (V, C), T, d = w.shape, tokens.numel(), w.device
    scale = C ** 0.5
    e, y, dy, de = (torch.empty(T, C, dtype=w.dtype, device=d) for _ in range(4))
    rstd, loss, lse = (torch.empty(T, device=d) for _ in range(3))
    dw, dweight = torch.empty_like(w), torch.empty_like(weight)
    bf, ends = (BF16, BF16, BF16), (BF16, I64, BF16)
    mm.check(mm.mm_embedding(w, tokens, e, T, C, V, C, C, ends, scale, stream))
    mm.check(mm.mm_rmsnorm(e, None, weight, None, y, None, rstd, T, C, C, 0, 0, C, bf, EPS, stream))
    mm.check(mm.mm_cross_entropy(y, w, targets, loss, lse, T, C, V, C, C, (BF16, I64, F32), stream))
    valid = (targets >= 0) & (targets < V)
    dloss = valid.float() / valid.sum().clamp_min(1)  # of the mean
    mm.check(mm.mm_cross_entropy_backward(y, w, targets, lse, dloss, dy, dw, T, C, V, C, C, C, C, ends, stream))
    mm.check(mm.mm_rmsnorm_backward(dy, None, e, weight, rstd, de, dweight, T, C, C, 0, C, C, bf, EPS, stream))
    # onto what the loss left, in place: only the rows of tokens that occur
    mm.check(mm.mm_embedding_backward(de, tokens, dw, dw, T, C, V, C, C, C, ends, scale, stream))
    return (loss * dloss).sum(), dw, dweight


def plain_train_step(w, weight, tokens, targets):
    w, weight = (t.float().requires_grad_() for t in (w, weight))
    e = w[tokens] * w.shape[1] ** 0.5
    y = e / (e.square().mean(1, keepdim=True) + EPS).sqrt() * weight
    loss = torch.nn.functional.cross_entropy(y @ w.t(), targets, ignore_index=-100)
    return (loss.detach(), *torch.autograd.grad(loss, (w, weight)))


def off(got, want):
    return ((got.float() - want.float()).norm() / want.float().norm()).item()


def run(tokens, hidden, vocab, seed=0):
    """{name: relative error} of a step."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = (torch.randn(vocab, hidden, generator=g, device="cuda") * hidden ** -0.5).bfloat16()
    weight = (1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).bfloat16()
    text = torch.randint(0, vocab, (tokens + 1,), generator=g, device="cuda")
    text[1:][torch.rand(tokens, generator=g, device="cuda") < 0.3] = text[0]  # one token often
    targets = text[1:].clone()
    targets[:tokens // 4] = -100  # the prompt
    got, want = (f(w, weight, text[:-1].contiguous(), targets) for f in (train_step, plain_train_step))
    mm.check(mm.mm_operator_status())
    return {name: off(a, b) for name, a, b in zip(("loss", "dW", "dweight"), got, want)}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args()
    for name, rel in run(a.tokens, a.hidden, a.vocab).items():
        print(f"{name:10s} relative error {rel:.2e}")


if __name__ == "__main__":
    main()
