"""A pre-norm pair of linear layers with quantised weights, and a training step
of its dense form: the operators of this library as a model uses them together.

Serving, for a batch of tokens (one to many):
    h, q, s = norm(x, residual)          e4m3 with one scale a token
    a       = (s q) . (sb B)^T           8-bit weights
    h, y    = norm(a, h)                 16-bit
    out     = y . W^T                    4-bit weights with group scales
Training, the first norm in front of a bf16 weight matrix:
    y = norm(x); out = y . V^T; dy = dout . V; dV = dout^T . y; dx, dw = norm'(dy)
where the three dense products are the library's autotuned ones.

    python examples/quantised_layer.py --tokens 16 --hidden 4096 --inner 8192

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
GROUP = 128
BF16, E4M3, F32 = mm.MM_BF16, mm.MM_E4M3, mm.MM_F32


def quantise_rows_e4m3(w):
    """Rows in e4m3 with one fp32 scale each."""
    scale = w.abs().amax(1).clamp_min(2.0 ** -126) / 448
    return (w / scale[:, None]).to(torch.float8_e4m3fn), scale


def quantise_groups_4bit(w, group=GROUP):
    """Codes 0..15 (zero point 8), two to a byte, with bf16 group scales."""
    n, k = w.shape
    g = w.view(n, k // group, group)
    scales = (g.abs().amax(2) / 7).clamp_min(1e-12).bfloat16()
    q = (g / scales.float()[:, :, None]).round().clamp(-8, 7).add(8).to(torch.uint8).view(n, k)
    return q[:, 0::2] | (q[:, 1::2] << 4), scales


def dequantise_4bit(codes, scales, group=GROUP):
    q = torch.stack([codes & 15, codes >> 4], 2).flatten(1).float() - 8
    return q * scales.float().repeat_interleave(group, 1)


class QuantisedLayers:
    """Weights in 8 and 4 bits, and the buffers of a step of at most `tokens`."""

    def __init__(self, up, down, norm1, norm2, tokens):
        self.b, self.sb = quantise_rows_e4m3(up)
        self.codes, self.scales = quantise_groups_4bit(down)
        self.norm1, self.norm2 = norm1, norm2
        self.inner, self.hidden = up.shape[0], up.shape[1]
        d, bf = up.device, torch.bfloat16
        self.q = torch.empty(tokens, self.hidden, dtype=torch.float8_e4m3fn, device=d)
        self.s = torch.empty(tokens, device=d)
        self.h = torch.empty(tokens, self.hidden, dtype=bf, device=d)
        self.a = torch.empty(tokens, self.inner, dtype=bf, device=d)
        self.y = torch.empty(tokens, self.inner, dtype=bf, device=d)
        self.out = torch.empty(tokens, down.shape[0], dtype=bf, device=d)

    def step(self, x, residual, stream=None):
        M, H, N = x.shape[0], self.hidden, self.inner
        O = self.out.shape[1]
        mm.check(mm.mm_rmsnorm(x, residual, self.norm1, self.h, self.q, self.s, None, M, H, H, H, H, H,
                               (BF16, BF16, E4M3), EPS, stream))
        mm.check(mm.mm_gemm_q8(self.q, self.b, self.s, self.sb, self.a, M, N, H, H, H, N,
                               (E4M3, E4M3, BF16), stream))
        mm.check(mm.mm_rmsnorm(self.a, None, self.norm2, None, self.y, None, None, M, N, N, 0, 0, N,
                               (BF16, BF16, BF16), EPS, stream))
        mm.check(mm.mm_gemm_w4(self.y, self.codes, self.scales, None, self.out, M, O, N, N, N,
                               self.scales.shape[1], O, GROUP, (BF16, BF16, BF16), stream))
        return self.h[:M], self.out[:M]

    def plain(self, x, residual):
        """The same in fp32 torch, from the quantised weights."""
        h = x.float() + residual.float()
        y = h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * self.norm1.float()
        a = y @ (self.b.float() * self.sb[:, None]).t()
        y = a / (a.square().mean(1, keepdim=True) + EPS).sqrt() * self.norm2.float()
        return h, y @ dequantise_4bit(self.codes, self.scales).t()


def train_step(x, weight, v, dout, stream=None):
    """Forward and backward of out = norm(x) . v^T in bf16: (out, dx, dweight, dv)."""
    (M, H), N = x.shape, v.shape[0]
    bf = (BF16, BF16, BF16)
    y, dy, dx = (torch.empty_like(x) for _ in range(3))
    rstd = torch.empty(M, device=x.device)
    out, dv = torch.empty_like(dout), torch.empty_like(v)
    dweight = torch.empty_like(weight)
    mm.check(mm.mm_rmsnorm(x, None, weight, None, y, None, rstd, M, H, H, 0, 0, H, bf, EPS, stream))
    mm.check(mm.mm_autotune_execute(y, v, out, M, N, H, H, H, N, bf, "NT", None, stream))
    mm.check(mm.mm_autotune_execute(dout, v, dy, M, H, N, N, H, H, bf, "NN", None, stream))
    mm.check(mm.mm_autotune_execute(dout, y, dv, N, H, M, N, H, H, bf, "TN", None, stream))
    mm.check(mm.mm_rmsnorm_backward(dy, None, x, weight, rstd, dx, dweight, M, H, H, 0, H, H, bf, EPS, stream))
    return out, dx, dweight, dv


def plain_train_step(x, weight, v, dout):
    x, weight, v = (t.float().requires_grad_() for t in (x, weight, v))
    out = (x / (x.square().mean(1, keepdim=True) + EPS).sqrt() * weight) @ v.t()
    return (out.detach(), *torch.autograd.grad(out, (x, weight, v), dout.float()))


def off(got, want):
    return ((got.float() - want.float()).norm() / want.float().norm()).item()


def run(tokens, hidden, inner, seed=0):
    """{name: relative error} of a serving and a training step."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    layers = QuantisedLayers(normal(inner, hidden, scale=hidden ** -0.5), normal(hidden, inner, scale=inner ** -0.5),
                             (1 + normal(hidden, scale=0.1)).bfloat16(), (1 + normal(inner, scale=0.1)).bfloat16(),
                             tokens)
    x, residual = normal(tokens, hidden).bfloat16(), normal(tokens, hidden, scale=2.0).bfloat16()
    h, out = layers.step(x, residual)
    want_h, want = layers.plain(x, residual)
    result = {"residual stream": off(h, want_h), "two quantised layers": off(out, want)}
    weight, v = layers.norm1, normal(inner, hidden, scale=hidden ** -0.5).bfloat16()
    dout = normal(tokens, inner).bfloat16()
    names = ("out", "dx", "dweight", "dv")
    for name, got, plain in zip(names, train_step(x, weight, v, dout), plain_train_step(x, weight, v, dout)):
        result["training " + name] = off(got, plain)
    mm.check(mm.mm_operator_status())
    return result


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=8192)
    a = ap.parse_args()
    for name, rel in run(a.tokens, a.hidden, a.inner).items():
        print(f"{name:24s} relative error {rel:.2e}")


if __name__ == "__main__":
    main()
