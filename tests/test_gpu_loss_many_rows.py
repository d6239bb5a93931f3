"""dW summed over many rows, all of one sign, so that what a sum over K loses adds up.

W is zero, so every share is exp(-lse), off by 2^-22 (1 + lse); g is the same for every row of a
token, exact in 16 bits but for the target's in bf16 (w, its unit roundoff).  A sum that truncates
falls short by at most 2^-23 of the partial sum at each step of 16 rows, and partial sums are half
the last one in the mean: over n rows n / 16 2^-24 of the sum.  Chains are 8192 rows at most; their
own additions are off by 2^-24 each.
"""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_embedding import I64
from test_gpu_loss_range import forward
from test_gpu_operators import BF, H, T, U, generator, out_rows, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1024, 1025, 9000, 65_536, 300_000, 1_048_653])
@pytest.mark.parametrize("cols,vocab,pad", [(64, 512, 0), (65, 128, 0), (8, 1024, 8), (200, 256, 3)])
@pytest.mark.parametrize("t", [BF, H])
def test_sums_over_rows(rows, cols, vocab, pad, t):
    torch = T()
    g = generator(rows + cols)
    x, w = rows_of(g, rows, cols, t), rows_of(g, vocab, cols, t)
    x.copy_(1 + torch.randint(0, 128, (rows, cols), generator=g, device="cuda") / 128)
    w.zero_()
    targets = torch.zeros(rows, dtype=torch.int64, device="cuda")
    none = torch.rand(rows, generator=g, device="cuda") < 0.1
    targets[none] = -100
    x[none] = float("nan")
    loss, lse = forward(x, w, targets)
    scale = 2.0 ** -6
    dloss = torch.full((rows,), scale, device="cuda")
    dx, _ = out_rows(rows, cols, t)
    dw, around = out_rows(vocab, cols, t, pad)
    mm.check(mm.mm_cross_entropy_backward(x, w, targets, lse, dloss, dx, dw, rows, cols, vocab, cols, cols, cols,
                                          dw.stride(0), (t, I64, t)))
    p = torch.exp(-lse[~none][0].double())
    sums = torch.zeros(cols, dtype=torch.float64, device="cuda")
    for r in range(0, rows, 1 << 18):
        sums += torch.where(none[r:r + (1 << 18), None], 0, x[r:r + (1 << 18)]).double().sum(0)
    want = (p * scale * sums).expand(vocab, cols).clone()
    want[0] = (p - 1) * scale * sums
    chain = min(rows, 8192) / 16 * 2.0 ** -24
    bound = want.abs() * (U[t] + 2.0 ** -22 * 8 + chain + 200 * 2.0 ** -24)
    bound[0] += want[0].abs() * U[t]
    bad = (dw.double() - want).abs() > bound
    assert not bool(bad.any()), ((dw.double() - want) / want).abs().max().item()
    around()
    assert not bool(dx.any())  # (times W)
