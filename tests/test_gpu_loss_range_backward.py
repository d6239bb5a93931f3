"""The gradients of the loss over the whole range of logits, against the formula in 64 bits with
lse as the forward pass left it.  The logits are products of two numbers each, exact in fp32.

Bounds, u = 2^-24, d = l - lse (exact where it is small, else off by u |d|), w the unit roundoff
of the 16-bit type:
  p      off by (1 + |d|) 2^-22 of itself: the exponential's own 2^-22, an argument rounded three
         times (d, its factor, their product)
  g      that, one subtraction, and w |g| of its rounding (up to 128 rows, in two values, w^2 |g|;
         f16: at least half the least value over 2^14), times |dloss|
  dx, dW the errors of g against |W|, |x|; 2^-23 (n + 16) sum|g W| of the sums; w of the result's
         rounding
"""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_embedding import I64
from test_gpu_loss_range import LARGER, SIZES, forward, one_column
from test_gpu_operators import BF, H, LEAST, T, U, close, out_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    assert mm.mm_operator_status() == mm.MM_OK, mm.mm_last_error()


@pytest.mark.parametrize("t,size", [(t, s) for t in (BF, H) for s in SIZES] + [(BF, s) for s in LARGER])
@pytest.mark.parametrize("rows,cols,vocab,offset", [(20, 8, 1000, 0), (300, 40, 1000, 0), (60, 72, 257, 1), (1, 1500, 20000, 0),
                                                    (129, 600, 5000, 0)])
def test_largest_logits(rows, cols, vocab, offset, t, size):
    """n tokens tie at the top; the first half's targets are one of them, the others' are not."""
    torch = T()
    x, w = one_column(rows, cols, vocab, t, size[:2], offset)
    c = cols // 2
    at = sorted({0, vocab // 3, vocab - 1})
    dloss = torch.full((rows,), 0.25, device="cuda")
    for n in range(1, len(at) + 1):
        w[at[n - 1], c] = size[2]
        targets = torch.full((rows,), at[n - 1], device="cuda")
        targets[rows // 2:] = 1
        _, lse = forward(x, w, targets)
        dx, dx_around = out_rows(rows, cols, t)
        dw, dw_around = out_rows(vocab, cols, t)
        mm.check(mm.mm_cross_entropy_backward(x, w, targets, lse, dloss, dx, dw, rows, cols, vocab, x.stride(0),
                                              w.stride(0), cols, cols, (t, I64, t)))
        l = x[:, c].double()[:, None] * w[:, c].double()[None]
        d = l - lse.double()[:, None]
        p = torch.exp(d)
        g = p.clone()
        g[torch.arange(rows), targets] -= 1
        off = p * (1 + d.abs().clamp(max=2000)) * 2.0 ** -22  # (p is 0 below)
        off += ((U[t] if rows > 128 else U[t] ** 2) + 2.0 ** -22) * g.abs()
        if t == H:
            off += LEAST[H] / 2 / 2 ** 14
        g, off = g * 0.25, off * 0.25
        for got, want, size_, miss, terms in (
                (dx, g @ w[:, c].double(), g.abs() @ w[:, c].double().abs(), off @ w[:, c].double().abs(), vocab),
                (dw, g.t() @ x[:, c].double(), g.abs().t() @ x[:, c].double().abs(), off.t() @ x[:, c].double().abs(), rows)):
            if t == H:  # 65504 is its largest number: 65520 and more round to infinity
                want = torch.where(want.abs() >= 65520, want.sign() * float("inf"), want)
            close(got[:, c], want, miss + 2.0 ** -23 * (terms + 16) * size_ + U[t] * (want.abs() + miss) + LEAST[t] / 2)
            got[:, c] = 0
            assert not bool(got.any())
        if n == 1 and not bool(p[0, 1]):  # a share of exactly 1
            assert bool((g[:rows // 2] == 0).all())
        dx_around()
        dw_around()


@pytest.mark.parametrize("rows", [20, 300])
@pytest.mark.parametrize("size", [1e4, 1e6, 1e8, 3e9, 1e12])
def test_the_only_token(rows, size):
    """A vocabulary of one: its share is 1, so there is no gradient, whatever the logit."""
    torch = T()
    root = size ** 0.5
    x, w = one_column(rows, 64, 1, BF, (root, root))
    x[1::2] *= -1
    targets = torch.zeros(rows, dtype=torch.int64, device="cuda")
    loss, lse = forward(x, w, targets)
    dx, dw = torch.ones_like(x), torch.ones_like(w)
    mm.check(mm.mm_cross_entropy_backward(x, w, targets, lse, None, dx, dw, rows, 64, 1, 64, 64, 64, 64, (BF, I64, BF)))
    assert not bool(loss.any()) and not bool(dx.any()) and not bool(dw.any())
