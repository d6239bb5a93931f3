"""The loss over the whole range of logits, and with its mass in one token anywhere in the
vocabulary.  The logits are sums that fp32 holds exactly, so what is measured is what becomes
of them.

Bounds, u = 2^-24, n the tokens that tie for the largest logit, R the others' shares of it
(together), V tokens.  The largest share is exp(0) = 1 exactly.
  s      = n + R.  R: its terms are off by 2^-21 of themselves and, as differences of 12 and
           more stay below that share, by 2^-19 (their argument is rounded twice); added
           up among themselves by K u, where K = 48 + V / 2048 is the longest chain of additions
           (ten in each of four blocks of 32 columns, halves of a tile, two for each tile that a
           thread joins, five between threads): 2^-17 R in all.  Added to n: K u s, but never
           more than R, as n alone is exact
  log s  off by the relative error of s, and by 2 u |log s| of its own
  loss   = (m - l[y]) + log s: two roundings, 2 u |loss|
  lse    = m + log s: one, u |lse|
"""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_embedding import I64
from test_gpu_operators import BF, F, H, T, close, generator, rows_of

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    assert mm.mm_operator_status() == mm.MM_OK, mm.mm_last_error()


def chain(vocab):
    return 48 + vocab // 2048


def forward(x, w, targets, ti=I64):
    torch = T()
    rows, (vocab, cols) = x.shape[0], w.shape
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    t = BF if x.dtype == torch.bfloat16 else H
    mm.check(mm.mm_cross_entropy(x, w, targets, loss, lse, rows, cols, vocab, x.stride(0), w.stride(0), (t, ti, F)))
    return loss, lse


def one_column(rows, cols, vocab, t, values, offset=0):
    """x and W of which one column is not zero: logits are a product of two numbers each."""
    torch = T()
    x, w = rows_of(generator(0), rows, cols, t, offset=offset), rows_of(generator(1), vocab, cols, t)
    x.zero_()
    w.zero_()
    x[:, cols // 2] = values[0]
    w[:, cols // 2] = torch.tensor(values[1], device="cuda").to(w.dtype).expand(vocab)
    return x, w


# x, and W of most tokens and of those that tie for the largest logit
SIZES = [(1.0, 0.0, 12.0), (1.0, 0.0, 30.0), (2.0, 0.0, 30.0), (4.0, 0.0, 25.0), (100.0, 0.0, 100.0), (-1000.0, 0.0, -1000.0),
         (1.0, -240.0, -120.0), (-1000.0, 2000.0, 1000.0), (2.0 ** 14, 0.0, 2.0 ** 15), (2.0 ** 16 - 256, 64.0, 2.0 ** 15),
         (-2.0 ** 15, 2.0 ** 15, 2.0 ** 14)]
LARGER = [(2.0 ** 20, 0.0, 2.0 ** 20), (-2.0 ** 20, 2.0 ** 22, 2.0 ** 20), (1.5 * 2.0 ** 50, 2.0 ** 12, 2.0 ** 50),
          (-2.0 ** 60, 2.0 ** 64, 2.0 ** 61), (2.0 ** 63, -2.0 ** 63, 1.5 * 2.0 ** 63)]


@pytest.mark.parametrize("t,size", [(t, s) for t in (BF, H) for s in SIZES] + [(BF, s) for s in LARGER])
@pytest.mark.parametrize("rows,cols,vocab,offset", [(20, 8, 1000, 0), (300, 40, 1000, 0), (60, 72, 257, 1), (1, 1500, 20000, 0),
                                                    (129, 600, 5000, 0)])
def test_largest_logits(rows, cols, vocab, offset, t, size):
    """n tokens tie at the top, the others far below (or far enough to be counted: 12)."""
    torch = T()
    x, w = one_column(rows, cols, vocab, t, size[:2], offset)
    at = sorted({0, vocab // 3, vocab - 1})
    for n in range(1, len(at) + 1):
        w[at[n - 1], cols // 2] = size[2]
        top, rest = (torch.tensor(float(x[0, cols // 2])).double() * float(w[v, cols // 2]) for v in (at[0], 1))
        R = (vocab - n) * torch.exp(rest - top)
        s = n + R
        targets = torch.full((rows,), at[n - 1], device="cuda")
        targets[rows // 2:] = 1
        loss, lse = forward(x, w, targets)
        off = min(1.01 * R, R * 2.0 ** -17 + chain(vocab) * U32 * s) / s + 2 * U32 * torch.log(s)
        want = torch.log(s).expand(rows).clone()
        want[rows // 2:] += top - rest
        close(loss, want.cuda(), (off + 2 * U32 * want).cuda())
        want = top + torch.log(s)
        close(lse, want.expand(rows).cuda(), (off + U32 * want.abs()).item())


def test_no_bias_over_many_positions():
    """Logits of up to 127 that fp32 holds exactly, the target among the few largest: the mean of
    what the losses are off by is that of roundings, whichever way the largest logit lies."""
    torch = T()
    g = generator(3)
    rows, vocab = 4096, 512
    x = torch.zeros(rows, 64, device="cuda")
    x[torch.arange(rows), torch.randint(0, 64, (rows,), generator=g, device="cuda")] = 1
    w = torch.randint(-100, 101, (vocab, 64), generator=g, device="cuda").float()
    w[:8] = torch.randint(120, 128, (8, 64), generator=g, device="cuda").float()
    for sign in (1, -1):
        l = (x @ w.t()).double() * sign
        targets = torch.randint(0, 8, (rows,), generator=g, device="cuda") if sign > 0 else l.argmax(1)
        loss, lse = forward((x * sign).bfloat16(), w.bfloat16(), targets)
        want = torch.logsumexp(l, 1)
        # terms of 2^-21 and of arguments up to 10 (2^-20.5), additions, roundings of the results
        miss = 2.0 ** -20 + chain(vocab) * U32
        assert bool(((lse.double() - want).abs() <= miss + U32 * want).all())
        want = want - l.gather(1, targets[:, None])[:, 0]
        off = loss.double() - want
        assert bool((off.abs() <= miss + 3 * U32 * want).all())
        # Roundings to the nearest fall both ways; exponentials need not, at 2^-21 each (and
        # arguments that differ by one, whose share is a third, by 2^-23): log2(e) rounded to fp32
        # as the only factor had put all losses off by -1.5e-8 of the largest logit, -1.9e-6
        assert abs(off.mean().item()) <= 2.0 ** -21 + 2.0 ** -23


@pytest.mark.parametrize("rows,vocab", [(40, 70_001), (128, 32_000), (8192, 70_001), (2048, 131_072), (128, 1_100_000),
                                        (300, 5000)])
def test_one_token_holds_the_mass(rows, vocab):
    """W's rows are codes of 64 signs and x is the code of a token: its logit is 64, the others'
    less by dozens.  Every tile of the vocabulary holds some row's token, so a tile that is left
    out, added twice or whose target is looked for elsewhere shows in full."""
    torch = T()
    g = generator(rows + vocab)
    w = torch.randint(0, 2, (vocab, 64), generator=g, device="cuda").mul_(2).sub_(1).bfloat16()
    for turn in range(1 if rows > 1000 else 4):
        targets = torch.randperm(vocab, generator=g, device="cuda")[:rows]
        edge = torch.tensor([0, vocab - 1, vocab // 2, 127, 128, 255, 256, vocab - 2], device="cuda")[:rows]
        targets[:len(edge)] = edge
        x = w[targets]
        loss, lse = forward(x, w, targets)
        R = torch.empty(rows, dtype=torch.float64, device="cuda")
        for r in range(0, rows, max(1, (1 << 28) // vocab)):
            at = slice(r, r + max(1, (1 << 28) // vocab))
            l = (x[at].float() @ w.float().t()).double() - 64
            R[at] = l.exp().scatter_(1, targets[at, None], 0.0).sum(1)
        want = torch.log1p(R)
        off = torch.minimum(1.01 * R, R * 2.0 ** -17 + chain(vocab) * U32 * (1 + R)) + 4 * U32 * want
        close(loss, want, off)
        close(lse, 64 + want, off + 65 * U32)


@pytest.mark.parametrize("rows,vocab", [(20, 1000), (300, 700)])
@pytest.mark.parametrize("t", [BF, H])
def test_infinite_logits(rows, vocab, t):
    """-infinity has no share (as a target, an infinite loss), +infinity leaves its rows NaN."""
    torch = T()
    x, w = one_column(rows, 16, vocab, t, (1.0, 3.0))
    c, inf = 8, float("inf")
    w[5, c] = w[400:, c] = -inf
    targets = torch.full((rows,), 7, device="cuda")
    targets[1] = 5
    loss, lse = forward(x, w, targets)
    want = torch.full((rows,), 399.0, dtype=torch.float64, device="cuda").log()
    off = chain(vocab) * U32 + 4 * U32 * want
    close(lse, 3 + want, off + 9 * U32)
    want[1] = inf
    close(loss, want, off)
    x[2] = 0
    x[2, c] = -1.0  # (so that -infinity becomes +infinity)
    x[3] *= -0.0
    w[:, c] = torch.where(torch.isinf(w[:, c]), 1.0, w[:, c].float()).to(w.dtype)
    w[650, c] = -inf
    targets[1] = 7
    loss, lse = forward(x, w, targets)
    assert bool(torch.isnan(loss[2:4]).all()) and bool(torch.isnan(lse[2:4]).all())  # (0 times infinity: NaN)
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[2:4] = False
    assert bool(torch.isfinite(loss[rest]).all()) and bool(torch.isfinite(lse[rest]).all())
