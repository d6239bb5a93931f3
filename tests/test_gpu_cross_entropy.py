"""The loss over a vocabulary and its gradients against their formulas in 64 bits.

Bounds, with e = 2^-23 (twice an fp32 rounding: sums on tensor cores may
truncate), u the unit roundoff of the 16-bit type, C columns, V tokens:
  a logit    L = e (C + 16) max_v sum|x W[v]|
  lse        L + e (V + 64 + 2 max|l|): V terms summed in fp32, exponentials of
             2^-22 whose arguments, up to 2 max|l| log2(e), round in fp32
             (natural logarithm: relative errors of the sum are absolute here),
             and its own rounding to fp32, e |lse|
  p          relative 2 L + e (8 + 4 max|l|): the exponential of a logit less lse,
             lse taken as given
  g          that on p, and u |g| of its rounding (up to 128 rows, where it is held in
             two values, u^2 |g|: the second is at most u |g| and off by u of itself;
             f16: and half the least value over 2^14, times the largest |dloss|)
  dx, dW     the errors of g against |W|, |x|; e (n + 16) sum|g W| of the sums;
             u of the result's rounding
"""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_embedding import I32, I64, tokens_of
from test_gpu_operators import BF, F, H, LEAST, T, U, close, generator, out_rows, rows_of

pytestmark = pytest.mark.gpu

E = 2.0 ** -23


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    assert mm.mm_operator_status() == mm.MM_OK, mm.mm_last_error()


class Problem:
    def __init__(self, rows, cols, vocab, t=BF, ti=I64, none=0.2, pads=(0, 0), offsets=(0, 0), size=2.0, seed=0,
                 dloss="weights"):
        torch = T()
        g = self.g = generator(rows * 7 + cols * 3 + vocab + seed)
        self.rows, self.cols, self.vocab, self.t, self.ti = rows, cols, vocab, t, ti
        self.x = rows_of(g, rows, cols, t, pads[0], offset=offsets[0])
        self.w = rows_of(g, vocab, cols, t, pads[1], size / cols ** 0.5, offsets[1])
        self.targets = tokens_of(g, rows, vocab, ti, none)
        self.ok = (self.targets.long() >= 0) & (self.targets.long() < vocab)
        self.x[~self.ok] = float("nan")  # never read
        self.dloss = torch.randn(rows, generator=g, device="cuda") * 0.5 if dloss == "weights" else None
        self.work()

    def work(self):
        torch = T()
        ok, n = self.ok, self.targets.long()
        x, w = torch.where(ok[:, None], self.x, 0).double(), self.w.double()
        self.l = x @ w.t()
        self.l_size = x.abs() @ w.abs().t()
        self.want_lse = torch.where(ok, torch.logsumexp(self.l, 1), 0.0)
        at = torch.where(ok, n, 0)[:, None]
        self.hit = self.l.gather(1, at)[:, 0]
        self.want_loss = torch.where(ok, self.want_lse - self.hit, 0.0)
        self.L = E * (self.cols + 16) * self.l_size.amax(1)
        self.top = self.l.abs().amax(1)

    def forward(self, stream=None, lse=True):
        torch = T()
        loss = torch.full((self.rows + 8,), 77.0, device="cuda")
        got_lse = torch.full((self.rows + 8,), 77.0, device="cuda") if lse else None
        mm.check(mm.mm_cross_entropy(self.x, self.w, self.targets, loss, got_lse, self.rows, self.cols, self.vocab,
                                     self.x.stride(0), self.w.stride(0), (self.t, self.ti, F), stream))
        return loss, got_lse

    def check_forward(self, loss, lse):
        torch = T()
        bound = self.L + E * (self.vocab + 64 + 2 * self.top)
        for got, want, own in ((lse, self.want_lse, bound), (loss, self.want_loss, bound + self.L)):
            if got is None:
                continue
            assert bool((got[self.rows:] == 77).all())
            close(got[:self.rows], want, own + E * want.abs())
            assert bool((got[:self.rows][~self.ok] == 0).all())

    def backward(self, dx=True, dw=True, pads=(0, 0), offsets=(0, 0), lse=None, stream=None):
        lse = self.want_lse.float() if lse is None else lse
        self.lse = lse[:self.rows]
        dx = out_rows(self.rows, self.cols, self.t, pads[0], offsets[0]) if dx else (None, None)
        dw = out_rows(self.vocab, self.cols, self.t, pads[1], offsets[1]) if dw else (None, None)
        mm.check(mm.mm_cross_entropy_backward(
            self.x, self.w, self.targets, lse, self.dloss, dx[0], dw[0], self.rows, self.cols, self.vocab,
            self.x.stride(0), self.w.stride(0), dx[0].stride(0) if dx[0] is not None else 0,
            dw[0].stride(0) if dw[0] is not None else 0, (self.t, self.ti, self.t), stream))
        return dx, dw

    def check_backward(self, dx, dw):
        torch = T()
        u, ok = U[self.t], self.ok[:, None]
        x, w = torch.where(ok, self.x, 0).double(), self.w.double()
        d = self.dloss.double()[:, None] if self.dloss is not None else torch.ones(self.rows, 1, device="cuda").double()
        d = torch.where(ok, d, 0.0)
        p = torch.exp(self.l - self.lse.double()[:, None])
        rel = (2 * self.L + E * (8 + 4 * self.top))[:, None]
        g = p.clone()
        at = torch.where(ok, self.targets.long()[:, None], 0)
        g.scatter_(1, at, g.gather(1, at) - 1)
        g = g * d
        off = rel * p * d.abs() * (1 + u) + ((u if self.rows > 128 else u * u) + 4 * E) * g.abs()
        if self.t == H:
            off = torch.where(ok, off + LEAST[H] / 2 / 2 ** 14 * d.abs().max(), 0.0)
        for got, want, size, miss, n in ((dx, g @ w, g.abs() @ w.abs(), off @ w.abs(), self.vocab),
                                         (dw, g.t() @ x, g.abs().t() @ x.abs(), off.t() @ x.abs(), self.rows)):
            if got[0] is None:
                continue
            close(got[0], want, miss + E * (n + 16) * size + u * (want.abs() + miss) + LEAST[self.t] / 2)
            got[1]()
        if dx[0] is not None:
            assert not bool(dx[0][~self.ok].any())


SIZES = [(1, 1, 1), (1, 64, 2), (2, 8, 300), (5, 100, 63), (64, 64, 64), (65, 72, 65), (127, 200, 257), (128, 256, 256),
         (129, 264, 511), (255, 31, 1000), (256, 512, 1024), (257, 1000, 1001), (300, 130, 5000), (700, 96, 777),
         (33, 2049, 333), (1, 4096, 1500), (16, 640, 20001)]


@pytest.mark.parametrize("rows,cols,vocab", SIZES)
@pytest.mark.parametrize("t,ti", [(BF, I64), (H, I32)])
def test_loss(rows, cols, vocab, t, ti):
    p = Problem(rows, cols, vocab, t, ti)
    p.check_forward(*p.forward())
    p.check_forward(*p.forward(lse=False))


@pytest.mark.parametrize("rows,cols,vocab", SIZES)
@pytest.mark.parametrize("t,ti", [(BF, I64), (H, I32)])
def test_gradients(rows, cols, vocab, t, ti):
    p = Problem(rows, cols, vocab, t, ti)
    p.check_backward(*p.backward())


@pytest.mark.parametrize("rows,cols,vocab", [(2000, 520, 3001), (1025, 1536, 9000), (5000, 136, 600), (40, 264, 70001)])
@pytest.mark.parametrize("t", [BF, H])
def test_larger(rows, cols, vocab, t):
    """Several tiles each way."""
    p = Problem(rows, cols, vocab, t, size=4.0)
    loss, lse = p.forward()
    p.check_forward(loss, lse)
    p.check_backward(*p.backward(lse=lse))


@pytest.mark.parametrize("rows,cols,vocab", [(20, 8, 1_100_000), (100, 24, 1_050_001), (5000, 64, 60_001), (9000, 32, 70_000)])
def test_several_pieces_of_the_vocabulary(rows, cols, vocab):
    """More g than is held at once, so dx is added up over pieces."""
    p = Problem(rows, cols, vocab)
    p.check_forward(*p.forward())
    p.check_backward(*p.backward())


@pytest.mark.parametrize("rows,cols,vocab", [(5000, 1096, 3000), (2500, 2100, 1500), (130, 20_000, 700), (30, 40_000, 1500)])
def test_whole_and_cut_tiles(rows, cols, vocab):
    """More tiles of dx than places: a last wave cut along K; few rows, and rows of
    many tiles."""
    p = Problem(rows, cols, vocab)
    p.check_backward(*p.backward())


def test_many_rows():
    p = Problem(70_000, 16, 300, none=0.5)
    p.check_forward(*p.forward())
    p.check_backward(*p.backward())


@pytest.mark.parametrize("want", [(True, False), (False, True)])
@pytest.mark.parametrize("rows", [50, 600])
def test_one_gradient_alone(rows, want):
    p = Problem(rows, 136, 1500, dloss=None)
    p.check_backward(*p.backward(*want))


@pytest.mark.parametrize("pads,offsets", [((0, 0), (1, 0)), ((0, 0), (0, 1)), ((3, 5), (0, 0)), ((8, 8), (8, 8)),
                                          ((1, 0), (3, 5)), ((0, 8), (4, 4))])
@pytest.mark.parametrize("rows,cols,vocab", [(140, 264, 600), (20, 127, 300), (300, 65, 513)])
def test_strides_and_alignments(rows, cols, vocab, pads, offsets):
    p = Problem(rows, cols, vocab, BF, I64, 0.2, pads, offsets)
    p.check_forward(*p.forward())
    p.check_backward(*p.backward(pads=pads[::-1], offsets=offsets[::-1]))


@pytest.mark.parametrize("rows", [1, 60, 300])
def test_no_row_counts(rows):
    torch = T()
    p = Problem(rows, 72, 500, none=0.0)
    p.targets.fill_(-100)
    p.ok[:] = False
    p.x.fill_(float("nan"))
    p.work()
    p.check_forward(*p.forward())
    dx, dw = p.backward()
    assert not bool(dx[0].any()) and not bool(dw[0].any())


@pytest.mark.parametrize("kept", [0, 1, 299])
def test_one_row_counts(kept):
    p = Problem(300, 72, 500, none=0.0)
    keep = p.targets[kept].item()
    p.targets.fill_(500)
    p.targets[kept] = keep
    p.ok[:] = False
    p.ok[kept] = True
    p.x[~p.ok] = float("nan")
    p.work()
    p.check_forward(*p.forward())
    p.check_backward(*p.backward())


@pytest.mark.parametrize("rows,vocab", [(0, 5), (5, 0), (7, 40)])
def test_empty(rows, vocab):
    """No rows, no vocabulary; no columns, which makes every logit 0."""
    torch = T()
    x, w = torch.ones(rows, 16, device="cuda").bfloat16(), torch.ones(vocab, 16, device="cuda").bfloat16()
    y = torch.zeros(rows, dtype=torch.int64, device="cuda")
    loss, lse = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    cols = 0 if rows and vocab else 16
    mm.check(mm.mm_cross_entropy(x, w, y, loss, lse, rows, cols, vocab, 16, 16, (BF, I64, F)))
    want = torch.tensor(float(vocab if vocab else 1)).log()
    close(loss, want.cuda().expand(rows), 1e-6)
    close(lse, want.cuda().expand(rows), 1e-6)
    if not cols:
        return
    dx, dw = torch.full_like(x, 7), torch.full_like(w, 7)
    mm.check(mm.mm_cross_entropy_backward(x, w, y, lse, None, dx, dw, rows, 16, vocab, 16, 16, 16, 16, (BF, I64, BF)))
    assert not bool(dx.any()) and not bool(dw.any())


@pytest.mark.parametrize("rows", [10, 400])
def test_dx_in_place_of_x(rows):
    p = Problem(rows, 136, 700, none=0.0)
    dx, dw = p.backward()
    x = p.x.clone()
    mm.check(mm.mm_cross_entropy_backward(x, p.w, p.targets, p.lse, p.dloss, x, dw[0], rows, 136, 700, 136, p.w.stride(0),
                                          136, dw[0].stride(0), (BF, I64, BF)))
    assert T().equal(x, dx[0])


@pytest.mark.parametrize("rows", [20, 300])
def test_large_logits(rows):
    """Logits of some thousands: every other token's share vanishes, or ties for the top."""
    p = Problem(rows, 64, 300, none=0.0, size=2000.0)
    p.w[7] = p.w[3]
    p.work()
    p.check_forward(*p.forward())
    p.check_backward(*p.backward())


@pytest.mark.parametrize("rows", [20, 300])
def test_not_numbers(rows):
    """A NaN or an infinity in a row that counts is that row's alone (and dW's)."""
    torch = T()
    p = Problem(rows, 72, 400, none=0.0)
    good = p.forward()[0].clone()
    p.x[3, 5] = float("nan")
    p.x[9, 0] = float("inf")
    loss, lse = p.forward()
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[[3, 9]] = True
    assert not bool(torch.isfinite(loss[:rows][bad]).any())
    assert torch.equal(loss[:rows][~bad], good[:rows][~bad])
    (dx, _), _ = p.backward(lse=lse)
    assert bool(torch.isfinite(dx[~bad]).all()) and not bool(torch.isfinite(dx[bad]).any())


@pytest.mark.parametrize("t", [BF, H])
@pytest.mark.parametrize("kind", ["zero", "tiny", "huge", "range"])
def test_weights_of_the_losses(t, kind):
    torch = T()
    p = Problem(90, 72, 400, t, none=0.1)
    if kind == "zero":
        p.dloss.zero_()
    elif kind == "tiny":
        p.dloss *= 2.0 ** -13 if t == H else 2.0 ** -80
    elif kind == "huge":
        p.dloss *= 2.0 ** 10 if t == H else 2.0 ** 100
    else:
        p.dloss *= torch.exp2(torch.randint(-18, 1, (90,), generator=p.g, device="cuda").float())
    p.check_backward(*p.backward())


def test_a_weight_that_is_infinite():
    """Only its row of dx, and dW, are lost."""
    torch = T()
    p = Problem(60, 72, 400, none=0.1)
    at = p.ok.nonzero()[2, 0]
    dx = p.backward()[0][0].clone()
    for bad in (float("inf"), float("nan")):
        p.dloss[at] = bad
        got = p.backward()[0][0]
        rest = torch.arange(60, device="cuda") != at
        assert not bool(torch.isfinite(got[at]).any()) and bool(torch.isfinite(got[rest]).all())


def test_equal_bits():
    torch = T()
    p = Problem(700, 264, 5000)
    first = [t.clone() for t in p.forward()] + [t[0].clone() for t in p.backward()]
    for _ in range(3):
        again = list(p.forward()) + [t[0] for t in p.backward()]
        for a, b in zip(first, again):
            assert torch.equal(a, b)


def test_gradients_by_differences():
    """<dx, s> + <dW, S> is the change of sum dloss loss along (s, S), in double
    the precision of the types: the step is exact in them."""
    torch = T()
    p = Problem(40, 64, 90, H, none=0.1, size=1.0)
    p.x[~p.ok] = 0
    x0, w0 = p.x.clone(), p.w.clone()
    sx = torch.randint(-1, 2, x0.shape, generator=p.g, device="cuda").double()
    sw = torch.randint(-1, 2, w0.shape, generator=p.g, device="cuda").double()
    grid = 2.0 ** -9  # values on a grid that holds them and their steps exactly
    x0, w0 = (x0.float() / grid).round().clamp(-1000, 1000) * grid, (w0.float() / grid).round().clamp(-1000, 1000) * grid
    p.x.copy_(x0), p.w.copy_(w0)
    p.work()
    dx, dw = (o[0].double() for o in p.backward())
    inner = (dx * sx).sum() + (dw * sw).sum()
    ends = []
    for s in (1, -1):
        p.x.copy_((x0.double() + s * grid * sx)), p.w.copy_((w0.double() + s * grid * sw))
        loss = p.forward()[0][:40]
        ends.append((torch.where(p.ok, loss.double() * p.dloss.double(), 0.0)).sum())
    along = (ends[0] - ends[1]) / (2 * grid)
    # the third derivative of the loss along the step, (grid max|dl|)^3 / 6 a row,
    # and the fp32 roundings of the losses over the step
    dl = (sx.abs() @ w0.double().abs().t() + x0.double().abs() @ sw.abs().t()).amax(1)
    cubic = (p.dloss.double().abs() * (grid * dl) ** 3).sum() / (6 * grid) * 4
    fp32 = (p.dloss.double().abs() * (p.want_loss.abs() + p.L / E + 100) * E).sum() / grid
    coded = 2 * U[H] * ((dx * sx).abs().sum() + (dw * sw).abs().sum())
    assert abs((along - inner).item()) <= (cubic + fp32 + coded).item()


@pytest.mark.parametrize("rows", [30, 500])
def test_on_a_stream_and_in_a_graph(rows):
    torch = T()
    p = Problem(rows, 200, 3000)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    loss, lse = p.forward(s)
    (dx, _), (dw, _) = p.backward(lse=lse, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        mm.check(mm.mm_cross_entropy(p.x, p.w, p.targets, loss, lse, rows, 200, 3000, p.x.stride(0), p.w.stride(0),
                                     (BF, I64, F), s))
        mm.check(mm.mm_cross_entropy_backward(p.x, p.w, p.targets, lse, p.dloss, dx, dw, rows, 200, 3000, p.x.stride(0),
                                              p.w.stride(0), 200, 200, (BF, I64, BF), s))
    for _ in range(3):  # other inputs, and another number of rows that count
        p.targets.copy_(tokens_of(p.g, rows, 3000, I64, 0.4))
        p.ok = (p.targets >= 0) & (p.targets < 3000)
        p.x.copy_(torch.randn(rows, 200, generator=p.g, device="cuda"))
        p.work()
        for o in (loss, lse, dx, dw):
            o.fill_(77)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        p.lse = lse[:rows]
        p.check_forward(loss, lse)
        p.check_backward((dx, lambda: None), (dw, lambda: None))


def test_past_32_bits():
    """Rows whose elements lie beyond 2^31 in every operand."""
    torch = T()
    far = 1 << 25
    p = Problem(80, 72, 90)
    for name in ("x", "w"):
        small = getattr(p, name)
        big = torch.empty(small.shape[0], far, dtype=torch.bfloat16, device="cuda")[:, :72]
        big.copy_(small)
        setattr(p, name, big)
    p.check_forward(*p.forward())
    p.check_backward(*p.backward(pads=(far - 72, far - 72)))
