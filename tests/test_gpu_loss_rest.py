"""Gradients of more than 128 positions: what the 16 bits of g lose at the targets is kept, so
that results which one target makes are as exact as their own rounding.

Bounds as in test_gpu_cross_entropy, but for g at a target, whose two values are off by u^2 |g|
(u the unit roundoff of the 16-bit type), the others by u |g|.
"""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_cross_entropy import E, Problem
from test_gpu_embedding import I32, I64
from test_gpu_operators import BF, H, LEAST, T, U, close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    assert mm.mm_operator_status() == mm.MM_OK, mm.mm_last_error()


def check(p, dx, dw):
    torch = T()
    u, ok = U[p.t], p.ok[:, None]
    x, w = torch.where(ok, p.x, 0).double(), p.w.double()
    d = p.dloss.double()[:, None] if p.dloss is not None else torch.ones(p.rows, 1, device="cuda").double()
    d = torch.where(ok, d, 0.0)
    l_p = torch.exp(p.l - p.lse.double()[:, None])
    at = torch.where(ok, p.targets.long()[:, None], 0)
    g = l_p.clone().scatter_add_(1, at, -torch.ones_like(d)) * d
    off = (2 * p.L + E * (8 + 4 * p.top))[:, None] * l_p * d.abs() * (1 + u) + (u + 4 * E) * g.abs()
    off.scatter_add_(1, at, -(u - u * u) * g.abs().gather(1, at))
    if p.t == H:
        off = torch.where(ok, off + LEAST[H] / 2 / 2 ** 14 * d.abs().max(), 0.0)
    for got, want, size, miss, n in ((dx, g @ w, g.abs() @ w.abs(), off @ w.abs(), p.vocab),
                                     (dw, g.t() @ x, g.abs().t() @ x.abs(), off.t() @ x.abs(), p.rows)):
        close(got[0], want, miss + E * (n + 16) * size + u * (want.abs() + miss) + LEAST[p.t] / 2)
        got[1]()
    assert not bool(dx[0][~p.ok].any())


SIZES = [(129, 264, 511), (256, 64, 256), (257, 72, 257), (300, 130, 5000), (700, 96, 777), (1024, 200, 300), (1025, 1096, 9000),
         (2000, 520, 3001), (5000, 64, 60_001), (600, 72, 131_072), (900, 40, 140_001), (2049, 130, 20_000), (4000, 65, 40)]


@pytest.mark.parametrize("rows,cols,vocab", SIZES)
@pytest.mark.parametrize("t,ti,none", [(BF, I64, 0.2), (H, I32, 0.5), (H, I64, 0.0)])
def test_gradients(rows, cols, vocab, t, ti, none):
    p = Problem(rows, cols, vocab, t, ti, none)
    check(p, *p.backward())


@pytest.mark.parametrize("kind", ["one token", "one tile", "all different", "last tile", "descending", "ends"])
@pytest.mark.parametrize("rows,cols,vocab", [(500, 136, 1000), (3000, 72, 5001)])
@pytest.mark.parametrize("t", [BF, H])
def test_targets_anywhere(rows, cols, vocab, kind, t):
    torch = T()
    p = Problem(rows, cols, vocab, t, none=0.0)
    i = torch.arange(rows, device="cuda")
    p.targets.copy_({"one token": 0 * i + vocab // 2, "one tile": 512 + i * 7 % 256, "all different": i * 977 % vocab,
                     "last tile": vocab - 1 - i % 3, "descending": (vocab - 1 - i) % vocab, "ends": (i & 1) * (vocab - 1)}[kind])
    p.work()
    check(p, *p.backward())


@pytest.mark.parametrize("pads,offsets", [((0, 0), (1, 0)), ((0, 0), (0, 1)), ((3, 5), (0, 0)), ((1, 0), (3, 5))])
@pytest.mark.parametrize("rows,cols,vocab", [(140, 264, 600), (1300, 65, 513), (300, 7, 900)])
def test_strides_and_alignments(rows, cols, vocab, pads, offsets):
    p = Problem(rows, cols, vocab, BF, I64, 0.2, pads, offsets)
    check(p, *p.backward(pads=pads[::-1], offsets=offsets[::-1]))


def test_equal_bits():
    torch = T()
    p = Problem(3000, 136, 2000, H)
    first = [o[0].clone() for o in p.backward()]
    for _ in range(5):
        assert all(torch.equal(a, b[0]) for a, b in zip(first, p.backward()))
