"""Embedding and its gradient against their formulas in 64 bits.

Bounds, elementwise, with u the unit roundoff of the output's type, e = 2^-24
that of fp32 and d half the output's least value:
  out      scale w is rounded to fp32, then to the output:  (u + e) |out| + d
  dweight  n rows summed in fp32, in any grouping:  e (n + 1) scale sum|dout|
           + (u + 2 e) (|base| + |scale sum|) + d
"""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_operators import BF, F, H, LEAST, T, U, close, generator, out_rows, rows_of

pytestmark = pytest.mark.gpu

I32, I64 = mm.MM_I32, mm.MM_I64
E = 2.0 ** -24


def index_type(t):
    return T().int32 if t == I32 else T().int64


def tokens_of(gen, rows, vocab, ti, none=0.0):
    """Numbers of which low ones occur often, and some that are no token."""
    torch = T()
    u = torch.rand(rows, generator=gen, device="cuda")
    t = (vocab * u ** 4).long().clamp(0, vocab - 1)
    bad = torch.tensor([-1, -100, vocab, 2 ** 31 - 1, -2 ** 31] + ([2 ** 40, -2 ** 63] if ti == I64 else []), device="cuda")
    pick = bad[torch.randint(0, len(bad), (rows,), generator=gen, device="cuda")]
    t = torch.where(torch.rand(rows, generator=gen, device="cuda") < none, pick, t)
    return t.to(index_type(ti))


def run_embed(w, tokens, t, scale=1.0, pad=0, offset=0, stream=None):
    rows, (vocab, cols) = tokens.shape[0], w.shape
    out, untouched = out_rows(rows, cols, t[2], pad, offset)
    mm.check(mm.mm_embedding(w, tokens, out, rows, cols, vocab, w.stride(0), out.stride(0), t, scale, stream))
    return out, untouched


def check_embed(w, tokens, t, scale, got):
    torch = T()
    out, untouched = got
    n = tokens.long()
    ok = (n >= 0) & (n < w.shape[0])
    s = torch.tensor(scale).double().item()  # (as the call takes it: fp32)
    want = torch.where(ok[:, None], w[torch.where(ok, n, 0)].double() * s, 0.0)
    close(out, want.to(out.dtype) if t[2] == F else want, (U[t[2]] + E) * want.abs() + LEAST[t[2]] / 2)
    untouched()


@pytest.mark.parametrize("rows,cols,vocab,pads", [
    (1, 1, 1, (0, 0)), (1, 4096, 1000, (0, 0)), (3, 8, 5, (0, 0)), (17, 24, 100, (8, 16)), (257, 64, 33, (0, 0)),
    (100, 1001, 777, (0, 0)), (33, 1023, 50, (1, 2)), (40, 4097, 300, (3, 0)), (5, 20000, 40, (0, 8)),
    (1000, 160, 5000, (0, 0)), (70, 15, 9, (0, 5)), (64, 2048, 1, (0, 0))])
@pytest.mark.parametrize("t", [(BF, I64, BF), (F, I32, H), (H, I64, F), (F, I64, F), (BF, I32, H)])
def test_embedding(rows, cols, vocab, pads, t):
    g = generator(rows + cols)
    w = rows_of(g, vocab, cols, t[0], pads[0])
    tokens = tokens_of(g, rows, vocab, t[1], 0.2)
    check_embed(w, tokens, t, 0.75, run_embed(w, tokens, t, 0.75, pads[1]))


@pytest.mark.parametrize("offsets", [(1, 0), (0, 1), (3, 5), (8, 4), (4, 8)])
@pytest.mark.parametrize("t", [(BF, I64, BF), (F, I64, BF), (BF, I64, F)])
def test_embedding_alignments(offsets, t):
    g = generator(5)
    w = rows_of(g, 60, 328, t[0], 8, offset=offsets[0])
    tokens = tokens_of(g, 50, 60, I64)
    check_embed(w, tokens, t, 3.0, run_embed(w, tokens, t, 3.0, 8, offsets[1]))


def test_embedding_values():
    """Infinities and NaN pass; no token gives zeros even where the scale is infinite."""
    torch = T()
    w = torch.tensor([[float("inf"), float("nan"), -1.0, 70000.0] * 4], device="cuda")
    tokens = torch.tensor([0, -1, 1], device="cuda")
    out = torch.full((3, 16), 7.0, dtype=torch.float16, device="cuda")
    mm.check(mm.mm_embedding(w, tokens, out, 3, 16, 1, 16, 16, (F, I64, H), 1.0))
    assert torch.isinf(out[0, 0]) and torch.isnan(out[0, 1]) and out[0, 2] == -1 and torch.isinf(out[0, 3])
    assert not bool(out[1:].any())
    mm.check(mm.mm_embedding(w, tokens, out, 3, 16, 1, 16, 16, (F, I64, H), float("inf")))
    assert not bool(out[1:].any())
    mm.check(mm.mm_embedding(None, tokens, out, 3, 16, 0, 16, 16, (F, I64, H), 1.0))  # no vocabulary
    assert not bool(out.any())


def test_embedding_past_32_bits():
    """Rows whose elements lie beyond 2^31, in the matrix and in the output."""
    torch = T()
    g = generator(8)
    w = torch.empty(70, 1 << 25, dtype=torch.bfloat16, device="cuda")[:, :40]
    w.copy_(torch.randn(70, 40, generator=g, device="cuda"))
    tokens = torch.arange(69, -1, -1, device="cuda")
    out = torch.empty(70, 1 << 25, dtype=torch.bfloat16, device="cuda")[:, :40]
    mm.check(mm.mm_embedding(w, tokens, out, 70, 40, 70, 1 << 25, 1 << 25, (BF, I64, BF), 1.0))
    assert torch.equal(out, w.flip(0))
    dw = torch.empty(70, 1 << 25, dtype=torch.bfloat16, device="cuda")[:, :40]
    mm.check(mm.mm_embedding_backward(out, tokens, None, dw, 70, 40, 70, 1 << 25, 0, 1 << 25, (BF, I64, BF), 1.0))
    assert torch.equal(dw, w)


# ------------------------------------------------------------------ gradient

def run_bwd(dout, tokens, base, vocab, t, scale=1.0, pad=0, offset=0, in_place=False, stream=None):
    rows, cols = dout.shape
    dw, untouched = out_rows(vocab, cols, t[0], pad, offset)
    if in_place:
        dw.copy_(base)
        base = dw
    mm.check(mm.mm_embedding_backward(dout, tokens, base, dw, rows, cols, vocab, dout.stride(0),
                                      base.stride(0) if base is not None else 0, dw.stride(0), t, scale, stream))
    return dw, untouched


def check_bwd(dout, tokens, base, vocab, t, scale, got):
    torch = T()
    dw, untouched = got
    n = tokens.long()
    ok = (n >= 0) & (n < vocab)
    d = dout[ok].double() * scale
    zero = torch.zeros(vocab, dout.shape[1], dtype=torch.float64, device="cuda")
    total = zero.index_add(0, n[ok], d)
    size = zero.index_add(0, n[ok], d.abs())
    times = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_add(0, n[ok], torch.ones_like(d[:, 0]))
    b = base.double() if base is not None else zero
    close(dw, b + total, E * (times[:, None] + 1) * size + (U[t[0]] + 2 * E) * (b.abs() + total.abs()) + LEAST[t[0]] / 2)
    untouched()


BWD_TYPES = [(BF, I64, BF), (F, I32, BF), (F, I64, F), (H, I64, F), (BF, I32, H)]


@pytest.mark.parametrize("rows,cols,vocab,pads", [
    (1, 1, 1, (0, 0)), (1, 4096, 100, (0, 0)), (7, 8, 3, (0, 0)), (8, 16, 1, (0, 0)), (9, 16, 2, (8, 8)),
    (64, 64, 10, (0, 0)), (100, 1001, 77, (0, 0)), (300, 130, 40, (3, 1)), (1025, 24, 70000, (0, 0)),
    (4095, 72, 300, (0, 0)), (4096, 40, 300, (0, 0)), (5000, 33, 65536, (0, 0)), (10000, 16, 257, (0, 0)),
    (40000, 24, 1000, (0, 8))])
@pytest.mark.parametrize("t", BWD_TYPES)
@pytest.mark.parametrize("base", ["none", "apart", "in place"])
def test_embedding_backward(rows, cols, vocab, pads, t, base):
    g = generator(rows * 3 + cols)
    dout = rows_of(g, rows, cols, t[2], pads[0])
    tokens = tokens_of(g, rows, vocab, t[1], 0.1)
    b = rows_of(g, vocab, cols, t[0], pads[1]) if base != "none" else None
    check_bwd(dout, tokens, b, vocab, t, 1.5,
              run_bwd(dout, tokens, b, vocab, t, 1.5, pads[1], in_place=base == "in place"))


@pytest.mark.parametrize("rows", [1, 8, 9, 31, 4096, 4128, 9000, 70000])
@pytest.mark.parametrize("kind", ["one", "two", "ends", "lengths", "none", "all different"])
def test_embedding_backward_runs(rows, kind):
    """Tokens that fill many chunks, begin and end on a chunk's border, never occur."""
    torch = T()
    g = generator(rows)
    vocab = 131000
    i = torch.arange(rows, device="cuda")
    tokens = {"one": torch.full_like(i, 70001), "two": torch.where(i % 3 == 0, 5, 130999),
              "ends": i // 32 * 11,
              "lengths": torch.repeat_interleave(i, torch.randint(1, 90, (rows,), generator=g, device="cuda"))[:rows],
              "none": torch.full_like(i, vocab), "all different": (i * 7919) % vocab}[kind]
    t = (F, I64, BF)
    dout = rows_of(g, rows, 40, BF)
    check_bwd(dout, tokens, None, vocab, t, 1.0, run_bwd(dout, tokens, None, vocab, t))


@pytest.mark.parametrize("rows,cols,vocab", [(5000, 8, 1_000_000), (3000, 12, 270_000), (600, 100_000, 3), (40, 30_001, 9),
                                             (300_000, 8, 511), (300_000, 5, 512)])
def test_embedding_backward_extents(rows, cols, vocab):
    """Three passes of the sort, rows of many slabs, many places; a vocabulary that ends
    at a power of two."""
    g = generator(rows + vocab)
    dout = rows_of(g, rows, cols, BF)
    tokens = tokens_of(g, rows, vocab, I32, 0.1)
    t = (F, I32, BF)
    check_bwd(dout, tokens, None, vocab, t, 1.0, run_bwd(dout, tokens, None, vocab, t))
    base = rows_of(g, vocab, cols, F)
    check_bwd(dout, tokens, base, vocab, t, 1.0, run_bwd(dout, tokens, base, vocab, t, in_place=True))


@pytest.mark.parametrize("offsets", [(1, 0), (0, 1), (2, 3), (8, 4)])
def test_embedding_backward_alignments(offsets):
    g = generator(6)
    for t in BWD_TYPES[:3]:
        dout = rows_of(g, 300, 328, t[2], 8, offset=offsets[0])
        tokens = tokens_of(g, 300, 60, t[1], 0.1)
        base = rows_of(g, 60, 328, t[0], 8)
        check_bwd(dout, tokens, base, 60, t, 1.0, run_bwd(dout, tokens, base, 60, t, 1.0, 8, offsets[1]))


def test_embedding_backward_without_rows():
    torch = T()
    dw = torch.full((30, 12), 7.0, device="cuda")
    mm.check(mm.mm_embedding_backward(None, None, None, dw, 0, 12, 30, 12, 0, 12, (F, I64, F), 1.0))
    assert not bool(dw.any())
    base = torch.randn(30, 20, device="cuda")[:, :12]
    mm.check(mm.mm_embedding_backward(None, None, base, dw, 0, 12, 30, 12, 20, 12, (F, I64, F), 1.0))
    assert torch.equal(dw, base)


def test_embedding_backward_leaves_nan_of_no_token():
    """Rows of dout without a token are not read, whatever they hold."""
    torch = T()
    g = generator(9)
    dout = rows_of(g, 500, 64, BF)
    tokens = tokens_of(g, 500, 40, I64, 0.3)
    ok = (tokens >= 0) & (tokens < 40)
    dout[~ok] = float("nan")
    check_bwd(dout, tokens, None, 40, (F, I64, BF), 1.0, run_bwd(dout, tokens, None, 40, (F, I64, BF)))
    dout[ok.nonzero()[0, 0], 3] = float("inf")
    dw, _ = run_bwd(dout, tokens, None, 40, (F, I64, BF))
    assert torch.isinf(dw).sum() == 1 and not bool(torch.isnan(dw).any())


def test_embedding_backward_equal_bits():
    torch = T()
    g = generator(10)
    dout = rows_of(g, 20000, 136, BF)
    tokens = tokens_of(g, 20000, 500, I64)
    first = run_bwd(dout, tokens, None, 500, (F, I64, BF))[0].clone()
    for _ in range(5):
        assert torch.equal(run_bwd(dout, tokens, None, 500, (F, I64, BF))[0], first)


def test_embedding_gradient_by_differences():
    """The product of the gradient with a direction is the change of <out, dout> along it."""
    torch = T()
    g = generator(11)
    w, step = (rows_of(g, 50, 72, F) for _ in range(2))
    dout = rows_of(g, 400, 72, F)
    tokens = tokens_of(g, 400, 50, I32, 0.2)
    t = (F, I32, F)
    dw = run_bwd(dout, tokens, None, 50, t, 0.5)[0].double()
    ends = [(run_embed(w + s * step, tokens, t, 0.5)[0].double() * dout.double()).sum() for s in (1.0, -1.0)]
    along = ((ends[0] - ends[1]) / 2).item()
    # out is linear in w: exact but for roundings, each 2^-24 of a term
    size = (dout.double().abs().sum() * (w.abs().max() + step.abs().max()).double()).item()
    assert abs(along - (dw * step.double()).sum().item()) <= 8 * E * size


@pytest.mark.parametrize("rows", [50, 6000])
def test_on_a_stream_and_in_a_graph(rows):
    torch = T()
    g = generator(12)
    vocab, cols, t = 300, 264, (BF, I64, BF)
    w, tokens = rows_of(g, vocab, cols, BF), tokens_of(g, rows, vocab, I64, 0.1)
    dout = rows_of(g, rows, cols, BF)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, _ = run_embed(w, tokens, t, 2.0, stream=s)
    dw, _ = run_bwd(dout, tokens, None, vocab, t, 2.0, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        mm.check(mm.mm_embedding(w, tokens, out, rows, cols, vocab, w.stride(0), out.stride(0), t, 2.0, s))
        mm.check(mm.mm_embedding_backward(dout, tokens, None, dw, rows, cols, vocab, dout.stride(0), 0, dw.stride(0),
                                          t, 2.0, s))
    for k in range(3):
        tokens.copy_(tokens_of(g, rows, vocab, I64, 0.1))
        dout.copy_(torch.randn(rows, cols, generator=g, device="cuda"))
        out.fill_(9)
        dw.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_embed(w, tokens, t, 2.0, (out, lambda: None))
        check_bwd(dout, tokens, None, vocab, t, 2.0, (dw, lambda: None))


def test_refused_in_a_capture_without_scratch():
    """A call whose scratch is not there leaves nothing in the graph."""
    torch = T()
    s = torch.cuda.Stream()
    dout, tokens = torch.ones(3_000_000, 8, device="cuda"), torch.zeros(3_000_000, dtype=torch.int64, device="cuda")
    dw = torch.full((4, 8), 5.0, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        st = mm.mm_embedding_backward(dout, tokens, None, dw, 3_000_000, 8, 4, 8, 0, 8, (F, I64, F), 1.0, s)
    assert st == mm.MM_ERR_UNSUPPORTED and "capture" in mm.mm_last_error()
    graph.replay()
    torch.cuda.synchronize()
    assert bool((dw == 5).all())
