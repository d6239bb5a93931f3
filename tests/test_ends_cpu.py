"""The operators at the ends of a language model: refusals and empty calls, which
need no GPU (the pointers are never dereferenced)."""
import pytest

import matmul_selection_gb300 as mm

BF, H, F, Q, I32, I64 = mm.MM_BF16, mm.MM_F16, mm.MM_F32, mm.MM_E4M3, mm.MM_I32, mm.MM_I64
BAD = mm.MM_ERR_INVALID_ARG


def embed(weight=0x1000, tokens=0x2000, out=0x3000, rows=4, cols=64, vocab=100, ldw=64, ldo=64,
          dt=(BF, I64, BF), scale=1.0):
    return mm.mm_embedding(weight, tokens, out, rows, cols, vocab, ldw, ldo, dt, scale)


def embed_bwd(dout=0x1000, tokens=0x2000, base=0x3000, dweight=0x4000, rows=4, cols=64, vocab=100, lddo=64,
              ldb=64, lddw=64, dt=(BF, I64, BF), scale=1.0):
    return mm.mm_embedding_backward(dout, tokens, base, dweight, rows, cols, vocab, lddo, ldb, lddw, dt, scale)


def loss(x=0x1000, weight=0x2000, targets=0x3000, loss=0x4000, lse=0x5000, rows=4, cols=64, vocab=100, ldx=64,
         ldw=64, dt=(BF, I64, F)):
    return mm.mm_cross_entropy(x, weight, targets, loss, lse, rows, cols, vocab, ldx, ldw, dt)


def loss_bwd(x=0x1000, weight=0x2000, targets=0x3000, lse=0x4000, dloss=0x5000, dx=0x6000, dweight=0x7000,
             rows=4, cols=64, vocab=100, ldx=64, ldw=64, lddx=64, lddw=64, dt=(BF, I64, BF)):
    return mm.mm_cross_entropy_backward(x, weight, targets, lse, dloss, dx, dweight, rows, cols, vocab, ldx, ldw,
                                        lddx, lddw, dt)


CALLS = (embed, embed_bwd, loss, loss_bwd)
REFUSED = [(c, {k: -1}, "negative") for c in CALLS for k in ("rows", "cols", "vocab")] + [
    (embed, dict(dt=(Q, I64, BF)), "types"), (embed, dict(dt=(BF, I64, Q)), "types"),
    (embed, dict(dt=(BF, F, BF)), "type of tokens"), (embed, dict(dt=(I32, I64, BF)), "types"),
    (embed, dict(dt=(BF, 6, BF)), "type of tokens"),
    (embed, dict(weight=None), "null weight"), (embed, dict(tokens=None), "null tokens"),
    (embed, dict(out=None), "null out"), (embed, dict(weight=0x1001), "element size"),
    (embed, dict(tokens=0x2004), "element size"), (embed, dict(tokens=0x2002, dt=(BF, I32, BF)), "element size"),
    (embed, dict(out=0x3002, dt=(BF, I64, F)), "element size"),
    (embed, dict(ldw=63), "leading dimension"), (embed, dict(ldo=63), "leading dimension"),
    (embed, dict(ldw=1 << 61), "address space"),
    (embed_bwd, dict(dt=(BF, BF, BF)), "type of tokens"), (embed_bwd, dict(dt=(Q, I64, BF)), "types"),
    (embed_bwd, dict(dout=None), "null dout"), (embed_bwd, dict(tokens=None), "null tokens"),
    (embed_bwd, dict(dweight=None), "null dweight"), (embed_bwd, dict(dout=0x1001), "element size"),
    (embed_bwd, dict(base=0x3001), "element size"), (embed_bwd, dict(dweight=0x4002, dt=(F, I64, BF), base=None), "element size"),
    (embed_bwd, dict(lddo=63), "leading dimension"), (embed_bwd, dict(ldb=63), "leading dimension"),
    (embed_bwd, dict(lddw=63), "leading dimension"),
    (embed_bwd, dict(base=0x4000, ldb=72), "another leading dimension"),
    (loss, dict(dt=(F, I64, F)), "type of x"), (loss, dict(dt=(Q, I64, F)), "type of x"),
    (loss, dict(dt=(BF, BF, F)), "type of targets"), (loss, dict(dt=(BF, I64, BF)), "type of loss"),
    (loss, dict(x=None), "null x"), (loss, dict(weight=None), "null weight"),
    (loss, dict(targets=None), "null targets"), (loss, dict(loss=None), "null loss"),
    (loss, dict(x=0x1001), "element size"), (loss, dict(weight=0x2001), "element size"),
    (loss, dict(targets=0x3001), "element size"), (loss, dict(loss=0x4002), "element size"),
    (loss, dict(lse=0x5002), "element size"), (loss, dict(ldx=63), "leading dimension"),
    (loss, dict(ldw=63), "leading dimension"),
    (loss_bwd, dict(dt=(F, I64, F)), "type of x"), (loss_bwd, dict(dt=(BF, I64, H)), "type of dx"),
    (loss_bwd, dict(dt=(BF, I64, F)), "type of dx"), (loss_bwd, dict(dt=(BF, F, BF)), "type of targets"),
    (loss_bwd, dict(x=None), "null x"), (loss_bwd, dict(weight=None), "null weight"),
    (loss_bwd, dict(targets=None), "null targets"), (loss_bwd, dict(lse=None), "null lse"),
    (loss_bwd, dict(dloss=0x5001), "element size"), (loss_bwd, dict(dx=0x6001), "element size"),
    (loss_bwd, dict(dweight=0x7001), "element size"), (loss_bwd, dict(ldx=63), "leading dimension"),
    (loss_bwd, dict(ldw=63), "leading dimension"), (loss_bwd, dict(lddx=63), "leading dimension"),
    (loss_bwd, dict(lddw=63), "leading dimension"), (loss_bwd, dict(dweight=0x2000), "in place"),
]


@pytest.mark.parametrize("call,args,says", REFUSED)
def test_refused_before_any_launch(call, args, says):
    before = mm.mm_get_stats()["launches"]
    assert call(**args) == BAD
    assert says in mm.mm_last_error()
    assert mm.mm_get_stats()["launches"] == before


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("args", [dict(rows=1 << 30), dict(vocab=1 << 30), dict(cols=1 << 30)])
def test_sizes_past_the_limits(call, args):
    lds = {k: 1 << 30 for k in ("ldw", "ldo", "lddo", "ldb", "lddw", "ldx", "lddx")
           if k in call.__code__.co_varnames[:call.__code__.co_argcount]}
    assert call(**args, **lds) == mm.MM_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", (embed, embed_bwd))
def test_rows_past_the_limit(call):
    ld = {"ldw": 1 << 30, "ldo": 1 << 30} if call is embed else {"lddo": 1 << 30, "ldb": 1 << 30, "lddw": 1 << 30}
    assert call(cols=1 << 23, **ld) == mm.MM_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,args", [
    (embed, dict(rows=0)), (embed, dict(cols=0)), (embed, dict(rows=0, weight=None, tokens=None, out=None)),
    (embed_bwd, dict(cols=0)), (embed_bwd, dict(vocab=0)), (embed_bwd, dict(vocab=0, dweight=None)),
    (loss, dict(rows=0)), (loss, dict(rows=0, x=None, weight=None, targets=None, loss=None)),
    (loss_bwd, dict(cols=0)), (loss_bwd, dict(dx=None, dweight=None)), (loss_bwd, dict(rows=0, dweight=None)),
    (loss_bwd, dict(rows=0, vocab=0)), (loss_bwd, dict(vocab=0, dx=None)),
])
def test_empty_calls_launch_nothing(call, args):
    before = mm.mm_get_stats()["launches"]
    assert call(**args) == mm.MM_OK
    assert mm.mm_get_stats()["launches"] == before


def test_argument_forms():
    for dt in ((BF, I64, BF), [BF, I64, BF], mm.mm_dtypes(BF, I64, BF)):
        assert embed(dt=dt, rows=0) == mm.MM_OK
        assert embed_bwd(dt=dt, vocab=0) == mm.MM_OK
        assert loss_bwd(dt=dt, cols=0) == mm.MM_OK
    assert loss(dt=[BF, I32, F], rows=0) == mm.MM_OK
    for bad in (lambda: embed(scale="1"), lambda: embed(weight=1.5), lambda: embed(rows="4"),
                lambda: embed_bwd(scale=None), lambda: loss(dt=(0, 0)), lambda: loss_bwd(lse="x")):
        with pytest.raises((TypeError, AttributeError)):
            bad()
    with pytest.raises(OverflowError):
        embed(vocab=1 << 70)
