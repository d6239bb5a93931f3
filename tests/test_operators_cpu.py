"""The operators around a quantised linear layer: refusals and empty calls,
which need no GPU (the pointers are never dereferenced)."""
import pytest

import matmul_selection_gb300 as mm

BF, H, F, Q = mm.MM_BF16, mm.MM_F16, mm.MM_F32, mm.MM_E4M3
BAD = mm.MM_ERR_INVALID_ARG


def norm(x=0x1000, residual=0x2000, weight=0x3000, h=0x4000, y=0x5000, scale=None, rstd=0x7000,
         rows=4, cols=64, ldx=64, ldr=64, ldh=64, ldy=64, dt=(BF, BF, BF), eps=1e-6):
    return mm.mm_rmsnorm(x, residual, weight, h, y, scale, rstd, rows, cols, ldx, ldr, ldh, ldy, dt, eps)


def bwd(dy=0x1000, dh=0x2000, h=0x3000, weight=0x4000, rstd=0x5000, dx=0x6000, dweight=0x7000,
        rows=4, cols=64, lddy=64, lddh=64, ldh=64, lddx=64, dt=(BF, BF, BF), eps=1e-6):
    return mm.mm_rmsnorm_backward(dy, dh, h, weight, rstd, dx, dweight, rows, cols, lddy, lddh, ldh,
                                  lddx, dt, eps)


def w4(A=0x1000, codes=0x2000, scales=0x3000, zeros=0x4000, out=0x5000, M=4, N=64, K=256, lda=256,
       ldw=256, lds=2, ldc=64, group=128, dt=(BF, BF, BF)):
    return mm.mm_gemm_w4(A, codes, scales, zeros, out, M, N, K, lda, ldw, lds, ldc, group, dt)


def q8(A=0x1000, B=0x2000, scale_a=0x3000, scale_b=0x4000, out=0x5000, M=4, N=64, K=256, lda=256,
       ldb=256, ldc=64, dt=(Q, Q, BF)):
    return mm.mm_gemm_q8(A, B, scale_a, scale_b, out, M, N, K, lda, ldb, ldc, dt)


NAN, INF = float("nan"), float("inf")

REFUSED = [
    (norm, dict(rows=-1), "negative"), (norm, dict(cols=-1), "negative"),
    (norm, dict(dt=(Q, BF, BF)), "types"), (norm, dict(dt=(BF, Q, BF)), "types"),
    (norm, dict(dt=(BF, BF, 4)), "types"),
    (norm, dict(eps=-1.0), "eps"), (norm, dict(eps=NAN), "eps"), (norm, dict(eps=INF), "eps"),
    (norm, dict(dt=(BF, BF, Q)), "scale"), (norm, dict(scale=0x6000), "scale"),
    (norm, dict(x=None), "null x"), (norm, dict(weight=None), "null weight"),
    (norm, dict(y=None), "null y"), (norm, dict(h=0x5000), "same buffer"),
    (norm, dict(x=0x1001), "element size"), (norm, dict(residual=0x2001), "element size"),
    (norm, dict(h=0x4001), "element size"), (norm, dict(y=0x5001), "element size"),
    (norm, dict(rstd=0x7002), "element size"), (norm, dict(weight=0x3002, dt=(BF, F, BF)), "element size"),
    (norm, dict(scale=0x6002, dt=(BF, BF, Q)), "element size"),
    (norm, dict(ldx=63), "leading dimension"), (norm, dict(ldr=63), "leading dimension"),
    (norm, dict(ldh=63), "leading dimension"), (norm, dict(ldy=63), "leading dimension"),
    (norm, dict(ldx=1 << 61), "address space"),
    (bwd, dict(rows=-1), "negative"), (bwd, dict(dt=(BF, BF, Q)), "types"),
    (bwd, dict(eps=-0.5), "eps"), (bwd, dict(dy=None), "null dy"), (bwd, dict(h=None), "null h"),
    (bwd, dict(weight=None), "null weight"), (bwd, dict(dx=None), "null dx"),
    (bwd, dict(dx=0x3000), "in place"), (bwd, dict(dweight=0x7001), "element size"),
    (bwd, dict(rstd=0x5001), "element size"), (bwd, dict(lddy=1), "leading dimension"),
    (bwd, dict(lddh=1), "leading dimension"), (bwd, dict(lddx=1), "leading dimension"),
    (w4, dict(M=-1), "negative"), (w4, dict(dt=(F, BF, BF)), "A's type"),
    (w4, dict(dt=(BF, Q, BF)), "types"), (w4, dict(dt=(BF, BF, Q)), "types"),
    (w4, dict(group=16), "group"), (w4, dict(group=0), "group"), (w4, dict(group=256), "group"),
    (w4, dict(ldw=257), "whole bytes"), (w4, dict(ldw=254), "leading dimension"),
    (w4, dict(lda=255), "leading dimension"), (w4, dict(lds=1), "leading dimension"),
    (w4, dict(ldc=63), "leading dimension"), (w4, dict(A=None), "null A"),
    (w4, dict(codes=None), "null codes"), (w4, dict(scales=None), "null scales"),
    (w4, dict(out=None), "null out"), (w4, dict(A=0x1001), "element size"),
    (w4, dict(scales=0x3001), "element size"), (w4, dict(out=0x5001), "element size"),
    (q8, dict(K=-1), "negative"), (q8, dict(dt=(BF, Q, BF)), "types"),
    (q8, dict(dt=(Q, Q, Q)), "types"), (q8, dict(A=None), "null A"), (q8, dict(B=None), "null B"),
    (q8, dict(out=None), "null out"), (q8, dict(lda=255), "leading dimension"),
    (q8, dict(ldb=255), "leading dimension"), (q8, dict(ldc=63), "leading dimension"),
    (q8, dict(scale_a=0x3002), "element size"), (q8, dict(scale_b=0x4001), "element size"),
    (q8, dict(out=0x5001), "element size"),
]


@pytest.mark.parametrize("call,args,says", REFUSED)
def test_refused_before_any_launch(call, args, says):
    assert call(**args) == BAD
    assert says in mm.mm_last_error()
    with pytest.raises(mm.MMError):
        mm.check(call(**args))


@pytest.mark.parametrize("call,args", [
    (norm, dict(cols=1 << 31, ldx=1 << 31, ldr=1 << 31, ldh=1 << 31, ldy=1 << 31)),
    (norm, dict(cols=1 << 30, ldx=1 << 31, ldr=1 << 31, ldh=1 << 31, ldy=1 << 31)),
    (bwd, dict(cols=1 << 31)), (bwd, dict(cols=1 << 30)),
    (w4, dict(M=1 << 30)), (w4, dict(N=1 << 30)), (w4, dict(K=1 << 30)),
    (q8, dict(M=1 << 30)), (q8, dict(N=1 << 30)), (q8, dict(K=1 << 30)),
])
def test_sizes_past_the_limits(call, args):
    assert call(**args) == mm.MM_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,args", [
    (norm, dict(rows=0)), (norm, dict(cols=0)), (norm, dict(rows=0, x=None, y=None)),
    (bwd, dict(cols=0)), (bwd, dict(rows=0, dweight=None)),
    (w4, dict(M=0)), (w4, dict(N=0)), (w4, dict(M=0, A=None, out=None)),
    (q8, dict(M=0)), (q8, dict(N=0, B=None, out=None)),
])
def test_empty_calls_launch_nothing(call, args):
    before = mm.mm_get_stats()["launches"]
    assert call(**args) == mm.MM_OK
    assert mm.mm_get_stats()["launches"] == before


def test_argument_forms():
    """Types as a tuple, a list or the struct; addresses as numbers, None or
    objects with data_ptr(); streams as numbers or objects with cuda_stream;
    anything else is a TypeError, before any call."""
    class Tensor:
        def data_ptr(self):
            return 0x1001

    class Stream:
        cuda_stream = 0

    for dt in ((BF, BF, BF), [BF, BF, BF], mm.mm_dtypes(BF, BF, BF)):
        assert norm(dt=dt, rows=0) == mm.MM_OK
        assert norm(dt=dt, x=Tensor()) == BAD and "x not aligned" in mm.mm_last_error()
    assert mm.mm_gemm_q8(None, None, None, None, None, 0, 1, 1, 1, 1, 1, (Q, Q, F), Stream()) == mm.MM_OK
    assert mm.mm_gemm_q8(None, None, None, None, None, 0, 1, 1, 1, 1, 1, (Q, Q, F), stream=0) == mm.MM_OK
    for bad in (lambda: norm(x="x"), lambda: norm(x=1.5), lambda: norm(rows="4"), lambda: norm(dt=(0, 0)),
                lambda: norm(dt=("a", 0, 0)), lambda: norm(eps="x"), lambda: w4(group=1.5),
                lambda: mm.mm_gemm_q8(None, None, None, None, None, 0, 1, 1, 1, 1, 1, (Q, Q, F), "stream")):
        with pytest.raises((TypeError, AttributeError)):
            bad()
    with pytest.raises(OverflowError):
        norm(rows=1 << 70)
