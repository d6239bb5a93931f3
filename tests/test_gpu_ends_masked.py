"""Gradients of batches in which no position counts, after calls that have left their
row numbers in the stream's scratch: nothing but the outputs' rows is written."""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_cross_entropy import Problem
from test_gpu_operators import BF, H, T, rows_of

pytestmark = pytest.mark.gpu

AROUND = 4096  # rows before and after dx, more than any row number that is left over


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    assert mm.mm_operator_status() == mm.MM_OK, mm.mm_last_error()


def masked_call(rows, cols, vocab, t, offset, dw):
    torch = T()
    p = Problem(8, cols, vocab, t)
    x = rows_of(p.g, rows, cols, t, offset=offset)
    x.fill_(float("nan"))
    targets = torch.full((rows,), -100, device="cuda")
    lse, dloss = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    flat = torch.full(((rows + 2 * AROUND) * cols,), 77.0, device="cuda").to(x.dtype)
    at = AROUND * cols
    dx = flat[at:at + rows * cols].view(rows, cols)
    dweight = torch.full((vocab, cols), 77.0, device="cuda").to(x.dtype) if dw else None
    mm.check(mm.mm_cross_entropy_backward(x, p.w, targets, lse, dloss, dx, dweight, rows, cols, vocab, cols,
                                          p.w.stride(0), cols, cols, (t, p.ti, t)))
    assert not bool(dx.any())
    assert bool((flat[:at] == 77).all()) and bool((flat[at + rows * cols:] == 77).all())
    assert dweight is None or not bool(dweight.any())


@pytest.mark.parametrize("dw", [True, False])
@pytest.mark.parametrize("rows,cols,offset", [(300, 72, 0), (129, 264, 0), (2000, 72, 0), (100, 72, 1), (1, 65, 3)])
@pytest.mark.parametrize("t", [BF, H])
def test_no_position_counts_after_a_larger_call(rows, cols, offset, dw, t):
    """The scratch starts at the same address for each call: the larger call's rows, whose
    first ones do not count and leave -1, lie where the masked call's row numbers would."""
    before = Problem(2000, cols, 500, t)
    before.targets[256:512] = -100
    before.ok[256:512] = False
    before.x[~before.ok] = float("nan")
    before.work()
    before.check_backward(*before.backward())
    masked_call(rows, cols, 500, t, offset, dw)
    before.check_backward(*before.backward())
