"""The backward pass forms the logits that the forward pass formed, bit for bit: where a token
holds a row's whole mass, lse is its logit, its share is exactly 1 and nothing is left to learn,
whatever the logits' size and however long the sums over K."""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_embedding import I64
from test_gpu_loss_range import forward
from test_gpu_operators import BF, H, T, generator, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    assert mm.mm_operator_status() == mm.MM_OK, mm.mm_last_error()


@pytest.mark.parametrize("cols", [64, 512, 520, 1001, 4096, 20_000])
@pytest.mark.parametrize("rows,vocab,offset", [(1, 1, 0), (20, 1, 0), (300, 1, 0), (33, 700, 0), (100, 3000, 1), (128, 300, 0),
                                               (129, 300, 0), (1500, 700, 0)])
@pytest.mark.parametrize("t", [BF, H])
def test_one_token_holds_all(rows, cols, vocab, offset, t):
    torch = T()
    g = generator(rows + cols + vocab)
    x, w = rows_of(g, rows, cols, t, offset=offset), rows_of(g, vocab, cols, t)
    # all products positive, so that the sums grow: logits of 25 to 330 thousand, the others' half
    x.copy_((x.abs() + 0.5) * 4)
    w.copy_((w.abs() + 0.5) * 4)
    top = vocab // 2
    w[:top] *= 0.25
    w[top + 1:] *= 0.25
    scale = max(1, 20_000 // cols) ** 0.5
    x.mul_(scale)
    targets = torch.full((rows,), top, device="cuda")
    loss, lse = forward(x, w, targets)
    assert not bool(loss.any()) and lse.min().item() > 8000
    dx, dw = torch.ones_like(x), torch.ones_like(w)
    mm.check(mm.mm_cross_entropy_backward(x, w, targets, lse, None, dx, dw, rows, cols, vocab, x.stride(0), w.stride(0),
                                          dx.stride(0), dw.stride(0), (t, I64, t)))
    assert not bool(dx.any()) and not bool(dw.any())


@pytest.mark.parametrize("cols", [520, 4096])
@pytest.mark.parametrize("t", [BF, H])
def test_backward_in_slices(cols, t):
    """lse of one call over all positions, gradients by calls over some of them, whose products
    have other tiles: the same logits still."""
    torch = T()
    g = generator(cols)
    rows, vocab = 700, 900
    x, w = rows_of(g, rows, cols, t), rows_of(g, vocab, cols, t)
    x.copy_((x.abs() + 0.5) * 4)
    w.copy_((w.abs() + 0.5) * 4)
    w[1:] *= 0.25
    targets = torch.zeros(rows, dtype=torch.int64, device="cuda")
    _, lse = forward(x, w, targets)
    for n in (1, 16, 100, 128, 129, 300):
        dx, dw = torch.ones_like(x), torch.ones_like(w)
        mm.check(mm.mm_cross_entropy_backward(x, w, targets, lse, None, dx, dw, n, cols, vocab, x.stride(0), w.stride(0),
                                              dx.stride(0), dw.stride(0), (t, I64, t)))
        assert not bool(dx[:n].any()) and not bool(dw.any()) and bool((dx[n:] == 1).all())
