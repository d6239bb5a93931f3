"""The embedding and its gradient at the largest numbers of columns, rows anywhere: bounds
as in test_gpu_embedding."""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_embedding import E, I32, I64, check_embed, run_bwd, run_embed
from test_gpu_operators import BF, F, LEAST, T, U, generator, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [64 * 65535 + 1, 2 ** 23 - 1, 2 ** 23 - 8])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_of_many_columns(cols, in_place):
    """A token of 30 places, over several chunks, one of 5, and some that are none."""
    torch = T()
    g = generator(cols)
    tokens = torch.tensor([1] * 9 + [0, -1, 3] + [1] * 21 + [0, 7, 0, 2, 0, 0], device="cuda")
    rows, vocab = len(tokens), 4
    dout = rows_of(g, rows, cols, BF)
    base = rows_of(g, vocab, cols, F) if in_place else None
    got, untouched = run_bwd(dout, tokens, base, vocab, (F, I64, BF), 0.5, in_place=in_place)
    for c in range(0, cols, 1 << 20):
        at = slice(c, min(cols, c + (1 << 20)))
        for v in range(vocab):
            these = dout[tokens == v][:, at].double()
            want = 0.5 * these.sum(0)
            bound = E * (len(these) + 1) * 0.5 * these.abs().sum(0) + (U[F] + 2 * E) * want.abs() + LEAST[F]
            if in_place:
                want = want + base[v, at].double()
                bound = bound + (U[F] + 2 * E) * base[v, at].abs()
            assert bool(((got[v, at].double() - want).abs() <= bound).all())
    untouched()


@pytest.mark.parametrize("cols", [64 * 65535 + 1, 2 ** 23 - 1])
def test_lookup_of_many_columns(cols):
    torch = T()
    w = rows_of(generator(cols), 3, cols, BF)
    tokens = torch.tensor([2, -1, 0, 1], dtype=torch.int32, device="cuda")
    check_embed(w, tokens, (BF, I32, F), 0.75, run_embed(w, tokens, (BF, I32, F), 0.75))
