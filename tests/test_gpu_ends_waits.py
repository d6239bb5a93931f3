"""Waits of the loss's products that run out: see test_gpu_operator_waits."""
import pytest

from test_gpu_cross_entropy import Problem
from test_gpu_operator_waits import gives_up_and_recovers, stalled  # noqa: F401
from test_gpu_operators import BF, H

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,vocab,t", [(20, 1000, 3000, BF), (128, 72, 600, H), (400, 1000, 5000, BF),
                                               (3000, 520, 2000, H), (140, 65, 300, BF)])
def test_products_that_give_up(rows, cols, vocab, t, stalled):  # noqa: F811
    p = Problem(rows, cols, vocab, t)
    gives_up_and_recovers(p.forward, lambda got: p.check_forward(*got), stalled)
    gives_up_and_recovers(p.backward, lambda got: p.check_backward(*got), stalled)
