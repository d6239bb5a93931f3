"""Outputs whose rows lie whole 16-byte pieces apart but end inside one: the
elements behind a row's end stay untouched, by every candidate."""
import pytest

import matmul_selection_gb300 as mm
from gpu_util import BF16, F16, F32, Case

pytestmark = pytest.mark.gpu
NAMES = mm.candidate_names()


@pytest.mark.parametrize("cand", range(len(NAMES)), ids=NAMES)
@pytest.mark.parametrize("N,ends", [(250, 6), (257, 7), (126, 2)])
def test_padding_behind_a_row_is_untouched(cand, N, ends):
    for dt in ((BF16, BF16, BF16), (F16, F16, F16), (BF16, BF16, F32)):
        for layout, K in (("NN", 200), ("NT", 2000)):
            c = Case(140, N, K, layout=layout, dt=dt, dist="int4", pad=(0, 0, ends), seed=N).device()
            st = mm.mm_execute_candidate(cand, *c.args())
            if st == mm.MM_ERR_UNSUPPORTED:
                continue
            assert st == mm.MM_OK, f"{NAMES[cand]}: {mm.mm_last_error()}"
            c.check(exact=True)
