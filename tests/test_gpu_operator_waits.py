"""Waits that run out: the test hook makes a kernel first wait, 1 ms, on a
barrier that nothing arrives on.  The kernel records that, lets its copies land
and returns; mm_operator_status reports it once; the next calls are right."""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_operators import (BF, F, H, check_bwd, check_q8, check_w4, generator, q8_rows, q8_scales, rows_of,
                                run_bwd, run_q8, run_w4, w4_weights)

pytestmark = pytest.mark.gpu


@pytest.fixture
def stalled():
    """Switches the hook on and off."""
    def switch(on):
        mm.check(mm.mm_set_option("wait_limit_us", "1000" if on else "2000000"))
        mm.check(mm.mm_set_option("wait_stall", "1" if on else "0"))
    yield switch
    switch(False)
    mm.mm_operator_status()


def gives_up_and_recovers(call, check, switch):
    assert mm.mm_operator_status() == mm.MM_OK
    switch(True)
    call()
    assert mm.mm_operator_status() == mm.MM_ERR_TIMEOUT and "gave up" in mm.mm_last_error()
    assert mm.mm_operator_status() == mm.MM_OK
    switch(False)
    for _ in range(2):
        check(call())
    assert mm.mm_operator_status() == mm.MM_OK


@pytest.mark.parametrize("rows,cols,t,pad", [
    (5000, 2048, (BF, BF, BF), 0), (3000, 4096, (BF, F, BF), 0), (2000, 8192, (F, F, F), 0),
    (2000, 16384, (H, H, H), 0), (4001, 1003, (BF, BF, BF), 0), (1500, 4097, (F, BF, F), 3), (700, 16383, (BF, BF, BF), 0),
    (400, 16388, (F, F, F), 0), (300, 40001, (BF, BF, BF), 5)])
def test_backward_whose_ring_gives_up(rows, cols, t, pad, stalled):
    """More rows than the rings hold at once, in each of the forms with a ring."""
    g = generator(cols)
    dy, dh, h = (rows_of(g, rows, cols, t[0], pad) for _ in range(3))
    w = rows_of(g, 1, cols, t[1])[0]
    gives_up_and_recovers(lambda: run_bwd(dy, dh, h, w, t, pad=pad),
                          lambda got: check_bwd(dy, dh, h, w, t, got), stalled)


def test_the_record_outlives_a_tuning_run(stalled):
    """Candidates are measured between an operator's call and the query."""
    from gpu_util import Case
    g = generator(1)
    dy, h = (rows_of(g, 1000, 4096, BF) for _ in range(2))
    w = rows_of(g, 1, 4096, BF)[0]
    stalled(True)
    run_bwd(dy, None, h, w, (BF, BF, BF))
    stalled(False)
    tunes = mm.mm_get_stats()["tunes"]
    c = Case(224, 96, 352, dist="int4", seed=77).device()
    mm.check(mm.mm_autotune_execute(*c.args()))
    c.check(exact=True)
    assert mm.mm_get_stats()["tunes"] == tunes + 1
    assert mm.mm_operator_status() == mm.MM_ERR_TIMEOUT
    assert mm.mm_operator_status() == mm.MM_OK


@pytest.mark.parametrize("M,N,K", [
    (1, 512, 4096), (3, 6000, 1000), (8, 6144, 2000),     # GEMV form, K split and not
    (1, 6400, 4096), (30, 512, 4096), (64, 300, 8192), (100, 4096, 1000), (300, 4096, 4096),  # swap
    (2000, 4096, 1000), (3000, 8192, 300)])               # pair
def test_8_bit_product_that_gives_up(M, N, K, stalled):
    g = generator(M)
    a, b = q8_rows(g, M, K, -K % 16), q8_rows(g, N, K, -K % 16)
    sa, sb = q8_scales(g, M), q8_scales(g, N)
    gives_up_and_recovers(lambda: run_q8(a, b, sa, sb, BF), lambda out: check_q8(a, b, sa, sb, BF, out), stalled)


@pytest.mark.parametrize("M,N,K", [
    (1, 512, 4096), (2, 20000, 1000), (4, 20000, 1000), (8, 20000, 1000), (16, 512, 4096), (16, 40000, 512),  # GEMV
    (20, 512, 4096), (50, 512, 4096), (100, 512, 4096), (250, 512, 4096),      # tiles, K split
    (32, 20000, 2048), (64, 20000, 2048), (128, 20000, 2048), (1000, 8192, 2048)])  # and not
def test_4_bit_product_that_gives_up(M, N, K, stalled):
    g = generator(M)
    t = (BF, BF, F)
    a = rows_of(g, M, K, BF)
    codes, ldw, s, z, w = w4_weights(g, N, K, 64, BF, True)
    gives_up_and_recovers(lambda: run_w4(a, codes, ldw, s, z, N, K, 64, t), lambda out: check_w4(a, w, t, out), stalled)
