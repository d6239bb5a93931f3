"""4-bit weights above 16 rows of A: scales outside f16's range with f16 A.
Bounds as in test_gpu_operators: a weight is rounded once to A's type."""
import pytest

from test_gpu_operators import BF, F, H, T, check_w4, generator, rows_of, run_w4, w4_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 16, 17, 40, 100, 300])
@pytest.mark.parametrize("slope", [1e-20, 2e-7, 1e-6, 1e-5, 1e-4, 1.0, 7e4, 1e20])
@pytest.mark.parametrize("ts", [F, BF])
def test_w4_f16_scales_of_any_size(M, slope, ts):
    g = generator(M)
    N, K, t = 130, 640, (H, ts, F)
    for group, zeros in ((32, True), (128, False)):
        a = rows_of(g, M, K, H)
        codes, ldw, s, z, w = w4_weights(g, N, K, group, ts, zeros, slope=slope)
        check_w4(a, w, t, run_w4(a, codes, ldw, s, z, N, K, group, t))


@pytest.mark.parametrize("M", [16, 20, 200])
def test_w4_f16_scales_of_many_sizes(M):
    """Rows of weights of very different sizes, groups of a row a thousand times
    apart, a row of zero scales, a zero weight under a large scale."""
    torch = T()
    g = generator(M)
    N, K, group, t = 300, 1000, 64, (H, F, F)
    a = rows_of(g, M, K, H)
    codes, ldw, s, z, w = w4_weights(g, N, K, group, F, True, slope=1.0)
    rows = torch.exp2((torch.arange(N, device="cuda") % 61 - 30).float())
    groups = torch.exp2(torch.randint(-5, 6, s.shape, generator=g, device="cuda").float())
    s.copy_(s * rows[:, None] * groups)
    s[7] = 0
    at = torch.arange(K, device="cuda") // group
    q = torch.stack([codes & 15, codes >> 4], 2).flatten(1)[:, :K].double()
    z[11] = 9
    codes[11] = 0x99  # every code its zero point
    s[11] = 1e30
    q[11] = 9
    w = (q - z.double()[:, at]) * s.double()[:, at]
    out = run_w4(a, codes, ldw, s, z, N, K, group, t)
    assert bool((out[:, 7] == 0).all()) and bool((out[:, 11] == 0).all())
    check_w4(a, w, t, out)
