"""The norm's 8-bit output for rows of very small values: the codes are
e4m3(y / scale) down to the scale's floor of 2^-126, whichever form a row's
length chooses.  Bounds as in test_gpu_operators."""
import pytest

from test_gpu_operators import BF, F, Q, T, check_norm, generator, rows_of, run_norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [40, 200, 1000, 1003, 4096, 4097, 40000, 70001])
@pytest.mark.parametrize("t", [(BF, BF, Q), (F, F, Q), (BF, F, Q)])
def test_norm_e4m3_tiny_rows(cols, t):
    """max|h w| from 1e-30 to below the floor, each row with zeros in it."""
    torch = T()
    g = generator(cols)
    sizes = [1e-30, 1e-34, 2e-36, 1e-36, 1e-37, 3e-38, 1e-39, 1e-41]
    x = rows_of(g, len(sizes), cols, F)
    x = (x.clamp(-2, 2) / 2 * torch.tensor(sizes, device="cuda")[:, None]).to(
        torch.bfloat16 if t[0] == BF else torch.float32)
    x[:, ::3] = 0
    x[:, 1] = torch.tensor(sizes, device="cuda").to(x.dtype)  # the row's largest
    w = torch.ones(cols, device="cuda").to(torch.bfloat16 if t[1] == BF else torch.float32)
    h, y, scale, rstd = run_norm(x, None, w, t)
    assert bool(torch.isfinite(scale).all()) and bool(torch.isfinite(y.float()).all())
    assert bool((y.float()[:, ::3] == 0).all())
    check_norm(x, None, w, t, (h, y, scale, rstd))


@pytest.mark.parametrize("cols", [64, 4096, 40000])
def test_norm_e4m3_tiny_weights(cols):
    """Ordinary rows, weights near the least normal float."""
    torch = T()
    g = generator(cols)
    x = rows_of(g, 3, cols, F)
    x[2] *= 1e-3
    w = rows_of(g, 1, cols, F, scale=1e-37)[0]
    w[::2] = 0
    t = (F, F, Q)
    check_norm(x, None, w, t, run_norm(x, None, w, t))
