"""Products of a few very long rows off 16 bytes, which are copied first by many blocks a row."""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_cross_entropy import Problem
from test_gpu_operators import F, T, generator

pytestmark = pytest.mark.gpu

E4M3 = mm.MM_E4M3


@pytest.mark.parametrize("M,N,K", [(32, 16, 1_000_001), (20, 64, 4_000_001), (17, 3, 65_551), (130, 130, 300_007), (9, 6200, 20_003)])
def test_gemm_q8(M, N, K):
    """Ones of either sign: sums that fp32 holds exactly."""
    torch = T()
    g = generator(K)
    a, b = (torch.randint(0, 2, (n, K), generator=g, device="cuda") for n in (M, N))
    out = torch.empty(M, N, device="cuda")
    codes = [(0x38 + 0x80 * v).to(torch.uint8) for v in (a, b)]
    mm.check(mm.mm_gemm_q8(*codes, None, None, out, M, N, K, K, K, N, (E4M3, E4M3, F)))
    want = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for k in range(0, K, 1 << 17):
        want += (1 - 2 * a[:, k:k + (1 << 17)]).double() @ (1 - 2 * b[:, k:k + (1 << 17)]).double().t()
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("rows,cols,vocab", [(5, 70_001, 40), (140, 33_001, 20), (3, 200_001, 3)])
def test_loss(rows, cols, vocab):
    p = Problem(rows, cols, vocab)
    p.check_forward(*p.forward())
    p.check_backward(*p.backward())
