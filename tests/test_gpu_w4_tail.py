"""Codes past K are never used, whatever weights they would make."""
import pytest

from test_gpu_operators import BF, F, H, T, check_w4, generator, run_w4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 3, 8, 16, 17, 40, 100, 300])
@pytest.mark.parametrize("K,group", [(1, 32), (33, 32), (130, 128), (200, 128), (255, 64), (321, 128), (1090, 128)])
def test_w4_large_scales_at_the_end(M, K, group):
    """In the last group's scale a code past K makes a weight beyond the type's
    range; those below K do not (4-bit differences of 1)."""
    torch = T()
    g = generator(K)
    N, ldw = 140, 2048
    for ta, ts, big in ((H, H, 2.0 ** 14), (BF, BF, 2.0 ** 126), (BF, F, 2.0 ** 126), (H, H, float("inf")),
                        (BF, F, float("inf")), (H, F, float("inf"))):
        q = torch.zeros(N, ldw, dtype=torch.uint8, device="cuda")  # past K: -8
        q[:, :K] = 9
        codes = q[:, 0::2] | (q[:, 1::2] << 4)
        groups = -(-K // group)
        scales = torch.full((N, groups), 0.5, device="cuda")
        scales[:, -1] = big
        scales = scales.to({BF: torch.bfloat16, H: torch.float16, F: torch.float32}[ts])
        a = torch.rand(M, K, generator=g, device="cuda").add(0.5).to(torch.float16 if ta == H else torch.bfloat16)
        a = a * 2.0 ** -8 if big == 2.0 ** 126 else a
        at = torch.arange(K, device="cuda") // group
        w = scales.double()[:, at]  # codes of 9 under zero points of 8
        t = (ta, ts, F)
        out = run_w4(a.contiguous(), codes.contiguous(), ldw, scales.contiguous(), None, N, K, group, t)
        assert not bool(torch.isnan(out).any()), (t, big)
        check_w4(a, w, t, out)
