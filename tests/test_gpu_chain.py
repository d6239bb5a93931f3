"""Calls back to back on one stream, each reading what the one before it wrote a
moment ago into buffers that the earlier calls had read with other contents."""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_operators import BF, F, Q, T, bits, generator, q8_rows, rows_of, ttype

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 2000, 1024), (4, 512, 2048), (40, 1000, 1024), (300, 512, 512), (2000, 2048, 512)])
def test_products_see_the_scales_of_the_norm_before_them(M, N, K):
    torch = T()
    g = generator(M)
    s = torch.cuda.Stream()
    xs = [rows_of(g, M, K, BF, scale=10.0 ** (i % 5 - 2)) for i in range(12)]
    w = rows_of(g, 1, K, BF)[0]
    b = q8_rows(g, N, K)
    q = torch.empty(M, K, dtype=ttype(Q), device="cuda")
    scale = torch.empty(M, device="cuda")
    outs = [torch.empty(M, N, device="cuda") for _ in xs]

    def step(x, out, stream):
        # eps large against the rows' squares: the scales differ as the rows do
        mm.check(mm.mm_rmsnorm(x, None, w, None, q, scale, None, M, K, K, 0, 0, K, (BF, BF, Q), 1e4, stream))
        mm.check(mm.mm_gemm_q8(q, b, scale, None, out, M, N, K, K, K, N, (Q, Q, F), stream))

    want = []
    for x, out in zip(xs, outs):
        step(x, out, s)
        torch.cuda.synchronize()
        want.append(bits([out])[0])
        out.fill_(0)
    torch.cuda.synchronize()
    for _ in range(20):
        for x, out in zip(xs, outs):
            step(x, out, s)
    s.synchronize()
    assert all(torch.equal(bits([out])[0], x) for out, x in zip(outs, want))
