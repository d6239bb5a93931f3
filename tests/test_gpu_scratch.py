"""Scratch of the operators and of split products in graphs."""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_operators import BF, EPS, F, T, bits, generator, q8_rows, rows_of, ttype

pytestmark = pytest.mark.gpu


def backward(g, rows, cols):
    torch = T()
    dy, h = rows_of(g, rows, cols, BF), rows_of(g, rows, cols, BF)
    w = rows_of(g, 1, cols, F)[0]
    dx, dw = torch.empty(rows, cols, dtype=ttype(BF), device="cuda"), torch.empty(cols, device="cuda")
    return (lambda s: mm.mm_rmsnorm_backward(dy, None, h, w, None, dx, dw, rows, cols, cols, cols, cols, cols,
                                             (BF, F, BF), EPS, s)), [dx, dw]


def product(g, M, N, K):
    """Operands off 16 bytes, copied into scratch."""
    torch = T()
    a, b = q8_rows(g, M, K, 3, 1), q8_rows(g, N, K, 5, 2)
    out = torch.empty(M, N, device="cuda")
    return (lambda s: mm.mm_gemm_q8(a, b, None, None, out, M, N, K, a.stride(0), b.stride(0), N,
                                    (mm.MM_E4M3, mm.MM_E4M3, F), s)), [out]


def split(g, M, N, K):
    """A split-K product of the autotuned family."""
    torch = T()
    i = mm.candidate_names().index("tc_splitk_128x64_s8")
    a, b = rows_of(g, M, K, BF), rows_of(g, K, N, BF)
    out = torch.empty(M, N, device="cuda")
    return (lambda s: mm.mm_execute_candidate(i, a, b, out, M, N, K, K, N, N, (BF, BF, F), "NN", None, s)), [out]


def test_graphs_keep_their_scratch():
    """A graph for each size, smallest first, each replayed after the larger
    calls that outgrew its scratch."""
    torch = T()
    g = generator(31)
    s = torch.cuda.Stream()
    graphs = []
    for k in (1, 3, 9):
        calls = [backward(g, 100 * k, 4096), product(g, 40, 900 * k, 3001), split(g, 128 * k, 256, 4096)]
        torch.cuda.synchronize()  # the inputs, made on another stream
        for call, _ in calls:
            mm.check(call(s))
        s.synchronize()
        want = [bits(outs) for _, outs in calls]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for call, _ in calls:
                mm.check(call(s))
        graphs.append((graph, calls, want))  # (the calls hold the inputs)
    # memory that was given back would be taken by these
    other = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(24)]
    for graph, calls, want in graphs + graphs[::-1]:
        outs = [o for _, o in calls]
        for o in sum(outs, []):
            o.view(torch.uint8).fill_(0xEE)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(bits(o), w))
    assert all(bool((o == 7).all()) for o in other)
