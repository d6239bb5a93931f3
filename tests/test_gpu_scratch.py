"""Scratch of the operators and of split products in graphs."""
import pytest

import matmul_selection_gb300 as mm
from test_gpu_operators import BF, EPS, F, H, T, bits, generator, q8_rows, rows_of, ttype

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


PER_THREAD = 2  # the handle of the calling thread's own default stream


def threads_at_one_time(todo, stream):
    """Each thread's calls over and over, all threads at one time: every one's
    results are those of its calls alone."""
    import threading
    torch = T()
    torch.cuda.synchronize()
    want = []
    for calls in todo:
        for call, _ in calls:
            mm.check(call(None))
        torch.cuda.synchronize()
        want.append([bits(outs) for _, outs in calls])
    for calls in todo:
        for _, outs in calls:
            for o in outs:
                o.view(torch.uint8).fill_(0xEE)
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(todo)), []

    def work(calls):
        start.wait()
        for _ in range(40):
            for call, _ in calls:
                if call(stream) != mm.MM_OK:
                    failed.append(mm.mm_last_error())

    threads = [threading.Thread(target=work, args=(c,)) for c in todo]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed[:3]
    for calls, w in zip(todo, want):
        for (_, outs), x in zip(calls, w):
            assert all(torch.equal(a, b) for a, b in zip(bits(outs), x))


def test_per_thread_streams_have_their_own_scratch():
    g = generator(33)
    threads_at_one_time([[backward(g, 200 + 50 * i, 4096), product(g, 30 + i, 2000, 3001),
                          split(g, 128, 256, 4096 + 512 * i)] for i in range(4)], PER_THREAD)


def test_threads_on_one_stream():
    """Calls of several launches, with scratch between them that other threads'
    calls of other sizes use and outgrow."""
    g = generator(34)
    s = T().cuda.Stream()
    threads_at_one_time([[backward(g, 60 * 3 ** i, 4096), product(g, 40, 700 * 3 ** i, 3001),
                          split(g, 64 * 3 ** i, 256, 4096)] for i in range(4)], s)


def test_a_call_refused_in_a_capture_launches_nothing():
    """4-bit weights with row factors and operands off 16 bytes: one kind of
    scratch is there from an earlier call, the other is not."""
    torch = T()
    g = generator(35)
    M, N, K = 40, 300, 512
    scales = {BF: rows_of(g, N, K // 64, BF, scale=0.01), F: rows_of(g, N, K // 64, F, scale=0.01)}
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    a = {t: rows_of(g, M, K, t, 3, offset=1) for t in (BF, H)}
    out = torch.empty(M, N, device="cuda")
    s = torch.cuda.Stream()

    def call(ta, ts, stream):
        return mm.mm_gemm_w4(a[ta], codes, scales[ts], None, out, M, N, K, K + 3, K, K // 64, N, 64, (ta, ts, F), stream)

    torch.cuda.synchronize()
    mm.check(call(BF, BF, s))
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        before = mm.mm_get_stats()["launches"]
        refused = call(H, F, s), mm.mm_get_stats()["launches"] - before
        mm.check(call(BF, BF, s))
    assert refused == (mm.MM_ERR_UNSUPPORTED, 0)
    want = bits([out])[0]
    out.fill_(0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits([out])[0], want)
