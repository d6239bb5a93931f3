"""The ends of a language model as they are used: one after another, beside one
another, on threads, in graphs."""
import importlib.util
import os
import threading

import pytest

import matmul_selection_gb300 as mm
from test_gpu_cross_entropy import Problem
from test_gpu_embedding import F, I64, check_bwd, check_embed, run_bwd, run_embed, tokens_of
from test_gpu_operators import BF, H, T, generator, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    assert mm.mm_operator_status() == mm.MM_OK, mm.mm_last_error()


@pytest.mark.parametrize("tokens,hidden,vocab", [(64, 256, 500), (700, 136, 3001), (2048, 512, 8000)])
def test_training_step_with_tied_weights(tokens, hidden, vocab):
    """The example's step.  Every result passes through a few roundings to bf16 (the
    embedded rows, the norm's output, dy, de, dW twice), each off by at most 2^-8 of a
    value and about 2^-8 / sqrt(3) in the norm; the loss is a mean in fp32 of what two
    of them feed (x and W enter the plain step as bf16 values too)."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "language_model_ends.py")
    spec = importlib.util.spec_from_file_location("language_model_ends", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    rel = ex.run(tokens, hidden, vocab)
    assert rel["loss"] < 2 * 2.0 ** -8, rel
    for name in ("dW", "dweight"):
        assert rel[name] < 6 * 2.0 ** -8, rel


@pytest.mark.parametrize("rows", [5, 40, 128, 400])
def test_operands_written_a_moment_ago(rows):
    """x, W, targets and dloss come from the kernels just before, in buffers that the
    calls before read with other contents (some of it is asked for ahead of time)."""
    torch = T()
    s = torch.cuda.Stream()
    t = (BF, I64, BF)
    problems = [Problem(rows, 520, 4000, seed=k) for k in range(6)]
    vocab = [torch.randperm(4000, generator=problems[0].g, device="cuda") for _ in problems]
    x, w = torch.zeros(rows, 520, device="cuda").bfloat16(), torch.zeros(4000, 520, device="cuda").bfloat16()
    targets, dloss = torch.zeros(rows, dtype=torch.int64, device="cuda"), torch.zeros(rows, device="cuda")
    loss, lse = (torch.zeros(len(problems), rows + 8, device="cuda") for _ in range(2))
    loss.fill_(77), lse.fill_(77)
    dx, dw = (torch.zeros(len(problems), n, 520, device="cuda").bfloat16() for n in (rows, 4000))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for k, p in enumerate(problems):
            targets.copy_(p.targets)
            dloss.copy_(p.dloss)
            x.copy_(p.x)
            # the library's own kernels write W: its rows as their own gradient
            mm.check(mm.mm_embedding_backward(p.w[vocab[k]].contiguous(), vocab[k], None, w, 4000, 520, 4000, 520, 0, 520,
                                              t, 1.0, s))
            mm.check(mm.mm_cross_entropy(x, w, targets, loss[k], lse[k], rows, 520, 4000, 520, 520, (BF, I64, F), s))
            mm.check(mm.mm_cross_entropy_backward(x, w, targets, lse[k], dloss, dx[k], dw[k], rows, 520, 4000, 520, 520,
                                                  520, 520, t, s))
    torch.cuda.synchronize()
    for k, p in enumerate(problems):
        p.lse = lse[k][:rows]
        p.check_forward(loss[k], lse[k])
        p.check_backward((dx[k], lambda: None), (dw[k], lambda: None))


def test_streams_beside_one_another():
    """Calls of every operator on three streams at once."""
    torch = T()
    g = generator(21)
    problems = [Problem(60, 200, 3000, seed=1), Problem(500, 264, 2000, seed=2), Problem(900, 72, 5000, H, seed=3)]
    rows = [(rows_of(g, n, 264, BF), tokens_of(g, n, 700, I64, 0.1)) for n in (30, 3000, 9000)]
    w = rows_of(g, 700, 264, BF)
    t = (BF, I64, BF)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for turn in range(4):
        for s, p, (dout, tokens) in zip(streams, problems, rows):
            with torch.cuda.stream(s):  # (what the calls' outputs are made on)
                loss = p.forward(s)
                grads = p.backward(lse=loss[1], stream=s)
                got.append((p, loss, grads, dout, tokens, run_embed(w, tokens, t, 2.0, stream=s),
                            run_bwd(dout, tokens, None, 700, (F, I64, BF), 2.0, stream=s)))
    torch.cuda.synchronize()
    for p, loss, grads, dout, tokens, out, dw in got:
        p.lse = loss[1][:p.rows]
        p.check_forward(*loss)
        p.check_backward(*grads)
        check_embed(w, tokens, t, 2.0, out)
        check_bwd(dout, tokens, None, 700, (F, I64, BF), 2.0, dw)


def test_threads_on_one_stream():
    """Threads whose calls need scratch of different sizes, on one stream."""
    torch = T()
    s = torch.cuda.Stream()
    problems = [Problem(rows, 136, vocab, seed=k) for k, (rows, vocab) in enumerate([(40, 900), (300, 2500), (700, 4000)])]
    torch.cuda.synchronize()
    results, errors = [[] for _ in problems], []

    def work(k):
        try:
            with torch.cuda.stream(s):
                for _ in range(6):
                    loss = problems[k].forward(s)
                    results[k].append((loss, problems[k].backward(lse=loss[1], stream=s)))
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(problems))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for p, got in zip(problems, results):
        for loss, grads in got:
            p.lse = loss[1][:p.rows]
            p.check_forward(*loss)
            p.check_backward(*grads)


def test_graphs_after_larger_calls():
    """A graph for each size, smallest first, replayed after the calls that outgrew its
    scratch."""
    torch = T()
    s = torch.cuda.Stream()
    kept = []
    for rows, cols, vocab in ((30, 72, 500), (300, 200, 3000), (1500, 264, 9000)):
        p = Problem(rows, cols, vocab)
        torch.cuda.synchronize()
        loss, lse = p.forward(s)
        (dx, _), (dw, _) = p.backward(lse=lse, stream=s)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            mm.check(mm.mm_cross_entropy(p.x, p.w, p.targets, loss, lse, rows, cols, vocab, cols, cols, (BF, I64, F), s))
            mm.check(mm.mm_cross_entropy_backward(p.x, p.w, p.targets, lse, p.dloss, dx, dw, rows, cols, vocab, cols, cols,
                                                  cols, cols, (BF, I64, BF), s))
        kept.append((graph, p, loss, lse, dx, dw))
    for graph, p, loss, lse, dx, dw in kept + kept[::-1]:
        for o in (loss, lse, dx, dw):
            o.fill_(77)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        p.lse = lse[:p.rows]
        p.check_forward(loss, lse)
        p.check_backward((dx, lambda: None), (dw, lambda: None))


def test_refused_in_a_capture_without_scratch():
    """Refused before anything is launched, at sizes past any scratch the stream has."""
    torch = T()
    p = Problem(3000, 1032, 3001, pads=(0, 1))  # (W is copied)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    loss = torch.full((3000,), 5.0, device="cuda")
    dw = torch.full((3001, 1032), 5.0, device="cuda").bfloat16()
    lse = p.want_lse.float()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        before = mm.mm_get_stats()["launches"]
        a = mm.mm_cross_entropy(p.x, p.w, p.targets, loss, None, 3000, 1032, 3001, p.x.stride(0), p.w.stride(0), (BF, I64, F), s)
        b = mm.mm_cross_entropy_backward(p.x, p.w, p.targets, lse, None, None, dw, 3000, 1032, 3001, p.x.stride(0),
                                         p.w.stride(0), 0, 1032, (BF, I64, BF), s)
        after = mm.mm_get_stats()["launches"]
    assert a == b == mm.MM_ERR_UNSUPPORTED and "capture" in mm.mm_last_error()
    assert after == before
    graph.replay()
    torch.cuda.synchronize()
    assert bool((loss == 5).all()) and bool((dw == 5).all())
