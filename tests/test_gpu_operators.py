"""The operators around a quantised linear layer against their formulas in 64
bits (torch on the GPU's float64), at the sizes, strides and values where they
can go wrong.

Bounds, elementwise, with u the unit roundoff of the output's type and e =
2^-23 (twice an fp32 rounding: sums on tensor cores may truncate):
  a sum of n products     e (n + 16) sum|products|  + u |result|
  statistics of a row     e (n + 16) relative (their terms are not negative)
  4-bit weights, M > 16   + u_A sum|products|  (each weight rounded once to A's type)
  e4m3 values             2^-4 |y| or half the least step, 2^-10 scale, whichever is larger
"""
import math

import pytest

import matmul_selection_gb300 as mm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    assert mm.mm_operator_status() == mm.MM_OK, mm.mm_last_error()

BF, H, F, Q = mm.MM_BF16, mm.MM_F16, mm.MM_F32, mm.MM_E4M3
U = {BF: 2.0 ** -8, H: 2.0 ** -11, F: 2.0 ** -24}
LEAST = {BF: 2.0 ** -133, H: 2.0 ** -24, F: 2.0 ** -149}  # least positive values
E = 2.0 ** -23
EPS = 1e-6


def T():
    import torch
    return torch


def ttype(t):
    torch = T()
    return {BF: torch.bfloat16, H: torch.float16, F: torch.float32, Q: torch.float8_e4m3fn}[t]


def generator(seed):
    g = T().Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows_of(gen, rows, cols, t, pad=0, scale=1.0, offset=0):
    """A rows x cols view of normal values; what lies between the rows, before
    them and after them is NaN."""
    torch = T()
    ld = cols + pad
    flat = torch.full((offset + rows * ld + 64,), float("nan"), dtype=ttype(t), device="cuda")
    v = flat[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    v.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * scale)
    return v


def out_rows(rows, cols, t, pad=0, offset=0):
    """An output view whose surroundings hold a sentinel, and a check of them."""
    torch = T()
    ld = cols + pad
    flat = torch.full((offset + rows * ld + 64,), 77.0, device="cuda").to(ttype(t))
    v = flat[offset:offset + rows * ld].view(rows, ld)[:, :cols]

    def untouched():
        mark = torch.ones(flat.shape, dtype=torch.bool, device="cuda")
        mark[offset:offset + rows * ld].view(rows, ld)[:, :cols] = False
        assert bool((flat.float()[mark] == torch.tensor(77.0).to(ttype(t)).float().item()).all()), \
            "written outside the output"
    return v, untouched


def close(got, want, bound):
    """Every element within its bound; NaN and infinities exactly where wanted."""
    torch = T()
    got, want = got.double(), want.double()
    assert bool((torch.isnan(got) == torch.isnan(want)).all())
    fine = torch.isfinite(want)
    assert bool((got[~fine & ~torch.isnan(want)] == want[~fine & ~torch.isnan(want)]).all())
    err = (got - want).abs()
    bad = fine & ~(err <= bound)
    if bool(bad.any()):
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} outside; first at {i}: "
                             f"{got[tuple(i)].item()} for {want[tuple(i)].item()}, "
                             f"off {err[tuple(i)].item():.3g}, bound "
                             f"{(bound[tuple(i)] if torch.is_tensor(bound) else bound):.3g}")


def e4m3_close(q, scale, y, slack):
    """8-bit values times their scale against y: half a step of e4m3."""
    torch = T()
    step = torch.maximum(y.abs() * 2.0 ** -4, scale.double()[:, None] * 2.0 ** -10)
    close(q.double() * scale.double()[:, None], y, step * (1 + 1e-5) + slack * y.abs())


# ------------------------------------------------------------------ norm

def run_norm(x, residual, w, t, eps=EPS, want_h=True, want_rstd=True, pad=0, offset=0, stream=None):
    torch = T()
    rows, cols = x.shape
    h, h_ok = out_rows(rows, cols, t[0], pad, offset) if want_h else (None, lambda: None)
    y, y_ok = out_rows(rows, cols, t[2], pad, offset)
    scale = torch.empty(rows, device="cuda") if t[2] == Q else None
    rstd = torch.empty(rows, device="cuda") if want_rstd else None
    mm.check(mm.mm_rmsnorm(x, residual, w, h, y, scale, rstd, rows, cols, x.stride(0),
                           residual.stride(0) if residual is not None else 0,
                           h.stride(0) if h is not None else 0, y.stride(0), t, eps, stream))
    torch.cuda.synchronize()
    h_ok()
    y_ok()
    return h, y, scale, rstd


def check_norm(x, residual, w, t, got, eps=EPS):
    h, y, scale, rstd = got
    cols = x.shape[1]
    h64 = x.double() + (residual.double() if residual is not None else 0)
    rstd64 = 1 / (h64.square().mean(1) + eps).sqrt()
    y64 = h64 * rstd64[:, None] * w.double()
    rel = E * (cols + 16)
    if h is not None:
        close(h, h64, U[t[0]] * h64.abs() * (1 + E) + E * h64.abs() + LEAST[t[0]])
    if rstd is not None:
        close(rstd, rstd64, rel * rstd64)
    if t[2] == Q:
        amax = y64.abs().amax(1)
        scale64 = amax / 448
        scale64 = T().where(amax == 0, 1.0, scale64.clamp_min(2.0 ** -126))
        close(scale, scale64, rel * scale64)
        e4m3_close(y, scale, y64, 2 * rel)
    else:
        close(y, y64, (U[t[2]] + rel) * y64.abs() + LEAST[t[2]])


@pytest.mark.parametrize("cols", [1, 2, 7, 8, 31, 64, 100, 255, 1024, 1025, 4096, 4097, 8192, 16384,
                                  16385, 40000, 70001])
@pytest.mark.parametrize("t", [(BF, BF, BF), (BF, BF, Q), (H, F, H), (H, BF, Q), (F, F, F), (F, H, Q),
                               (BF, F, F)])
def test_norm_sizes(cols, t):
    g = generator(cols)
    for rows, pad, residual in ((1, 0, True), (5, 3, True), (3, 8, False)):
        x = rows_of(g, rows, cols, t[0], pad)
        r = rows_of(g, rows, cols, t[0], pad, 2.0) if residual else None
        w = rows_of(g, 1, cols, t[1])[0]
        check_norm(x, r, w, t, run_norm(x, r, w, t, pad=pad, want_h=residual))


@pytest.mark.parametrize("rows", [1, 2, 127, 1000, 4097])
@pytest.mark.parametrize("cols", [33, 512, 1000])
def test_norm_many_rows(rows, cols):
    g = generator(rows + cols)
    for t in ((BF, BF, Q), (F, F, F)):
        x, r = rows_of(g, rows, cols, t[0]), rows_of(g, rows, cols, t[0], 5)
        w = rows_of(g, 1, cols, t[1])[0]
        check_norm(x, r, w, t, run_norm(x, r, w, t))
        check_norm(x, r, w, t, run_norm(x, r, w, t, want_h=False, want_rstd=False))


@pytest.mark.parametrize("offset", [1, 2, 4, 8])
@pytest.mark.parametrize("t", [(BF, BF, Q), (H, H, H), (F, F, F)])
def test_norm_bases_off_16_bytes(offset, t):
    g = generator(offset)
    for cols, pad in ((256, 0), (256, 8), (4096, 0)):
        x = rows_of(g, 4, cols, t[0], pad, offset=offset)
        r = rows_of(g, 4, cols, t[0], pad)
        w = rows_of(g, 1, cols, t[1], offset=1)[0]
        check_norm(x, r, w, t, run_norm(x, r, w, t, pad=pad, offset=offset))


@pytest.mark.parametrize("cols", [1, 9, 14, 15, 16, 23, 24, 30, 31, 37, 129, 257, 263, 300, 511, 520, 601, 1003,
                                  1030, 2051, 4100, 8203, 16387])
@pytest.mark.parametrize("t", [(BF, BF, BF), (BF, F, Q), (H, H, F), (F, F, F), (F, BF, Q)])
def test_norm_rows_that_start_anywhere(cols, t):
    """Every operand at its own offset and row distance."""
    torch = T()
    g = generator(cols)
    rows = 9
    for i, (px, pr, ph, py) in enumerate(((0, 0, 0, 0), (1, 1, 1, 1), (3, 0, 5, 0), (0, 1, 2, 3), (5, 7, 0, 1))):
        x, r = rows_of(g, rows, cols, t[0], px, offset=i), rows_of(g, rows, cols, t[0], pr, 2.0, offset=3 * i)
        w = rows_of(g, 1, cols, t[1], offset=i)[0]
        h, h_ok = out_rows(rows, cols, t[0], ph, 2 * i)
        y, y_ok = out_rows(rows, cols, t[2], py, i)
        scale = torch.empty(rows, device="cuda") if t[2] == Q else None
        rstd = torch.empty(rows, device="cuda")

        def run(x, r, h):
            mm.check(mm.mm_rmsnorm(x, r, w, h, y, scale, rstd, rows, cols, x.stride(0), r.stride(0), h.stride(0),
                                   y.stride(0), t, EPS))
            torch.cuda.synchronize()
            y_ok()
        run(x, r, h)
        h_ok()
        check_norm(x, r, w, t, (h, y, scale, rstd))
        x0, r0 = x.clone(), r.clone()
        run(x, r, x)  # h over x
        check_norm(x0, r0, w, t, (x, y, scale, rstd))
        x.copy_(x0)
        run(x, r, r)  # h over the residual
        check_norm(x0, r0, w, t, (r, y, scale, rstd))


@pytest.mark.parametrize("cols", [64, 4096, 4099, 70001])
def test_norm_in_place(cols):
    torch = T()
    t = (BF, BF, BF)
    g = generator(cols)
    x, r = rows_of(g, 7, cols, BF), rows_of(g, 7, cols, BF)
    w = rows_of(g, 1, cols, BF)[0]
    h0, y0, _, _ = run_norm(x, r, w, t)
    x1, r1 = x.clone(), r.clone()  # h over the residual, y over x
    mm.check(mm.mm_rmsnorm(x1, r1, w, r1, x1, None, None, 7, cols, cols, cols, cols, cols, t, EPS))
    torch.cuda.synchronize()
    assert torch.equal(r1, h0) and torch.equal(x1, y0)


@pytest.mark.parametrize("cols", [48, 4096, 70001])
@pytest.mark.parametrize("t", [(BF, BF, BF), (BF, BF, Q), (F, F, Q)])
def test_norm_odd_values(cols, t):
    """Rows of zeros, tiny and large values, and rows with a NaN or an
    infinity, which stay in their rows."""
    torch = T()
    g = generator(5)
    x = rows_of(g, 8, cols, t[0])
    w = rows_of(g, 1, cols, t[1])[0]
    x[1] = 0
    x[2] *= 1e-18
    x[3] *= 1e15
    x[4, cols // 2] = float("nan")
    x[5, cols // 3] = float("inf")
    h, y, scale, rstd = run_norm(x, None, w, t)
    keep = torch.tensor([0, 1, 2, 3, 6, 7], device="cuda")
    sub = lambda v: None if v is None else v[keep]  # noqa: E731
    check_norm(x[keep], None, w, t, (h[keep], y.float()[keep] if t[2] != Q else y.view(torch.uint8)[keep].view(ttype(Q)),
                                     sub(scale), sub(rstd)))
    assert bool((y[1].float() == 0).all())
    if scale is not None:
        assert scale[1].item() == 1.0 and math.isnan(scale[4].item()) and math.isnan(scale[5].item())
        assert bool(torch.isnan(y[4].float()).all())
    else:
        assert bool(torch.isnan(y[4].float()).all())
        bad = torch.isnan(y[5].float())
        assert int(bad.sum()) == 1 and bool(bad[cols // 3]) and bool((y[5].float()[~bad] == 0).all())
    assert rstd[5].item() == 0.0


def test_norm_weight_with_a_nan_poisons_the_scale():
    t = (BF, BF, Q)
    g = generator(9)
    x, w = rows_of(g, 3, 640, BF), rows_of(g, 1, 640, BF)[0]
    w[639] = float("nan")
    _, y, scale, _ = run_norm(x, None, w, t)
    assert bool(T().isnan(scale).all()) and bool(T().isnan(y.float()).all())


def test_norm_offsets_past_32_bits():
    torch = T()
    cols, ld, rows = 4096, (1 << 30) + 8, 4
    flat = torch.empty(ld * (rows - 1) + cols, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((rows, cols), (ld, 1))
    g = generator(1)
    x.copy_(torch.randn(rows, cols, generator=g, device="cuda"))
    w = rows_of(g, 1, cols, BF)[0]
    t = (BF, BF, BF)
    check_norm(x, None, w, t, run_norm(x, None, w, t))
    dy = rows_of(g, rows, cols, BF)
    check_bwd(dy, None, x, w, t, run_bwd(dy, None, x, w, t))


# ------------------------------------------------------------------ norm, backward

def run_bwd(dy, dh, h, w, t, rstd=None, want_dw=True, pad=0, eps=EPS, stream=None):
    torch = T()
    rows, cols = h.shape
    dx, dx_ok = out_rows(rows, cols, t[0], pad)
    dw, dw_ok = out_rows(1, cols, t[1]) if want_dw else (None, lambda: None)
    mm.check(mm.mm_rmsnorm_backward(dy, dh, h, w, rstd, dx, dw, rows, cols, dy.stride(0),
                                    dh.stride(0) if dh is not None else 0, h.stride(0), dx.stride(0),
                                    t, eps, stream))
    torch.cuda.synchronize()
    dx_ok()
    dw_ok()
    return dx, dw[0] if want_dw else None


def check_bwd(dy, dh, h, w, t, got, rstd=None, eps=EPS):
    dx, dw = got
    rows, cols = h.shape
    h64, dy64, w64 = h.double(), dy.double(), w.double()
    r = 1 / (h64.square().mean(1, keepdim=True) + eps).sqrt() if rstd is None else rstd.double()[:, None]
    g = dy64 * w64
    c = r * r * (g * h64).mean(1, keepdim=True)
    c_abs = r * r * (g * h64).abs().mean(1, keepdim=True)
    d = dh.double() if dh is not None else T().zeros_like(h64)
    want = d + r * (g - h64 * c)
    size = d.abs() + r * (g.abs() + h64.abs() * c_abs)
    close(dx, want, E * 2 * (cols + 16) * size + U[t[0]] * want.abs() + LEAST[t[0]])
    if dw is not None:
        terms = dy64 * h64 * r
        extra = cols + 16 if rstd is None else 4
        close(dw, terms.sum(0), E * (rows + 16 + extra) * terms.abs().sum(0) + U[t[1]] * terms.sum(0).abs()
              + LEAST[t[1]])


@pytest.mark.parametrize("cols", [1, 7, 64, 255, 1000, 1024, 4096, 4097, 8192, 16384, 16385, 40001])
@pytest.mark.parametrize("t", [(BF, BF, BF), (H, F, H), (F, F, F), (BF, F, F), (F, BF, BF)])
def test_bwd_sizes(cols, t):
    g = generator(cols)
    for rows, pad, stream in ((1, 0, True), (5, 3, False), (33, 8, True)):
        dy, h = rows_of(g, rows, cols, t[2], pad), rows_of(g, rows, cols, t[0], pad, 2.0)
        dh = rows_of(g, rows, cols, t[0], pad) if stream else None
        w = rows_of(g, 1, cols, t[1])[0]
        check_bwd(dy, dh, h, w, t, run_bwd(dy, dh, h, w, t, pad=pad))
        rstd = (1 / (h.float().square().mean(1) + EPS).sqrt()).contiguous()
        check_bwd(dy, dh, h, w, t, run_bwd(dy, dh, h, w, t, rstd=rstd, pad=pad), rstd=rstd)


@pytest.mark.parametrize("rows", [2, 151, 1000, 5000])
@pytest.mark.parametrize("cols", [40, 513, 2048])
def test_bwd_many_rows(rows, cols):
    g = generator(rows)
    for t in ((BF, BF, BF), (F, F, F)):
        dy, dh, h = (rows_of(g, rows, cols, t[0]) for _ in range(3))
        w = rows_of(g, 1, cols, t[1])[0]
        got = run_bwd(dy, dh, h, w, t)
        check_bwd(dy, dh, h, w, t, got)
        again = run_bwd(dy, dh, h, w, t)
        assert T().equal(got[0], again[0]) and T().equal(got[1], again[1])
        dx, none = run_bwd(dy, dh, h, w, t, want_dw=False)
        assert none is None and T().equal(dx, got[0])


@pytest.mark.parametrize("cols", [3, 29, 129, 200, 257, 335, 511, 513, 527, 601, 1003, 1039, 2050, 4103, 8199, 16391])
@pytest.mark.parametrize("t", [(BF, BF, BF), (H, F, H), (F, F, F), (F, BF, F)])
def test_bwd_rows_that_start_anywhere(cols, t):
    """Every operand at its own offset and row distance; few rows, and more than
    the grid has blocks."""
    torch = T()
    g = generator(cols)
    for i, (py, pd, ph, px) in enumerate(((0, 0, 0, 0), (1, 1, 1, 1), (3, 3, 3, 0), (0, 5, 2, 7), (1, 0, 0, 3))):
        rows = 3001 if i % 2 and cols < 4200 else 700 if i % 2 else 11
        dy, dh = rows_of(g, rows, cols, t[0], py, offset=i), rows_of(g, rows, cols, t[0], pd, offset=5 * i)
        h = rows_of(g, rows, cols, t[0], ph, 2.0, offset=3 * i)
        w = rows_of(g, 1, cols, t[1], offset=i)[0]
        rstd = (1 / (h.float().square().mean(1) + EPS).sqrt()).contiguous() if i > 1 else None
        check_bwd(dy, dh, h, w, t, run_bwd(dy, dh, h, w, t, rstd=rstd, pad=px), rstd=rstd)
        for over in (dy, dh):  # in place
            kept = dy.clone(), dh.clone()
            dw = torch.empty(cols, dtype=ttype(t[1]), device="cuda")
            mm.check(mm.mm_rmsnorm_backward(dy, dh, h, w, rstd, over, dw, rows, cols, dy.stride(0), dh.stride(0),
                                            h.stride(0), over.stride(0), t, EPS))
            torch.cuda.synchronize()
            check_bwd(*kept, h, w, t, (over, dw), rstd=rstd)
            dy.copy_(kept[0])
            dh.copy_(kept[1])


@pytest.mark.parametrize("cols", [8196, 16400, 30001, 65537, 70001, 131071, 131101])
@pytest.mark.parametrize("rows", [1, 16, 130, 700])
def test_bwd_long_rows(cols, rows):
    """Rows held by several blocks, and longer ones."""
    g = generator(cols + rows)
    for t, pad in (((F, F, F), 0), ((BF, F, BF), 3), ((H, H, H), 8)):
        dy, dh, h = (rows_of(g, rows, cols, t[0], pad) for _ in range(3))
        w = rows_of(g, 1, cols, t[1], offset=1)[0]
        rstd = (1 / (h.float().square().mean(1) + EPS).sqrt()).contiguous() if pad else None
        got = run_bwd(dy, dh, h, w, t, rstd=rstd)
        check_bwd(dy, dh, h, w, t, got, rstd=rstd)
        again = run_bwd(dy, None if rows == 16 else dh, h, w, t, rstd=rstd)
        if rows == 16:
            check_bwd(dy, None, h, w, t, again, rstd=rstd)
        else:
            assert T().equal(got[0], again[0]) and T().equal(got[1], again[1])


def test_bwd_no_rows_writes_zeros():
    torch = T()
    dw = torch.full((100,), 3.0, device="cuda")
    mm.check(mm.mm_rmsnorm_backward(None, None, None, None, None, None, dw, 0, 100, 100, 100, 100, 100,
                                    (F, F, F), EPS))
    torch.cuda.synchronize()
    assert bool((dw == 0).all())


@pytest.mark.parametrize("cols", [128, 4097, 40001])
@pytest.mark.parametrize("over", ["dy", "dh"])
def test_bwd_in_place(cols, over):
    torch = T()
    t = (F, F, F)
    g = generator(cols)
    dy, dh, h = (rows_of(g, 9, cols, F).contiguous() for _ in range(3))
    w = rows_of(g, 1, cols, F)[0]
    dx, dw = run_bwd(dy, dh, h, w, t)
    buf = (dy if over == "dy" else dh).clone()
    a, b = (buf, dh) if over == "dy" else (dy, buf)
    dw1 = torch.empty(cols, device="cuda")
    mm.check(mm.mm_rmsnorm_backward(a, b, h, w, None, buf, dw1, 9, cols, cols, cols, cols, cols, t, EPS))
    torch.cuda.synchronize()
    assert torch.equal(buf, dx) and torch.equal(dw1, dw)


def test_bwd_against_differences():
    """dx and dweight against central differences of the forward formula in
    64 bits: L = sum(dy y) + sum(dh h)."""
    torch = T()
    rows, cols = 3, 24
    g = generator(3)
    t = (F, F, F)
    h, dy, dh = (rows_of(g, rows, cols, F) for _ in range(3))
    w = rows_of(g, 1, cols, F)[0]

    def loss(h64, w64):
        y = h64 * (1 / (h64.square().mean(1, keepdim=True) + EPS).sqrt()) * w64
        return (dy.double() * y).sum() + (dh.double() * h64).sum()

    step = 2.0 ** -13
    dx_num, dw_num = torch.zeros(rows, cols, dtype=torch.float64), torch.zeros(cols, dtype=torch.float64)
    for j in range(cols):
        d = torch.zeros(cols, dtype=torch.float64, device="cuda")
        d[j] = step
        dw_num[j] = (loss(h.double(), w.double() + d) - loss(h.double(), w.double() - d)) / (2 * step)
        for i in range(rows):
            e = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
            e[i, j] = step
            dx_num[i, j] = (loss(h.double() + e, w.double()) - loss(h.double() - e, w.double())) / (2 * step)
    dx, dw = run_bwd(dy, dh, h, w, t)
    # truncation: step^2 / 6 times a third derivative of order 100 at most here; fp32: 1e-5 of values of order 10
    assert (dx.double().cpu() - dx_num).abs().max().item() < 1e-4
    assert (dw.double().cpu() - dw_num).abs().max().item() < 1e-4


# ------------------------------------------------------------------ 4-bit weights

def w4_weights(gen, N, K, group, ts, zeros, ldw=None, pad_s=0, slope=0.01):
    """codes, scales, zeros and the weights' values in 64 bits."""
    torch = T()
    ldw = ldw or (K + 1) // 2 * 2
    groups = -(-K // group)
    q = torch.randint(0, 16, (N, ldw), generator=gen, device="cuda", dtype=torch.uint8)
    codes = q[:, 0::2] | (q[:, 1::2] << 4)
    scales = rows_of(gen, N, groups, ts, pad_s, slope)
    z = None
    if zeros:
        z = torch.full((N, groups + pad_s), 255, dtype=torch.uint8, device="cuda")[:, :groups]
        z.copy_(torch.randint(0, 16, (N, groups), generator=gen, device="cuda"))
    at = torch.arange(K, device="cuda") // group
    w = (q[:, :K].double() - (z.double()[:, at] if zeros else 8)) * scales.double()[:, at]
    return codes.contiguous(), ldw, scales, z, w


def run_w4(a, codes, ldw, scales, z, N, K, group, t, pad=0, stream=None):
    M = a.shape[0]
    out, ok = out_rows(M, N, t[2], pad)
    mm.check(mm.mm_gemm_w4(a, codes, scales, z, out, M, N, K, a.stride(0), ldw, scales.stride(0),
                           out.stride(0), group, t, stream))
    T().cuda.synchronize()
    ok()
    return out


def check_w4(a, w, t, out):
    M, K = a.shape
    want, size = a.double() @ w.t(), a.double().abs() @ w.abs().t()
    exact_weights = M <= 16
    bound = E * (K + 16) * size + U[t[2]] * want.abs() + LEAST[t[2]]
    close(out, want, bound if exact_weights else bound + U[t[0]] * size)


@pytest.mark.parametrize("M", [1, 2, 3, 7, 8, 9, 15, 16, 17, 33, 64, 65, 100, 129, 256, 300])
@pytest.mark.parametrize("N,K,group", [(64, 128, 32), (130, 256, 128), (257, 1000, 64), (65, 4100, 128),
                                       (512, 2048, 64)])
def test_w4_sizes(M, N, K, group):
    g = generator(M + N + K)
    for t, zeros in (((BF, BF, BF), False), ((H, F, F), True)):
        a = rows_of(g, M, K, t[0], 8 if zeros else 0)
        codes, ldw, s, z, w = w4_weights(g, N, K, group, t[1], zeros, (K + 31) // 32 * 32, 1 if zeros else 0)
        check_w4(a, w, t, run_w4(a, codes, ldw, s, z, N, K, group, t, 3 if zeros else 0))


@pytest.mark.parametrize("M", [1, 16, 100, 250, 300])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_long_k(M, group):
    """The rings of the main loops wrap many times; equal calls, equal bits."""
    g = generator(M + group)
    N, K, t = 512, 12288, (BF, BF, BF)
    a = rows_of(g, M, K, BF)
    codes, ldw, s, z, w = w4_weights(g, N, K, group, BF, True)
    first = run_w4(a, codes, ldw, s, z, N, K, group, t)
    check_w4(a, w, t, first)
    for _ in range(8):
        assert T().equal(run_w4(a, codes, ldw, s, z, N, K, group, t), first)


@pytest.mark.parametrize("M", [1, 3, 8, 13, 16])
@pytest.mark.parametrize("N,K,group", [(40009, 300, 32), (40009, 1100, 64), (20011, 2500, 128)])
def test_w4_many_rows_of_weights(M, N, K, group):
    """More tiles than the device holds at a time: a block takes several in turn."""
    g = generator(M + N + K)
    t = (H, F, F) if group == 64 else (BF, BF, BF)
    a = rows_of(g, M, K, t[0])
    codes, ldw, s, z, w = w4_weights(g, N, K, group, t[1], group != 128)
    first = run_w4(a, codes, ldw, s, z, N, K, group, t)
    check_w4(a, w, t, first)
    for _ in range(4):
        assert T().equal(run_w4(a, codes, ldw, s, z, N, K, group, t), first)


@pytest.mark.parametrize("M", [1, 5, 16, 40])
@pytest.mark.parametrize("K", [1, 2, 15, 31, 32, 33, 63, 64, 127, 129, 255, 257])
def test_w4_short_k(M, K):
    g = generator(K)
    for t, group in (((BF, F, F), 32), ((H, H, BF), 64), ((BF, BF, BF), 128)):
        a = rows_of(g, M, K, t[0], 1)
        codes, ldw, s, z, w = w4_weights(g, 37, K, group, t[1], True)
        check_w4(a, w, t, run_w4(a, codes, ldw, s, z, 37, K, group, t))


@pytest.mark.parametrize("M", [1, 16, 48])
@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 63, 127, 128, 129])
def test_w4_few_columns(M, N):
    g = generator(N)
    t = (BF, H, BF)
    a = rows_of(g, M, 1024, BF)
    codes, ldw, s, z, w = w4_weights(g, N, 1024, 64, H, True)
    check_w4(a, w, t, run_w4(a, codes, ldw, s, z, N, 1024, 64, t))


@pytest.mark.parametrize("M", [1, 9, 50])
@pytest.mark.parametrize("shift,pad,byte", [(0, 1, 0), (1, 0, 0), (3, 4, 1), (4, 4, 3), (8, 8, 8)])
def test_w4_alignments(M, shift, pad, byte):
    """Rows of A and of the codes that start anywhere."""
    torch = T()
    g = generator(shift + byte)
    N, K, group, t = 100, 512, 64, (BF, BF, BF)
    a = rows_of(g, M, K, BF, pad, offset=shift)
    codes, ldw, s, z, w = w4_weights(g, N, K, group, BF, True, K + 2 * byte)
    flat = torch.zeros(codes.numel() + 64, dtype=torch.uint8, device="cuda")
    moved = flat[byte:byte + codes.numel()].view(codes.shape)
    moved.copy_(codes)
    check_w4(a, w, t, run_w4(a, moved, ldw, s, z, N, K, group, t, pad))


@pytest.mark.parametrize("M", [1, 16, 20])
def test_w4_values(M):
    """Each code and zero point on its own, with A and scales that make the
    results whole numbers: equal, not near."""
    torch = T()
    N, K, group, t = 16 * 16, 64, 32, (BF, F, F)
    q = torch.arange(N, device="cuda") % 16
    z = (torch.arange(N, device="cuda") // 16).to(torch.uint8)[:, None].expand(N, 2).contiguous()
    codes = (q | (q << 4)).to(torch.uint8)[:, None].expand(N, K // 2).contiguous()
    scales = torch.tensor([1.0, 4.0], device="cuda").expand(N, 2).contiguous()
    a = torch.randint(-4, 5, (M, K), generator=generator(2), device="cuda").to(torch.bfloat16)
    out = run_w4(a, codes, K, scales, z, N, K, group, t)
    w = (q.double() - z[:, 0].double())
    want = (a.double()[:, :32].sum(1)[:, None] + 4 * a.double()[:, 32:].sum(1)[:, None]) * w
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("M", [1, 40])
def test_w4_nothing_past_k_is_used(M):
    """K ends inside a group; A's padding is NaN, codes past K are arbitrary;
    an infinity in A reaches its own row only."""
    torch = T()
    g = generator(11)
    N, K, group, t = 70, 130, 128, (BF, BF, F)
    a = rows_of(g, M, K, BF, 126)
    codes, ldw, s, z, w = w4_weights(g, N, K, group, BF, False, 256)
    out = run_w4(a, codes, ldw, s, z, N, K, group, t)
    check_w4(a, w, t, out)
    if M > 1:
        a[3, 5] = float("inf")
        w[7] = w[7]
        out2 = run_w4(a, codes, ldw, s, z, N, K, group, t)
        rest = [i for i in range(M) if i != 3]
        assert torch.equal(out2[rest], out[rest])
        assert not bool(torch.isfinite(out2[3][w[:, 5] != 0]).any())


def test_w4_offsets_past_32_bits():
    torch = T()
    N, K, group, t = 3, 256, 64, (BF, BF, BF)
    g = generator(4)
    small, _, s, z, w = w4_weights(g, N, K, group, BF, True)
    ldw = (1 << 32) + 64
    flat = torch.empty(ldw // 2 * (N - 1) + K // 2, dtype=torch.uint8, device="cuda")
    codes = flat.as_strided((N, K // 2), (ldw // 2, 1))
    codes.copy_(small)
    for M in (1, 30):
        a = rows_of(g, M, K, BF)
        check_w4(a, w, t, run_w4(a, codes, ldw, s, z, N, K, group, t))


def test_w4_k_zero_writes_zeros():
    torch = T()
    out = torch.full((5, 40), 7.0, device="cuda")
    mm.check(mm.mm_gemm_w4(None, None, None, None, out, 5, 40, 0, 0, 0, 0, 40, 64, (BF, BF, F)))
    torch.cuda.synchronize()
    assert bool((out == 0).all())


# ------------------------------------------------------------------ 8-bit products

def q8_rows(gen, rows, cols, pad=0, offset=0, scale=30.0):
    """e4m3 rows among NaN bytes."""
    torch = T()
    ld = cols + pad
    flat = torch.full((offset + rows * ld + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    v = flat[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    x = (torch.randn(rows, cols, generator=gen, device="cuda") * scale).clamp(-448, 448)
    v.copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
    return v.view(torch.float8_e4m3fn)


def run_q8(a, b, sa, sb, tc, pad=0, stream=None):
    M, K = a.shape
    N = b.shape[0]
    out, ok = out_rows(M, N, tc, pad)
    mm.check(mm.mm_gemm_q8(a, b, sa, sb, out, M, N, K, a.stride(0), b.stride(0), out.stride(0),
                           (Q, Q, tc), stream))
    T().cuda.synchronize()
    ok()
    return out


def check_q8(a, b, sa, sb, tc, out):
    one = T().ones(1, dtype=T().float64, device="cuda")
    s = (sa.double() if sa is not None else one)[:, None] * (sb.double() if sb is not None else one)
    want = (a.double() @ b.double().t()) * s
    size = (a.double().abs() @ b.double().abs().t()) * s.abs()
    close(out, want, E * (a.shape[1] + 16) * size + U[tc] * want.abs() + LEAST[tc])


def q8_scales(gen, n):
    return T().rand(n, generator=gen, device="cuda") * 0.01 + 0.001


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 255, 257, 300, 520])
@pytest.mark.parametrize("N,K", [(64, 128), (130, 256), (257, 1040), (65, 4112), (768, 512), (1000, 100)])
def test_q8_sizes(M, N, K):
    g = generator(M + N + K)
    for tc, pad in ((BF, 0), (F, 3)):
        a, b = q8_rows(g, M, K, -K % 16), q8_rows(g, N, K, -K % 16)
        sa, sb = q8_scales(g, M), q8_scales(g, N)
        check_q8(a, b, sa, sb, tc, run_q8(a, b, sa, sb, tc, pad))


@pytest.mark.parametrize("M", [1, 2, 4, 8])
@pytest.mark.parametrize("N,K", [(6100, 130), (6144, 2064), (5000, 900)])
def test_q8_many_rows_of_weights(M, N, K):
    """More tiles than the device holds at a time: a block takes several in turn."""
    g = generator(M + N + K)
    a, b = q8_rows(g, M, K), q8_rows(g, N, K)
    sa, sb = q8_scales(g, M), q8_scales(g, N)
    check_q8(a, b, sa, sb, F, run_q8(a, b, sa, sb, F))


@pytest.mark.parametrize("N", [2041, 2046, 2048, 2049, 2051, 2175])
@pytest.mark.parametrize("tc", [BF, H, F])
def test_q8_many_rows_that_end_anywhere(N, tc):
    """Rows of the output that start on any element, many tiles of them."""
    g = generator(N)
    M, K = 2311, 208
    a, b = q8_rows(g, M, K), q8_rows(g, N, K)
    sa, sb = q8_scales(g, M), q8_scales(g, N)
    for pad in (0, 1, 2):
        check_q8(a, b, sa, sb, tc, run_q8(a, b, sa, sb, tc, pad))


@pytest.mark.parametrize("M", [1, 12, 70, 300])
@pytest.mark.parametrize("K", [1, 3, 16, 31, 32, 33, 127, 129, 257])
def test_q8_short_k(M, K):
    g = generator(K)
    a, b = q8_rows(g, M, K, -K % 16), q8_rows(g, 90, K, -K % 16)
    check_q8(a, b, None, None, F, run_q8(a, b, None, None, F))


@pytest.mark.parametrize("M", [1, 16, 130])
@pytest.mark.parametrize("N", [1, 2, 15, 17, 127, 129, 255])
def test_q8_few_columns(M, N):
    g = generator(N)
    a, b = q8_rows(g, M, 640), q8_rows(g, N, 640)
    sa, sb = q8_scales(g, M), q8_scales(g, N)
    check_q8(a, b, sa, None, H, run_q8(a, b, sa, None, H))
    check_q8(a, b, None, sb, BF, run_q8(a, b, None, sb, BF, 1))


@pytest.mark.parametrize("M", [1, 9, 50, 200])
@pytest.mark.parametrize("shift_a,shift_b,pad_a,pad_b", [(1, 0, 0, 0), (0, 8, 0, 0), (0, 0, 1, 0),
                                                         (0, 0, 0, 4), (3, 5, 7, 9), (0, 0, 100, 100)])
def test_q8_alignments(M, shift_a, shift_b, pad_a, pad_b):
    g = generator(M)
    a, b = q8_rows(g, M, 512, pad_a, shift_a), q8_rows(g, 200, 512, pad_b, shift_b)
    sa, sb = q8_scales(g, M), q8_scales(g, 200)
    check_q8(a, b, sa, sb, BF, run_q8(a, b, sa, sb, BF))


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_q8_every_value(M):
    """Each finite e4m3 value times small powers of two: equal, not near."""
    torch = T()
    v = torch.arange(256, dtype=torch.uint8, device="cuda")
    v = v[(v & 0x7F) != 0x7F]
    N, K = v.numel(), 128
    b = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
    b[:, 77] = v
    a = torch.zeros(M, K, device="cuda")
    a[:, 77] = 2.0 ** (torch.arange(M, device="cuda") % 4)
    out = run_q8(a.to(torch.float8_e4m3fn), b.view(torch.float8_e4m3fn), None, None, F)
    want = v.view(torch.float8_e4m3fn).double() * a[:, 77:78].double()
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("M", [2, 40, 300])
def test_q8_nan_stays_in_its_row(M):
    torch = T()
    g = generator(6)
    a, b = q8_rows(g, M, 256), q8_rows(g, 100, 256)
    out = run_q8(a, b, None, None, F)
    a.view(torch.uint8)[1, 100] = 0x7F
    out2 = run_q8(a, b, None, None, F)
    rest = [i for i in range(M) if i != 1]
    assert torch.equal(out2[rest], out[rest]) and bool(torch.isnan(out2[1]).all())


def test_q8_large_k():
    g = generator(8)
    for M in (1, 16, 100, 256):
        a, b = q8_rows(g, M, 65536, scale=1.0), q8_rows(g, 128, 65536, scale=1.0)
        check_q8(a, b, None, None, F, run_q8(a, b, None, None, F))


def test_q8_offsets_past_32_bits():
    torch = T()
    g = generator(4)
    N, K, ld = 5, 256, (1 << 30) + 16
    flat = torch.empty(ld * (N - 1) + K, dtype=torch.uint8, device="cuda")
    b = flat.as_strided((N, K), (ld, 1))
    b.copy_(q8_rows(g, N, K).view(torch.uint8))
    b = b.view(torch.float8_e4m3fn)
    for M in (1, 30, 200):
        a = q8_rows(g, M, K)
        check_q8(a, b, None, None, BF, run_q8(a, b, None, None, BF))


def test_q8_k_zero_writes_zeros():
    torch = T()
    out = torch.full((5, 40), 7.0, device="cuda")
    mm.check(mm.mm_gemm_q8(None, None, None, None, out, 5, 40, 0, 0, 0, 40, (Q, Q, F)))
    torch.cuda.synchronize()
    assert bool((out == 0).all())


# ------------------------------------------------------------------ streams, graphs, calls in a row

def one_of_each(g):
    """(call(stream), outputs) of each operator, inputs made once."""
    torch = T()
    todo = []
    x, r = rows_of(g, 64, 1000, BF), rows_of(g, 64, 1000, BF)
    w = rows_of(g, 1, 1000, BF)[0]
    y, h = torch.empty(64, 1000, dtype=ttype(Q), device="cuda"), torch.empty(64, 1000, dtype=ttype(BF), device="cuda")
    sc, rs = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    todo.append((lambda s: mm.mm_rmsnorm(x, r, w, h, y, sc, rs, 64, 1000, 1000, 1000, 1000, 1000,
                                         (BF, BF, Q), EPS, s), [y, h, sc, rs]))
    dx, dw = torch.empty_like(h), torch.empty(1000, dtype=ttype(BF), device="cuda")
    todo.append((lambda s: mm.mm_rmsnorm_backward(x, None, r, w, None, dx, dw, 64, 1000, 1000, 1000, 1000,
                                                  1000, (BF, BF, BF), EPS, s), [dx, dw]))
    for M in (1, 8, 16, 100, 700):
        a = rows_of(g, M, 2048, BF)
        codes, ldw, s4, z, _ = w4_weights(g, 400, 2048, 64, BF, True)
        o = torch.empty(M, 400, dtype=ttype(BF), device="cuda")
        todo.append((lambda s, M=M, a=a, codes=codes, ldw=ldw, s4=s4, z=z, o=o: mm.mm_gemm_w4(
            a, codes, s4, z, o, M, 400, 2048, 2048, ldw, s4.stride(0), 400, 64, (BF, BF, BF), s), [o]))
        qa, qb = q8_rows(g, M, 2048), q8_rows(g, 400, 2048)
        o8 = torch.empty(M, 400, dtype=ttype(BF), device="cuda")
        todo.append((lambda s, M=M, qa=qa, qb=qb, o8=o8: mm.mm_gemm_q8(
            qa, qb, None, None, o8, M, 400, 2048, 2048, 2048, 400, (Q, Q, BF), s), [o8]))
    return todo


def bits(outs):
    return [o.clone().view(T().uint8) for o in outs]


def test_other_streams_and_repeats_give_the_same_bits():
    torch = T()
    todo = one_of_each(generator(21))
    torch.cuda.synchronize()
    want = []
    for call, outs in todo:
        mm.check(call(None))
        torch.cuda.synchronize()
        want.append(bits(outs))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rnd in range(3):
        for s in streams:
            for _, outs in todo:
                for o in outs:
                    o.view(torch.uint8).fill_(0xEE)
            torch.cuda.synchronize()
            for call, _ in todo:  # back to back, nothing waits between
                mm.check(call(s))
            s.synchronize()
            for (_, outs), w in zip(todo, want):
                assert all(torch.equal(a, b) for a, b in zip(bits(outs), w))


def test_graph_capture_and_replay():
    torch = T()
    todo = one_of_each(generator(22))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call, _ in todo:  # scratch is allocated before the capture
        mm.check(call(s))
    s.synchronize()
    want = [bits(outs) for _, outs in todo]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for call, _ in todo:
            mm.check(call(s))
    for _ in range(2):
        for _, outs in todo:
            for o in outs:
                o.view(torch.uint8).fill_(0xEE)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for (_, outs), w in zip(todo, want):
            assert all(torch.equal(a, b) for a, b in zip(bits(outs), w))


def test_kernels_are_the_librarys_own():
    """Each call launches kernels of the library."""
    for call, _ in one_of_each(generator(23)):
        before = mm.mm_get_stats()["launches"]
        mm.check(call(None))
        assert mm.mm_get_stats()["launches"] > before
    T().cuda.synchronize()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("tokens", [1, 16, 200])
def test_example_runs_the_operators_together(tokens):
    """examples/quantised_layer.py against its plain form.  The serving step
    rounds its activations to e4m3 (2^-4 at most a value, about 2.6e-2 in the
    mean square) and three times to bf16; the training step rounds twice to
    bf16 before each gradient (2^-8 a value at most, each)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "quantised_layer.py")
    spec = importlib.util.spec_from_file_location("quantised_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for name, rel in example.run(tokens, 1024, 2048).items():
        bound = 2.0 ** -8 if name == "residual stream" else 2.0 ** -4 if "quantised" in name else 3 * 2.0 ** -8
        assert rel <= bound, (name, rel)
