"""What the operators around a quantised linear layer are measured on.

Four operators, reached as a user reaches them (``own`` true) or computed in
their plain form (``own`` false: elementary torch operations in 32 bits,
rounded once at the end):

  norm      h = x + residual;  rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd w,
            y rounded to its type, or held in 8 bits (e4m3) with one scale a
            row: scale = max|y| / 448, q = e4m3(y / scale)
  norm_bwd  the gradients of y = h rstd w: g = dy w,
            dx = dh + rstd (g - h rstd^2 mean(g h)),  dw = sum over rows of
            dy h rstd  (dh: the gradient that reaches h past the norm)
  w4        out[m, n] = sum_k a[m, k] s[n, k / group] (q[n, k] - z[n, k / group]),
            q four-bit codes, two to a byte along k, the even k in the low
            half; z four-bit zero points, 8 where there are none
  q8        out[m, n] = sa[m] sb[n] sum_k a[m, k] b[n, k], a and b e4m3
"""
import math

import torch

own = False

if torch.cuda.is_available():
    DEVICE = "cuda"
else:
    DEVICE = "cpu"

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn}
CODE = {"bf16": 0, "f16": 1, "f32": 2, "e4m3": 3}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases

def _norm(rows, cols, x, w, y, residual=True, pad=0, **more):
    return dict(op="norm", rows=rows, cols=cols, x=x, w=w, y=y, residual=residual, pad=pad, **more)


def _norm_bwd(rows, cols, x, w, dy, stream=True, pad=0, **more):
    return dict(op="norm_bwd", rows=rows, cols=cols, x=x, w=w, dy=dy, stream=stream, pad=pad, **more)


def _w4(M, N, K, group, x, s, zeros, pad=0, **more):
    return dict(op="w4", M=M, N=N, K=K, group=group, x=x, s=s, zeros=zeros, pad=pad, **more)


def _q8(M, N, K, out, **more):
    return dict(op="q8", M=M, N=N, K=K, out=out, **more)


def listed():
    return [
        # one token of a decode step in front of an 8-bit product: latency
        _norm(1, 4096, "bf16", "bf16", "e4m3", name="norm_q8_decode_1x4096"),
        # a long prompt (or a large batch of them) in front of an 8-bit product
        _norm(8192, 4096, "bf16", "bf16", "e4m3", name="norm_q8_prefill_8192x4096"),
        # a ragged batch whose rows are views of wider ones, 16-bit output, the
        # weights kept in 32 bits: odd sizes, nothing 16-byte aligned
        _norm(1000, 4097, "f16", "f32", "f16", pad=3, name="norm_f16_ragged_1000x4097"),
        # the backward pass of a training step
        _norm_bwd(8192, 4096, "bf16", "bf16", "bf16", name="norm_bwd_8192x4096"),
        # the backward pass of few long rows in 32 bits, odd sizes
        _norm_bwd(127, 16385, "f32", "f32", "f32", stream=False, name="norm_bwd_f32_127x16385"),
        # one token through 4-bit weights
        _w4(1, 4096, 4096, 128, "bf16", "bf16", False, name="w4_decode_1x4096x4096"),
        # a small batch of tokens through large 4-bit weights with zero points
        _w4(16, 16384, 8192, 64, "f16", "f16", True, name="w4_batch_16x16384x8192"),
        # odd sizes: K ends inside a group, N inside any tile, padded rows of A
        _w4(5, 1001, 4100, 32, "bf16", "f32", True, pad=4, name="w4_ragged_5x1001x4100"),
        # a prompt through 4-bit weights
        _w4(1000, 4096, 4096, 128, "bf16", "bf16", False, name="w4_prefill_1000x4096x4096"),
        # one token through 8-bit weights
        _q8(1, 4096, 4096, "bf16", name="q8_decode_1x4096x4096"),
        # a ragged prompt through 8-bit weights
        _q8(127, 4097, 4100, "f16", name="q8_ragged_127x4097x4100"),
        # a large batch of prompts through large 8-bit weights
        _q8(8192, 8192, 8192, "bf16", name="q8_prefill_8192x8192x8192"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _round_or_odd(rng, n):
    """A layer's size near n: a multiple of 160 mostly, else odd."""
    return max(160, n // 160 * 160) if rng.random() < 0.6 else n | 1


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "w4", "q8"])
    if op in ("norm", "norm_bwd"):
        cols = _log(rng, 64, 16385)
        rows = min(_log(rng, 1, 8192), 8192 * 4096 // (cols + 1))
        cols = _round_or_odd(rng, cols)
        x, w = rng.choice(["bf16", "f16", "f32"]), rng.choice(["bf16", "f16", "f32"])
        pad = rng.choice([0, 0, 3, 8])
        if op == "norm":
            return _norm(rows, cols, x, w, rng.choice(["e4m3", "e4m3", x]), rng.random() < 0.7, pad)
        return _norm_bwd(rows, cols, x, w, x, rng.random() < 0.7, pad)
    N, K = _round_or_odd(rng, _log(rng, 64, 16384)), _round_or_odd(rng, _log(rng, 64, 16384))
    if op == "w4":
        M = _log(rng, 1, 4096)
        M = max(1, min(M, (1 << 36) // (N * K)))
        x = rng.choice(["bf16", "f16"])
        return _w4(M, N, K, rng.choice([32, 64, 128]), x, rng.choice([x, "f32"]),
                   rng.random() < 0.5, rng.choice([0, 0, 4, 8]))
    M = _log(rng, 1, 8192)
    M = max(1, min(M, (1 << 38) // (N * K)))
    return _q8(M, N, K, rng.choice(["bf16", "f16"]))


def _up(n, m):
    return -(-n // m) * m


def work(case):
    c = case
    if c["op"] in ("norm", "norm_bwd"):
        n = c["rows"] * c["cols"]
        if c["op"] == "norm":
            e = SIZE[c["x"]] * (3 if c["residual"] else 1) + SIZE[c["y"]]
            stats = 8 if c["y"] == "e4m3" else 4
            return {"bytes": n * e + c["cols"] * SIZE[c["w"]] + c["rows"] * stats, "flops": 6 * n}
        e = SIZE[c["x"]] * (3 if c["stream"] else 2) + SIZE[c["dy"]]
        return {"bytes": n * e + 2 * c["cols"] * SIZE[c["w"]] + 4 * c["rows"], "flops": 10 * n}
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] == "w4":
        groups = _up(K, c["group"]) // c["group"]
        weights = N * _up(K, 2) // 2 + N * groups * (SIZE[c["s"]] + (1 if c["zeros"] else 0))
        return {"bytes": weights + (M * K + M * N) * SIZE[c["x"]], "flops": 2 * M * N * K}
    return {"bytes": M * K + N * K + 4 * (M + N) + M * N * SIZE[c["out"]], "flops": 2 * M * N * K}


# ------------------------------------------------------------------ the inputs

def _wide(rows, cols, pad, dtype):
    """A rows x cols view of rows that are cols + pad apart."""
    return torch.empty(rows, cols + pad, dtype=dtype, device=DEVICE)[:, :cols]


def _normal(gen, rows, cols, pad, dtype, scale=1.0):
    v = _wide(rows, cols, pad, dtype)
    v.copy_(torch.randn(rows, cols, generator=gen, device=DEVICE) * scale)
    return v


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    s = dict(c)
    if own:
        import matmul_selection_gb300 as mm
        s["mm"] = mm
    if c["op"] in ("norm", "norm_bwd"):
        rows, cols, pad = c["rows"], c["cols"], c["pad"]
        tx, tw = TYPES[c["x"]], TYPES[c["w"]]
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=gen, device=DEVICE)).to(tw)
        if c["op"] == "norm":
            s["xin"] = _normal(gen, rows, cols, pad, tx)
            # the residual stream: a few channels are many times the others
            s["res"] = s["h"] = None
            if c["residual"]:
                s["res"] = _normal(gen, rows, cols, pad, tx, 2.0)
                s["res"][:, torch.randint(0, cols, (4,), generator=gen, device=DEVICE)] *= 20
                s["h"] = torch.empty(rows, cols, dtype=tx, device=DEVICE)
            s["out"] = torch.empty(rows, cols, dtype=TYPES[c["y"]], device=DEVICE)
            s["rstd"] = torch.empty(rows, dtype=torch.float32, device=DEVICE)
            s["scale"] = (torch.empty(rows, dtype=torch.float32, device=DEVICE)
                          if c["y"] == "e4m3" else None)
        else:
            s["h"] = _normal(gen, rows, cols, pad, tx, 2.0)
            s["dyin"] = _normal(gen, rows, cols, pad, TYPES[c["dy"]])
            s["dh"] = _normal(gen, rows, cols, pad, tx) if c["stream"] else None
            # as the forward pass left it
            s["rstd"] = 1 / (s["h"].float().square().mean(1) + EPS).sqrt()
            s["dx"] = torch.empty(rows, cols, dtype=tx, device=DEVICE)
            s["dweight"] = torch.empty(cols, dtype=tw, device=DEVICE)
        return s
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] == "w4":
        groups, ldw = _up(K, c["group"]) // c["group"], _up(K, 32)
        s["a"] = _normal(gen, M, K, c["pad"], TYPES[c["x"]])
        s["codes"] = torch.empty(N, ldw // 2, dtype=torch.uint8, device=DEVICE)
        rows = max(1, (1 << 26) // ldw)
        for n in range(0, N, rows):  # bell-shaped codes, a slice of rows at a time
            e = torch.randn(min(rows, N - n), ldw, generator=gen, device=DEVICE)
            e = (e * 2.7 + 8).round_().clamp_(0, 15).to(torch.uint8)
            s["codes"][n:n + rows] = e[:, 0::2] | (e[:, 1::2] << 4)
        v = torch.rand(N, groups, generator=gen, device=DEVICE)
        s["scales"] = ((0.5 + v) * 0.01).to(TYPES[c["s"]])
        s["zeros"] = None
        if c["zeros"]:
            s["zeros"] = torch.randint(6, 11, (N, groups), generator=gen, device=DEVICE).to(torch.uint8)
        s["out_type"] = c["x"]
    else:
        ld = _up(K, 16)  # rows start on 16 bytes, as 8-bit rows are kept
        a = torch.randn(M, ld, generator=gen, device=DEVICE)
        s["sa"] = a[:, :K].abs().amax(1) / E4M3_MAX
        s["a"] = (a / s["sa"][:, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(TYPES["e4m3"])[:, :K]
        b = torch.randn(N, ld, generator=gen, device=DEVICE) * 0.02
        s["sb"] = b[:, :K].abs().amax(1) / E4M3_MAX
        s["b"] = (b / s["sb"][:, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(TYPES["e4m3"])[:, :K]
        s["out_type"] = c["out"]
    s["out"] = torch.empty(M, N, dtype=TYPES[s["out_type"]], device=DEVICE)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _own_norm(s):
    mm, x, r, h, y = s["mm"], s["xin"], s["res"], s["h"], s["out"]
    mm.check(mm.mm_rmsnorm(x, r, s["weight"], h, y, s["scale"], s["rstd"], s["rows"], s["cols"],
                           x.stride(0), r.stride(0) if r is not None else 0,
                           h.stride(0) if h is not None else 0, y.stride(0),
                           (CODE[s["x"]], CODE[s["w"]], CODE[s["y"]]), EPS))
    return {"y": y, "h": h, "scale": s["scale"], "rstd": s["rstd"]}


def _plain_norm(s):
    h = s["xin"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    rstd = 1 / ((h * h).mean(1) + EPS).sqrt()
    y = h * rstd[:, None] * s["weight"].float()
    scale = None
    if s["scale"] is not None:
        amax = y.abs().amax(1)
        scale = torch.where(amax == 0, torch.ones_like(amax), amax / E4M3_MAX)
        y = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return {"y": y.to(s["out"].dtype), "h": None if s["res"] is None else h.to(s["xin"].dtype),
            "scale": scale, "rstd": rstd}


def _own_norm_bwd(s):
    mm, dy, dh, h, dx = s["mm"], s["dyin"], s["dh"], s["h"], s["dx"]
    mm.check(mm.mm_rmsnorm_backward(dy, dh, h, s["weight"], s["rstd"], dx, s["dweight"], s["rows"],
                                    s["cols"], dy.stride(0), dh.stride(0) if dh is not None else 0,
                                    h.stride(0), dx.stride(0),
                                    (CODE[s["x"]], CODE[s["w"]], CODE[s["dy"]]), EPS))
    return {"dx": dx, "dweight": s["dweight"]}


def _plain_norm_bwd(s):
    dy, h, rstd = s["dyin"].float(), s["h"].float(), s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = rstd * (g - h * (rstd * rstd * (g * h).mean(1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    dweight = (dy * h * rstd).sum(0)
    return {"dx": dx.to(s["h"].dtype), "dweight": dweight.to(s["weight"].dtype)}


def _own_w4(s):
    mm, a, out, t = s["mm"], s["a"], s["out"], CODE[s["x"]]
    mm.check(mm.mm_gemm_w4(a, s["codes"], s["scales"], s["zeros"], out, s["M"], s["N"], s["K"],
                           a.stride(0), 2 * s["codes"].stride(0), s["scales"].stride(0),
                           out.stride(0), s["group"], (t, CODE[s["s"]], t)))
    return out


def _plain_w4(s):
    K, group = s["K"], s["group"]
    q = torch.stack([s["codes"] & 15, s["codes"] >> 4], 2).flatten(1)[:, :K].float()
    at = torch.arange(K, device=q.device) // group
    z = s["zeros"].float()[:, at] if s["zeros"] is not None else 8.0
    w = (q - z) * s["scales"].float()[:, at]
    return (s["a"].float() @ w.t()).to(s["out"].dtype)


def _own_q8(s):
    mm, a, b, out = s["mm"], s["a"], s["b"], s["out"]
    mm.check(mm.mm_gemm_q8(a, b, s["sa"], s["sb"], out, s["M"], s["N"], s["K"], a.stride(0),
                           b.stride(0), out.stride(0), (3, 3, CODE[s["out_type"]])))
    return out


def _plain_q8(s):
    acc = s["a"].float() @ s["b"].float().t()
    return (acc * s["sa"][:, None] * s["sb"]).to(s["out"].dtype)


_OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "w4": _own_w4, "q8": _own_q8}
_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "w4": _plain_w4, "q8": _plain_q8}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["xin"].double()
        if s["res"] is not None:
            h = torch.add(h, s["res"].double())
        length = torch.einsum("rc,rc->r", h, h) / case["cols"] + EPS
        rstd = torch.pow(length, -0.5)
        y = torch.einsum("rc,r,c->rc", h, rstd, s["weight"].double())
        scale = None
        if case["y"] == "e4m3":
            scale = torch.linalg.vector_norm(y, ord=float("inf"), dim=1) / E4M3_MAX
            y = torch.einsum("rc,r->rc", y, torch.reciprocal(scale))
        return {"y": y, "h": h if s["res"] is not None else None, "scale": scale, "rstd": rstd}
    if op == "norm_bwd":
        h, dy, w = s["h"].double(), s["dyin"].double(), s["weight"].double()
        rstd = s["rstd"].double()
        unit = torch.einsum("rc,r->rc", h, rstd)  # h at length one
        along = torch.einsum("rc,c,rc->r", dy, w, unit) / case["cols"]
        dx = torch.einsum("rc,c,r->rc", dy, w, rstd) - torch.einsum("rc,r,r->rc", unit, along, rstd)
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, unit)}
    M, N, K = case["M"], case["N"], case["K"]
    out = torch.empty(M, N, dtype=torch.float64, device=DEVICE)
    rows = max(1, (1 << 26) // K)
    if op == "w4":
        group, groups = case["group"], s["scales"].shape[1]
        a = torch.zeros(M, groups * group, dtype=torch.float64, device=DEVICE)
        a[:, :K] = s["a"]
        for n in range(0, N, rows):
            q = torch.zeros(min(rows, N - n), groups * group, dtype=torch.float64, device=DEVICE)
            b = s["codes"][n:n + rows].int()
            q[:, 0:K:2] = (b % 16)[:, :(K + 1) // 2].double()
            q[:, 1:K:2] = torch.div(b, 16, rounding_mode="floor")[:, :K // 2].double()
            q = q.view(-1, groups, group)
            zero = 8.0 if s["zeros"] is None else s["zeros"][n:n + rows, :, None].double()
            w = torch.mul(torch.sub(q, zero), s["scales"][n:n + rows, :, None].double())
            out[:, n:n + rows] = torch.einsum("mk,nk->mn", a, w.flatten(1))
        return out
    a = torch.mul(s["a"].double(), s["sa"].double()[:, None])
    for n in range(0, N, rows):
        b = torch.mul(s["b"][n:n + rows].double(), s["sb"][n:n + rows, None].double())
        out[:, n:n + rows] = torch.einsum("mk,nk->mn", a, b)
    return out
