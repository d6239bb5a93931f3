"""What the two ends of a language model are measured on: the lookup of its
tokens' rows and the loss over its vocabulary, each with its gradient.

Four operators, reached as a user reaches them (``own`` true) or computed in
their plain form (``own`` false: elementary torch operations in 32 bits,
rounded once at the end).  W has a row of C values for each of V tokens:

  embed      out[t] = scale W[token[t]]
  embed_bwd  dW[v] = base[v] + scale sum over {t: token[t] = v} of dout[t]
             (base: the gradient that reaches W from elsewhere, or none)
  loss       l[t, v] = sum_c x[t, c] W[v, c];  lse[t] = log sum_v exp l[t, v];
             loss[t] = lse[t] - l[t, target[t]]
  loss_bwd   g[t, v] = dloss[t] (exp(l[t, v] - lse[t]) - [v = target[t]]),
             dx = g W,  dW = g^T x

A token or target outside 0 .. V - 1 stands for none (padding, a prompt that is
not trained on): its row of out, loss, lse and dx is zero, and it adds nothing
to dW.
"""
import math

import torch

own = False

if torch.cuda.is_available():
    DEVICE = "cuda"
else:
    DEVICE = "cpu"

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
         "i32": torch.int32, "i64": torch.int64}
CODE = {"bf16": 0, "f16": 1, "f32": 2, "i32": 4, "i64": 5}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "i32": 4, "i64": 8}
NONE = -100  # the target of a position that is not trained on


# ------------------------------------------------------------------ the cases

def _embed(T, C, V, w, out, index="i64", none=0.0, pad=0, **more):
    return dict(op="embed", T=T, C=C, V=V, w=w, out=out, index=index, none=none, pad=pad, **more)


def _embed_bwd(T, C, V, dw, dout, index="i64", none=0.0, pad=0, base=False, **more):
    return dict(op="embed_bwd", T=T, C=C, V=V, dw=dw, dout=dout, index=index, none=none, pad=pad,
                base=base, **more)


def _loss(T, C, V, x, index="i64", none=0.0, pad=0, **more):
    return dict(op="loss", T=T, C=C, V=V, x=x, index=index, none=none, pad=pad, **more)


def _loss_bwd(T, C, V, x, index="i64", none=0.0, pad=0, weighted=False, **more):
    return dict(op="loss_bwd", T=T, C=C, V=V, x=x, index=index, none=none, pad=pad,
                weighted=weighted, **more)


def listed():
    return [
        # one token of a decode step: latency
        _embed(1, 4096, 32000, "bf16", "bf16", name="embed_decode_1x4096"),
        # the batch of a training step, or a long prompt
        _embed(8192, 4096, 131072, "bf16", "bf16", name="embed_train_8192x4096"),
        # a padded batch, the matrix kept in 32 bits, odd sizes, rows that start
        # anywhere
        _embed(1000, 4097, 50257, "f32", "f16", "i32", 0.1, 3, name="embed_ragged_1000x4097"),
        # the gradient of a training step's batch, alone in dW
        _embed_bwd(8192, 4096, 32000, "bf16", "bf16", name="embed_bwd_8192x4096"),
        # tied weights: added to what the loss left; padded batch, odd sizes
        _embed_bwd(5000, 1001, 50257, "f32", "f32", "i32", 0.2, 3, True,
                   name="embed_bwd_tied_5000x1001"),
        # a large batch through a narrow model, its gradients kept in 32 bits
        _embed_bwd(65536, 1024, 131072, "f32", "bf16", name="embed_bwd_65536x1024"),
        # the loss of a few positions (an evaluation, a short answer): the matrix
        # is read once, whatever they are
        _loss(16, 4096, 32000, "bf16", name="loss_few_16x4096x32000"),
        # a ragged batch, a fifth of it prompts, odd sizes, rows that start anywhere
        _loss(1000, 1001, 50257, "f16", "i32", 0.2, 3, name="loss_ragged_1000x1001x50257"),
        # the batch of a training step over a large vocabulary
        _loss(8192, 4096, 131072, "bf16", name="loss_train_8192x4096x131072"),
        # the gradients of a few positions
        _loss_bwd(16, 4096, 32000, "bf16", name="loss_bwd_few_16x4096x32000"),
        # the gradients of a ragged batch whose positions weigh differently
        _loss_bwd(1000, 1001, 50257, "f16", "i32", 0.2, 3, True,
                  name="loss_bwd_ragged_1000x1001x50257"),
        # the gradients of a training step, a quarter of its positions prompts
        _loss_bwd(8192, 4096, 32000, "bf16", none=0.25, name="loss_bwd_train_8192x4096x32000"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _round_or_odd(rng, n):
    """A size near n: a multiple of 160 mostly, else odd."""
    return max(32, n // 160 * 160) if rng.random() < 0.6 else n | 1


def draw(rng):
    op = rng.choice(["embed", "embed_bwd", "loss", "loss_bwd"])
    index, none, pad = rng.choice(["i32", "i64"]), rng.choice([0.0, 0.1, 0.5]), rng.choice([0, 0, 3, 8])
    V = _round_or_odd(rng, _log(rng, 64, 131000))
    if op in ("embed", "embed_bwd"):
        C = _round_or_odd(rng, _log(rng, 32, 8000))
        w, o = rng.choice(["bf16", "f16", "f32"]), rng.choice(["bf16", "f16", "f32"])
        if op == "embed":
            T = min(_log(rng, 1, 60000), (1 << 24) // C)
            return _embed(T, C, V, w, o, index, none, pad)
        T, V = min(_log(rng, 1, 60000), (1 << 25) // C), min(V, (1 << 26) // C)
        return _embed_bwd(T, C, V, w, o, index, none, pad, rng.random() < 0.4)
    C, x = _round_or_odd(rng, _log(rng, 64, 8000)), rng.choice(["bf16", "f16"])
    V = min(V, (1 << 29) // C)
    if op == "loss":
        return _loss(max(1, min(_log(rng, 1, 8192), (1 << 42) // (V * C))), C, V, x, index, none, pad)
    T = max(1, min(_log(rng, 1, 8192), (1 << 39) // (V * C)))
    return _loss_bwd(T, C, V, x, index, none, pad, rng.random() < 0.4)


def _nones(case):
    return int(case["T"] * case["none"])


def work(case):
    c = case
    T, C, V = c["T"], c["C"], c["V"]
    valid = T - _nones(c)
    index = T * SIZE[c["index"]]
    if c["op"] == "embed":
        return {"bytes": min(valid, V) * C * SIZE[c["w"]] + T * C * SIZE[c["out"]] + index, "flops": T * C}
    if c["op"] == "embed_bwd":
        w = V * C * SIZE[c["dw"]] * (2 if c["base"] else 1)
        return {"bytes": w + valid * C * SIZE[c["dout"]] + index, "flops": valid * C}
    if c["op"] == "loss":
        return {"bytes": (valid + V) * C * SIZE[c["x"]] + index + 8 * T, "flops": 2 * valid * V * C}
    return {"bytes": (valid + T + 2 * V) * C * SIZE[c["x"]] + index + 8 * T, "flops": 6 * valid * V * C}


# ------------------------------------------------------------------ the inputs

def _wide(rows, cols, pad, dtype):
    """A rows x cols view of rows that are cols + pad apart."""
    return torch.empty(rows, cols + pad, dtype=dtype, device=DEVICE)[:, :cols]


def _normal(gen, rows, cols, pad, dtype, scale=1.0):
    v = _wide(rows, cols, pad, dtype)
    step = max(1, (1 << 26) // cols)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        v[r:r + n] = torch.randn(n, cols, generator=gen, device=DEVICE) * scale
    return v


def _indices(gen, case):
    """Token numbers as text has them: the n-th most frequent in proportion to
    1 / n, frequent ones mostly (not always) the low numbers; some of none."""
    T, V = case["T"], case["V"]
    u = torch.rand(T, generator=gen, device=DEVICE, dtype=torch.float64)
    t = (torch.exp(u * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
    moved = t * 7919 % V
    t = torch.where(torch.rand(T, generator=gen, device=DEVICE) < 0.3, moved, t)
    at = torch.randperm(T, generator=gen, device=DEVICE)[:_nones(case)]
    t[at] = NONE
    return t.to(TYPES[case["index"]])


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    s = dict(c)
    if own:
        import matmul_selection_gb300 as mm
        s["mm"] = mm
    T, C, V, pad = c["T"], c["C"], c["V"], c["pad"]
    index = _indices(gen, c)
    if c["op"] == "embed":
        s["tokens"], s["scale"] = index, math.sqrt(C)
        s["weight"] = _normal(gen, V, C, pad, TYPES[c["w"]], 1 / math.sqrt(C))
        s["out_"] = torch.empty(T, C, dtype=TYPES[c["out"]], device=DEVICE)
        return s
    if c["op"] == "embed_bwd":
        s["tokens"], s["scale"] = index, math.sqrt(C)
        s["dout_"] = _normal(gen, T, C, pad, TYPES[c["dout"]], 0.01)
        s["base_"] = _normal(gen, V, C, pad, TYPES[c["dw"]], 0.1) if c["base"] else None
        s["dweight"] = torch.empty(V, C, dtype=TYPES[c["dw"]], device=DEVICE)
        return s
    # logits of about 1.3 in size, and the target's higher by up to a dozen, as
    # in a model that has learnt something
    dtype = TYPES[c["x"]]
    s["targets"] = index
    w = s["weight"] = _normal(gen, V, C, pad, dtype, 1.28 / math.sqrt(C))
    x = torch.randn(T, C, generator=gen, device=DEVICE)
    toward = w[index.long().clamp(0, V - 1)].float()
    toward /= toward.norm(dim=1, keepdim=True).clamp_min(1e-6)
    x += toward * torch.rand(T, 1, generator=gen, device=DEVICE) * 10
    s["xin"] = _wide(T, C, pad, dtype)
    s["xin"].copy_(x)
    s["loss"] = torch.empty(T, device=DEVICE)
    s["lse"] = torch.empty(T, device=DEVICE)
    if c["op"] == "loss_bwd":
        valid = (index >= 0) & (index < V)
        # as the forward pass left it
        step = max(1, (1 << 28) // V)
        for r in range(0, T, step):
            s["lse"][r:r + step] = torch.logsumexp(s["xin"][r:r + step].float() @ w.float().t(), 1)
        s["lse"] *= valid
        # of the mean over the positions that count; in 16 bits of narrow range
        # the loss is scaled up
        n = max(1, T - _nones(c))
        g = (min(64.0 * n, 32768.0) if c["x"] == "f16" else 1.0) / n
        s["dloss"] = torch.full((T,), g, device=DEVICE)
        if c["weighted"]:  # positions weigh differently, some against
            s["dloss"] *= torch.randn(T, generator=gen, device=DEVICE)
        s["dx"] = torch.empty(T, C, dtype=dtype, device=DEVICE)
        s["dweight"] = torch.empty(V, C, dtype=dtype, device=DEVICE)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _valid(s, index):
    return (index >= 0) & (index < s["V"])


def _own_embed(s):
    mm, w, out = s["mm"], s["weight"], s["out_"]
    mm.check(mm.mm_embedding(w, s["tokens"], out, s["T"], s["C"], s["V"], w.stride(0), out.stride(0),
                             (CODE[s["w"]], CODE[s["index"]], CODE[s["out"]]), s["scale"]))
    return out


def _plain_embed(s):
    ok = _valid(s, s["tokens"])
    rows = s["weight"][torch.where(ok, s["tokens"], 0).long()].float() * s["scale"]
    return torch.where(ok[:, None], rows, 0.0).to(s["out_"].dtype)


def _own_embed_bwd(s):
    mm, dout, base, dw = s["mm"], s["dout_"], s["base_"], s["dweight"]
    mm.check(mm.mm_embedding_backward(dout, s["tokens"], base, dw, s["T"], s["C"], s["V"],
                                      dout.stride(0), base.stride(0) if base is not None else 0,
                                      dw.stride(0), (CODE[s["dw"]], CODE[s["index"]], CODE[s["dout"]]),
                                      s["scale"]))
    return dw


def _plain_embed_bwd(s):
    ok = _valid(s, s["tokens"])
    at = torch.where(ok, s["tokens"], s["V"]).long()
    dw = torch.zeros(s["V"] + 1, s["C"], device=at.device)
    dw.index_add_(0, at, s["dout_"].float())
    dw = dw[:s["V"]] * s["scale"]
    if s["base_"] is not None:
        dw = dw + s["base_"].float()
    return dw.to(s["dweight"].dtype)


def _own_loss(s):
    mm, x, w = s["mm"], s["xin"], s["weight"]
    mm.check(mm.mm_cross_entropy(x, w, s["targets"], s["loss"], s["lse"], s["T"], s["C"], s["V"],
                                 x.stride(0), w.stride(0),
                                 (CODE[s["x"]], CODE[s["index"]], CODE["f32"])))
    return {"loss": s["loss"], "lse": s["lse"]}


def _plain_loss(s):
    ok = _valid(s, s["targets"])
    l = s["xin"].float() @ s["weight"].float().t()
    top = l.amax(1)
    lse = top + (l - top[:, None]).exp().sum(1).log()
    hit = l.gather(1, torch.where(ok, s["targets"], 0).long()[:, None])[:, 0]
    return {"loss": torch.where(ok, lse - hit, 0.0), "lse": torch.where(ok, lse, 0.0)}


def _own_loss_bwd(s):
    mm, x, w, dx, dw = s["mm"], s["xin"], s["weight"], s["dx"], s["dweight"]
    mm.check(mm.mm_cross_entropy_backward(x, w, s["targets"], s["lse"], s["dloss"], dx, dw, s["T"],
                                          s["C"], s["V"], x.stride(0), w.stride(0), dx.stride(0),
                                          dw.stride(0), (CODE[s["x"]], CODE[s["index"]], CODE[s["x"]])))
    return {"dx": dx, "dweight": dw}


def _plain_loss_bwd(s):
    ok = _valid(s, s["targets"])
    x, w = s["xin"].float(), s["weight"].float()
    g = (x @ w.t() - s["lse"][:, None]).exp()
    at = torch.where(ok, s["targets"], 0).long()[:, None]
    g.scatter_(1, at, g.gather(1, at) - 1)
    g = torch.where(ok[:, None], g * s["dloss"][:, None], 0.0)
    return {"dx": (g @ w).to(s["dx"].dtype), "dweight": (g.t() @ x).to(s["dweight"].dtype)}


_OWN = {"embed": _own_embed, "embed_bwd": _own_embed_bwd, "loss": _own_loss, "loss_bwd": _own_loss_bwd}
_PLAIN = {"embed": _plain_embed, "embed_bwd": _plain_embed_bwd, "loss": _plain_loss,
          "loss_bwd": _plain_loss_bwd}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    op = case["op"]
    if op in ("loss", "loss_bwd") and work(case)["flops"] > 1.2e13:
        return None  # 64-bit products at about 1 TFLOP/s
    s = prepare(case, seed)
    T, C, V = case["T"], case["C"], case["V"]
    index = s["tokens" if op.startswith("embed") else "targets"].long()
    rows = torch.nonzero(torch.logical_and(index.ge(0), index.lt(V)))[:, 0]
    if op == "embed":
        out = torch.zeros(T, C, dtype=torch.float64, device=DEVICE)
        out[rows] = torch.mul(torch.index_select(s["weight"], 0, index[rows]).double(), s["scale"])
        return out
    if op == "embed_bwd":
        dw = torch.zeros(V, C, dtype=torch.float64, device=DEVICE)
        if s["base_"] is not None:
            dw += s["base_"]
        dw.index_put_((index[rows],), torch.mul(s["dout_"][rows].double(), s["scale"]), accumulate=True)
        return dw
    w = s["weight"].double()
    step = max(1, (1 << 29) // V)
    if op == "loss":
        out = {k: torch.zeros(T, dtype=torch.float64, device=DEVICE) for k in ("loss", "lse")}
        for r in torch.split(rows, step):
            l = torch.einsum("tc,vc->tv", s["xin"][r].double(), w)
            lse = torch.logsumexp(l, 1)
            out["lse"][r] = lse
            out["loss"][r] = torch.sub(lse, l[torch.arange(len(r), device=DEVICE), index[r]])
        return out
    dx = torch.zeros(T, C, dtype=torch.float64, device=DEVICE)
    dw = torch.zeros(V, C, dtype=torch.float64, device=DEVICE)
    for r in torch.split(rows, step):
        x, d = s["xin"][r].double(), s["dloss"][r].double()
        g = torch.einsum("tc,vc->tv", x, w)
        g = torch.exp(torch.sub(g, s["lse"][r].double()[:, None], out=g), out=g)
        g[torch.arange(len(r), device=DEVICE), index[r]] -= 1.0
        dx[r] = torch.einsum("tv,vc,t->tc", g, w, d)
        dw += torch.einsum("tv,tc->vc", g, torch.mul(x, d[:, None]))
    return {"dx": dx, "dweight": dw}
