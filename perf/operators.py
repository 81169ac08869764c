"""The per-rank layer operators whose gradients the collectives reduce, as a program calls them, with plain forms beside them.

A data-parallel step of one virtual rank is, at its ends, an embedding lookup and its gradient, layer norms and their gradients, and
activations kept between the two passes.  The operators here are

* ``lookup``      -- rows of a table taken by token and scaled; a token outside the table gives a row of zeros;
* ``lookup_grad`` -- the table's gradient: the rows of the output's gradient summed by token, in the order of the tokens, and added to
  what the table's gradient holds from elsewhere;
* ``norm``        -- layer norm over the last axis, with each row's mean and reciprocal deviation;
* ``norm_grad``   -- its gradient: the input's, and the weight's and bias's summed over the rows;
* ``pack8``       -- an activation kept in 8 bits with one scale for each 128 columns of a row, and taken back;
* ``saved_norm``  -- a layer norm's forward and backward pass with nothing kept between them but the normalised input in 8 bits: its
  output taken back for the product that follows, and the three gradients computed from the kept form.

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is true, with the library's calls.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
BLOCK = 128  # columns that share one scale of an 8-bit activation
TINY = 2.0 ** -100  # a block whose largest magnitude is below this is kept as zeros
EPS = 1e-5


def listed():
    return [
        # one decode step of 32 sequences: a few rows out of a large table, all latency
        {"name": "lookup_decode", "op": "lookup", "n": 32, "vocab": 32000, "width": 4096, "type": "bf16", "index": "i64", "scale": 1.0, "pad": 0.0},
        # a long prompt or a training batch, with padding, and the square root of the width as the scale
        {"name": "lookup_batch", "op": "lookup", "n": 65536, "vocab": 128000, "width": 4096, "type": "bf16", "index": "i64", "scale": 64.0, "pad": 0.02},
        # a small model's micro-batch in full precision: small enough for launches to count
        {"name": "grad_small", "op": "lookup_grad", "n": 1000, "vocab": 5000, "width": 320, "type": "f32", "grad": "f32", "index": "i32", "scale": 1.0,
         "pad": 0.0, "base": False},
        # one rank's micro-batch of a mid-sized model, its gradient kept in 32 bits for the allreduce
        {"name": "grad_batch", "op": "lookup_grad", "n": 16384, "vocab": 32000, "width": 2048, "type": "bf16", "grad": "f32", "index": "i64", "scale": 1.0,
         "pad": 0.02, "base": False},
        # a tied table of odd sizes, whose gradient from the output projection is added on the way; many padded tokens
        {"name": "grad_tied_odd", "op": "lookup_grad", "n": 50021, "vocab": 49999, "width": 1001, "type": "f32", "grad": "f32", "index": "i64",
         "scale": 31.6, "pad": 0.3, "base": True},
        # the largest: a quarter of a million tokens, a large vocabulary, everything in bf16
        {"name": "grad_long", "op": "lookup_grad", "n": 262144, "vocab": 128000, "width": 4096, "type": "bf16", "grad": "bf16", "index": "i64", "scale": 1.0,
         "pad": 0.02, "base": False},
        # decoding: the norm of a handful of tokens
        {"name": "norm_decode", "op": "norm", "n": 7, "width": 4096, "type": "bf16"},
        # a prefill or training batch of a wide model
        {"name": "norm_batch", "op": "norm", "n": 32768, "width": 8192, "type": "bf16"},
        # the training batch's backward pass
        {"name": "norm_grad_batch", "op": "norm_grad", "n": 32768, "width": 4096, "type": "bf16"},
        # a ragged batch of odd width in full precision
        {"name": "norm_grad_odd", "op": "norm_grad", "n": 6007, "width": 1001, "type": "f32"},
        # an activation kept from the forward to the backward pass in full precision, its last block ragged
        {"name": "pack8_ragged", "op": "pack8", "n": 9001, "width": 2052, "type": "f32"},
        # a training step's layer norm that keeps 8 bits for each value
        {"name": "saved_norm_batch", "op": "saved_norm", "n": 16384, "width": 4096, "type": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Half of the widths are multiples of 64 as models have them, the others any number."""
    w = _spread(rng, lo, hi)
    return w if rng.random() < 0.5 else max(64, w // 64 * 64)


def _cost(case):
    w = work(case)
    return w["bytes"] + w["flops"] / 100.0


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0.0), _cost(c))
    op = rng.choice(["lookup", "lookup_grad", "lookup_grad", "norm", "norm_grad", "pack8", "saved_norm"])
    while True:
        c = {"op": op, "n": _spread(rng, 1, 262144), "width": _width(rng, 33, 8192), "type": rng.choice(["f32", "bf16"])}
        if op == "saved_norm":
            c["type"] = "bf16"
        if op in ("lookup", "lookup_grad"):
            c["vocab"] = _spread(rng, 1000, 128000)
            c["index"] = rng.choice(["i32", "i64"])
            c["scale"] = rng.choice([1.0, round(math.sqrt(c["width"]), 3)])
            c["pad"] = rng.choice([0.0, 0.02, 0.3])
        if op == "lookup_grad":
            c["base"] = rng.random() < 0.3
            c["grad"] = rng.choice(["f32", c["type"]])
        if _cost(c) <= most[op]:
            return c


def _popularity(vocab):
    """How often each token is met: nearly inverse to its rank, as in text."""
    p = 1.0 / (np.arange(vocab, dtype=np.float64) + 2.7)
    return p / p.sum()


def _met(case):
    """The expected number of tokens inside the table, and of different ones among them."""
    n = case["n"] * (1.0 - case["pad"])
    return n, float((-np.expm1(n * np.log1p(-_popularity(case["vocab"])))).sum())


def work(case):
    n, d, s = case["n"], case["width"], BYTES[case["type"]]
    blocks = -(-d // BLOCK)
    kept = n * (d + 4 * blocks)
    op = case["op"]
    if op == "lookup":
        _, rows = _met(case)
        return {"bytes": n * (8 if case["index"] == "i64" else 4) + rows * d * s + n * d * s, "flops": n * d}
    if op == "lookup_grad":
        inside, rows = _met(case)
        table = case["vocab"] * d * (2 if case["base"] else 1)
        return {"bytes": n * (8 if case["index"] == "i64" else 4) + inside * d * s + table * BYTES[case["grad"]], "flops": inside * d + rows * d}
    if op == "norm":
        return {"bytes": 2 * n * d * s + 2 * d * s + 8 * n, "flops": 8 * n * d}
    if op == "norm_grad":
        return {"bytes": 3 * n * d * s + 3 * d * s + 8 * n, "flops": 14 * n * d}
    if op == "pack8":  # x read, the kept form written, read again, and x written
        return {"bytes": 2 * n * d * s + 2 * kept, "flops": 5 * n * d}
    # saved_norm: x read, y and the kept form written; the kept form read and y written; it and y's gradient read and x's written
    return {"bytes": 5 * n * d * s + 3 * kept + 5 * d * s + 8 * n, "flops": 28 * n * d}


def _activations(g, n, d, dtype):
    """Rows of a residual stream: columns of different sizes, a few of them large, and an offset."""
    size = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    size[torch.rand(d, generator=g, device="cuda") < 0.005] *= 20.0
    x = torch.randn(n, d, generator=g, device="cuda")
    return x.mul_(size).add_(0.3).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    n, d, dtype = case["n"], case["width"], TYPES[case["type"]]
    state = {"case": case}
    if case["op"] in ("lookup", "lookup_grad"):
        v = case["vocab"]
        cdf = torch.from_numpy(np.cumsum(_popularity(v))).cuda()
        tokens = torch.searchsorted(cdf, torch.rand(n, generator=g, device="cuda", dtype=torch.float64)).clamp_(max=v - 1)
        tokens[torch.rand(n, generator=g, device="cuda") < case["pad"]] = -1
        state["tokens"] = tokens.to(torch.int32 if case["index"] == "i32" else torch.int64)
        if case["op"] == "lookup":
            state["table"] = torch.randn(v, d, generator=g, device="cuda").mul_(0.02).to(dtype)
        else:
            state["gout"] = torch.randn(n, d, generator=g, device="cuda").mul_(1e-3).to(dtype)
            if case["base"]:  # a tied table's gradient from the output projection
                state["base"] = torch.randn(v, d, generator=g, device="cuda").mul_(1e-2).to(TYPES[case["grad"]])
        return state
    state["x"] = _activations(g, n, d, dtype)
    if case["op"] == "pack8":
        return state
    state["weight"] = torch.randn(d, generator=g, device="cuda").mul_(0.1).add_(1.0).to(dtype)
    state["bias"] = torch.randn(d, generator=g, device="cuda").mul_(0.1).to(dtype)
    if case["op"] != "norm":
        state["gout"] = torch.randn(n, d, generator=g, device="cuda").to(dtype)
    if case["op"] == "norm_grad":  # kept by the forward pass
        x = state["x"].float()
        state["mean"] = x.mean(1)
        state["rstd"] = torch.rsqrt(x.sub_(state["mean"][:, None]).square_().mean(1) + EPS)
    return state


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------- plain forms

def _lookup(tokens, table, scale):
    inside = (tokens >= 0) & (tokens < table.shape[0])
    rows = table[tokens.clamp(0, table.shape[0] - 1).long()].float() * scale
    return (rows * inside[:, None]).to(table.dtype)


def _lookup_grad(tokens, gout, vocab, scale, dtype, into):
    inside = (tokens >= 0) & (tokens < vocab)
    total = torch.zeros(vocab + 1, gout.shape[1], device=gout.device)  # the last row takes what lies outside
    total.index_add_(0, torch.where(inside, tokens.long(), vocab), gout.float())
    total = total[:vocab] * scale
    return (total if into is None else into.float() + total).to(dtype)


def _norm(x, weight, bias):
    x = x.float()
    mean = x.mean(1)
    centred = x - mean[:, None]
    rstd = torch.rsqrt((centred * centred).mean(1) + EPS)
    normal = centred * rstd[:, None]
    return normal * weight.float() + bias.float(), mean, rstd, normal


def _norm_grad(gout, normal, rstd, weight):
    gout = gout.float()
    g = gout * weight.float()
    gx = (g - g.mean(1, keepdim=True) - normal * (g * normal).mean(1, keepdim=True)) * rstd[:, None]
    return gx, (gout * normal).sum(0), gout.sum(0)


def _pack8(x):
    n, d = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -d % BLOCK)).view(n, -1, BLOCK)
    top = x.abs().amax(2)
    top = torch.where(top < TINY, torch.zeros_like(top), top)
    full = torch.full_like(top, 127.0)
    unit = torch.where(top > 0, full / top, torch.zeros_like(top))
    return torch.round(x * unit[:, :, None]).to(torch.int8), top / full


def _unpack8(codes, scales, d):
    return (codes.float() * scales[:, :, None]).flatten(1)[:, :d]


def _run_plain(state):
    case = state["case"]
    op, dtype, d = case["op"], TYPES[case["type"]], case["width"]
    if op == "lookup":
        return {"out": _lookup(state["tokens"], state["table"], case["scale"])}
    if op == "lookup_grad":
        return {"table": _lookup_grad(state["tokens"], state["gout"], case["vocab"], case["scale"], TYPES[case["grad"]], state.get("base"))}
    if op == "pack8":
        return {"out": _unpack8(*_pack8(state["x"]), d).to(dtype)}
    if op == "norm":
        y, mean, rstd, _ = _norm(state["x"], state["weight"], state["bias"])
        return {"y": y.to(dtype), "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        normal = (state["x"].float() - state["mean"][:, None]) * state["rstd"][:, None]
        gx, gw, gb = _norm_grad(state["gout"], normal, state["rstd"], state["weight"])
        return {"x": gx.to(dtype), "weight": gw.to(dtype), "bias": gb.to(dtype)}
    y, _, rstd, normal = _norm(state["x"], state["weight"], state["bias"])
    normal = _unpack8(*_pack8(normal), d)
    again = normal * state["weight"].float() + state["bias"].float()
    gx, gw, gb = _norm_grad(state["gout"], normal, rstd, state["weight"])
    return {"y": y.to(dtype), "rstd": rstd, "y_again": again.to(dtype), "x": gx.to(dtype), "weight": gw.to(dtype), "bias": gb.to(dtype)}


# ------------------------------------------------------- the library's calls

def _run_own(state):
    import collective_reduction_virtual_gb300 as vc
    case = state["case"]
    op = case["op"]
    if op == "lookup":
        return {"out": vc.embedding(state["tokens"], state["table"], scale=case["scale"])}
    if op == "lookup_grad":
        return {"table": vc.embedding_backward(state["gout"], state["tokens"], case["vocab"], scale=case["scale"], base=state.get("base"),
                                               dtype=TYPES[case["grad"]])}
    if op == "pack8":
        kept = vc.checkpoint8(state["x"])
        return {"out": vc.checkpoint8_restore(kept, dtype=TYPES[case["type"]])}
    if op == "norm":
        y, mean, rstd = vc.layer_norm(state["x"], state["weight"], state["bias"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        gx, gw, gb = vc.layer_norm_backward(state["gout"], state["x"], state["mean"], state["rstd"], state["weight"])
        return {"x": gx, "weight": gw, "bias": gb}
    y, rstd, kept = vc.layer_norm_checkpoint8(state["x"], state["weight"], state["bias"], eps=EPS)
    again = vc.checkpoint8_restore(kept, state["weight"], state["bias"], dtype=y.dtype)
    gx, gw, gb = vc.layer_norm_backward_checkpoint8(state["gout"], kept, rstd, state["weight"])
    return {"y": y, "rstd": rstd, "y_again": again, "x": gx, "weight": gw, "bias": gb}


# ------------------------------------------- the definitions, in 64 bits

def _exact_kept(x):
    """Each value of x (64 bits) as 8 bits and a scale stand for it, block by block of columns."""
    out = torch.empty_like(x)
    for a in range(0, x.shape[1], BLOCK):
        part = x[:, a:a + BLOCK]
        step = part.abs().max(1, keepdim=True).values / 127.0
        out[:, a:a + BLOCK] = torch.where(step * 127.0 < TINY, 0.0, torch.round(part / torch.where(step > 0, step, 1.0)) * step)
    return out


def _exact_norm(x):
    x = x.double()
    var, mean = torch.var_mean(x, 1, correction=0)
    rstd = 1.0 / torch.sqrt(var + EPS)
    return x.sub_(mean[:, None]).mul_(rstd[:, None]), mean, rstd


def _exact_norm_grad(gout, normal, rstd, weight):
    gout = gout.double()
    gw, gb = torch.einsum("nd,nd->d", gout, normal), gout.sum(0)
    gout = gout.mul_(weight.double())
    a, b = gout.mean(1, keepdim=True), torch.einsum("nd,nd->n", gout, normal)[:, None] / gout.shape[1]
    return gout.sub_(a).addcmul_(normal, b, value=-1.0).mul_(rstd[:, None]), gw, gb


def _exact_lookup_grad(case, state):
    tokens, gout, v = state["tokens"].long(), state["gout"], case["vocab"]
    keep = torch.nonzero((tokens >= 0) & (tokens < v)).flatten()
    order = keep[torch.argsort(tokens[keep], stable=True)]
    ends = torch.searchsorted(tokens[order], torch.arange(v + 1, device="cuda"))  # token t's rows lie at ends[t] .. ends[t + 1]
    out = torch.empty(v, case["width"], dtype=torch.float64, device="cuda")
    for a in range(0, case["width"], 256):
        part = gout[:, a:a + 256].double()[order]
        sums = torch.cat([part.new_zeros(1, part.shape[1]), part.cumsum(0)])
        out[:, a:a + 256] = sums[ends[1:]] - sums[ends[:-1]]
    out *= float(case["scale"])
    if case["base"]:
        out += state["base"]
    return out


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        tokens, table = state["tokens"].long(), state["table"]
        padded = torch.cat([table, table.new_zeros(1, table.shape[1])])
        return {"out": padded[torch.where((tokens < 0) | (tokens >= case["vocab"]), case["vocab"], tokens)].double() * case["scale"]}
    if op == "lookup_grad":
        return {"table": _exact_lookup_grad(case, state)}
    if op == "pack8":
        return {"out": _exact_kept(state["x"].double())}
    if op == "norm":
        normal, mean, rstd = _exact_norm(state["x"])
        return {"y": normal.mul_(state["weight"].double()).add_(state["bias"].double()), "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        normal = (state["x"].double() - state["mean"].double()[:, None]) * state["rstd"].double()[:, None]
        gx, gw, gb = _exact_norm_grad(state["gout"], normal, state["rstd"].double(), state["weight"])
        return {"x": gx, "weight": gw, "bias": gb}
    normal, _, rstd = _exact_norm(state["x"])
    y = normal * state["weight"].double() + state["bias"].double()
    normal = _exact_kept(normal)
    again = normal * state["weight"].double() + state["bias"].double()
    gx, gw, gb = _exact_norm_grad(state["gout"], normal, rstd, state["weight"])
    return {"y": y, "rstd": rstd, "y_again": again, "x": gx, "weight": gw, "bias": gb}
