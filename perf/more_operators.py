"""The two products that most of a rank's training step is spent in, as a program calls them, with plain forms beside them.

Between the layer norms of a model stands a feed-forward block, and at its end the projection to the vocabulary with the loss.  The
operators here are

* ``loss``      -- softmax cross entropy of rows against a table of the vocabulary (the embedding's, where it is tied), with each row's
  logarithm of the sum of exponentials; the logits are not kept.  A target outside the table is padding: its loss is zero;
* ``loss_grad`` -- its gradient: the rows' and the table's, the latter added to what the table's gradient holds from elsewhere;
* ``ff``        -- a gated feed-forward block: two projections of a row, the activation of the first times the second;
* ``ff_grad``   -- its gradient from the two projections kept in the forward pass: the rows' and both weights'.

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is true, with the library's calls.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


def listed():
    return [
        # scoring a handful of tokens: the table is read once, and that is all
        {"name": "loss_tokens", "op": "loss", "n": 7, "vocab": 32000, "width": 4096, "type": "bf16", "index": "i64", "pad": 0.0},
        # the evaluation of a long batch against a large vocabulary, with padding
        {"name": "loss_batch", "op": "loss", "n": 8192, "vocab": 128000, "width": 4096, "type": "bf16", "index": "i64", "pad": 0.02},
        # a small model's micro-batch in full precision
        {"name": "loss_grad_small", "op": "loss_grad", "n": 1000, "vocab": 5000, "width": 320, "type": "f32", "index": "i32", "pad": 0.0, "base": False},
        # a ragged batch of odd sizes, many padded tokens, the table's gradient added to an earlier micro-batch's
        {"name": "loss_grad_odd", "op": "loss_grad", "n": 2021, "vocab": 49999, "width": 1001, "type": "bf16", "index": "i64", "pad": 0.3, "base": True},
        # one rank's micro-batch against a large vocabulary
        {"name": "loss_grad_batch", "op": "loss_grad", "n": 4096, "vocab": 128000, "width": 4096, "type": "bf16", "index": "i64", "pad": 0.02, "base": False},
        # one token of one sequence: all the time goes into reading the weights
        {"name": "ff_token", "op": "ff", "n": 1, "width": 4096, "inner": 11008, "type": "bf16", "act": "silu", "keep": False},
        # a decode step of 48 sequences
        {"name": "ff_decode", "op": "ff", "n": 48, "width": 4096, "inner": 11008, "type": "bf16", "act": "silu", "keep": False},
        # a training batch, both projections kept for the backward pass
        {"name": "ff_batch", "op": "ff", "n": 16384, "width": 4096, "inner": 11008, "type": "bf16", "act": "silu", "keep": True},
        # a ragged batch of odd sizes in full precision, with the other activation
        {"name": "ff_odd", "op": "ff", "n": 777, "width": 1001, "inner": 2671, "type": "f32", "act": "gelu", "keep": True},
        # a small model's micro-batch in full precision, backward
        {"name": "ff_grad_small", "op": "ff_grad", "n": 512, "width": 320, "inner": 1280, "type": "f32", "act": "gelu", "keep": True},
        # a ragged batch of odd sizes, backward
        {"name": "ff_grad_odd", "op": "ff_grad", "n": 3001, "width": 1001, "inner": 2671, "type": "bf16", "act": "gelu_tanh", "keep": True},
        # the training batch's backward pass
        {"name": "ff_grad_batch", "op": "ff_grad", "n": 16384, "width": 4096, "inner": 11008, "type": "bf16", "act": "silu", "keep": True},
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
    return w["bytes"] + w["flops"] / 100.0 * (4 if case["type"] == "f32" else 1)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0.0), _cost(c))
    op = rng.choice(["loss", "loss_grad", "ff", "ff_grad"])
    while True:
        c = {"op": op, "n": _spread(rng, 1, 16384), "width": _width(rng, 33, 8192), "type": rng.choice(["f32", "bf16", "bf16"])}
        if op in ("loss", "loss_grad"):
            c["vocab"] = _spread(rng, 1000, 128000)
            c["index"] = rng.choice(["i32", "i64"])
            c["pad"] = rng.choice([0.0, 0.02, 0.3])
        if op == "loss_grad":
            c["base"] = rng.random() < 0.3
        if op in ("ff", "ff_grad"):
            c["inner"] = _width(rng, 64, 16384)
            c["act"] = rng.choice(["silu", "silu", "gelu", "gelu_tanh"])
            c["keep"] = op == "ff_grad" or rng.random() < 0.5
        if _cost(c) <= most[op]:
            return c


def work(case):
    n, d, s, op = case["n"], case["width"], BYTES[case["type"]], case["op"]
    if op in ("loss", "loss_grad"):
        v = case["vocab"]
        rows = n * (8 if case["index"] == "i64" else 4) + 8 * n  # targets; loss and lse, or lse and the loss's gradient
        if op == "loss":
            return {"bytes": (n + v) * d * s + rows, "flops": 2.0 * n * v * d}
        return {"bytes": (2 * n + (3 if case["base"] else 2) * v) * d * s + rows, "flops": 6.0 * n * v * d}
    f = case["inner"]
    if op == "ff":
        return {"bytes": (n * d + 2 * f * d + (3 if case["keep"] else 1) * n * f) * s, "flops": 4.0 * n * d * f}
    return {"bytes": (2 * n * d + 4 * f * d + 3 * n * f) * s, "flops": 8.0 * n * d * f}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    n, d, dtype = case["n"], case["width"], TYPES[case["type"]]
    state = {"case": case}
    x = normal(n, d)  # rows as a layer norm leaves them
    if case["op"] in ("loss", "loss_grad"):
        v = case["vocab"]
        table = normal(v, d).mul_(1.3 / math.sqrt(d))  # logits of a few units
        targets = torch.randint(0, v, (n,), generator=g, device="cuda")
        # a trained model's rows point to their targets, some more than others
        x.addcmul_(table[targets], 8.0 * torch.rand(n, 1, generator=g, device="cuda"))
        targets[torch.rand(n, generator=g, device="cuda") < case["pad"]] = -1
        state["x"], state["table"] = x.to(dtype), table.to(dtype)
        state["targets"] = targets.to(torch.int32 if case["index"] == "i32" else torch.int64)
        if case["op"] == "loss_grad":
            # the mean's gradient over the tokens that count, and lse as the forward pass gave it
            state["gloss"] = torch.full((n,), 1.0 / max(1, int((targets >= 0).sum())), device="cuda")
            state["lse"] = torch.logsumexp(state["x"].float() @ state["table"].float().t(), 1)
            if case["base"]:
                state["base"] = normal(v, d).mul_(1e-5).to(dtype)
        return state
    f = case["inner"]
    state["x"] = x.to(dtype)
    state["w_gate"] = normal(f, d).mul_(1.0 / math.sqrt(d)).to(dtype)
    state["w_up"] = normal(f, d).mul_(1.0 / math.sqrt(d)).to(dtype)
    if case["op"] == "ff_grad":
        state["gh"] = normal(n, f).mul_(1e-3).to(dtype)
        state["gate"] = (state["x"].float() @ state["w_gate"].float().t()).to(dtype)
        state["up"] = (state["x"].float() @ state["w_up"].float().t()).to(dtype)
    return state


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------- plain forms

def _act(gate, kind):
    """The activation and its derivative."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-gate))
        return gate * s, s * (1.0 + gate * (1.0 - s))
    if kind == "gelu":
        phi = 0.5 * (1.0 + torch.erf(gate * math.sqrt(0.5)))
        return gate * phi, phi + gate * torch.exp(-0.5 * gate * gate) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (gate + 0.044715 * gate * gate * gate))
    return 0.5 * gate * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * gate * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * gate * gate)


def _run_plain(state):
    case = state["case"]
    op, dtype = case["op"], TYPES[case["type"]]
    x = state["x"].float()
    if op in ("loss", "loss_grad"):
        table, targets = state["table"].float(), state["targets"].long()
        inside = (targets >= 0) & (targets < case["vocab"])
        at = targets.clamp(0, case["vocab"] - 1)[:, None]
        z = x @ table.t()
        if op == "loss":
            top = z.amax(1, keepdim=True)
            picked = z.gather(1, at)
            lse = top + torch.log(torch.exp(z.sub_(top)).sum(1, keepdim=True))
            return {"loss": ((lse - picked)[:, 0]) * inside, "lse": lse[:, 0]}
        e = torch.exp(z.sub_(state["lse"][:, None]))
        e.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=e.dtype))
        e *= (state["gloss"] * inside)[:, None]
        gtable = e.t() @ x
        if case["base"]:
            gtable += state["base"].float()
        return {"x": (e @ table).to(dtype), "table": gtable.to(dtype)}
    w_gate, w_up = state["w_gate"].float(), state["w_up"].float()
    if op == "ff":
        gate, up = x @ w_gate.t(), x @ w_up.t()
        h = _act(gate, case["act"])[0] * up
        return {"h": h.to(dtype), "gate": gate.to(dtype), "up": up.to(dtype)} if case["keep"] else {"h": h.to(dtype)}
    gh = state["gh"].float()
    a, slope = _act(state["gate"].float(), case["act"])
    ggate, gup = gh * state["up"].float() * slope, gh * a
    return {"x": (ggate @ w_gate + gup @ w_up).to(dtype), "w_gate": (ggate.t() @ x).to(dtype), "w_up": (gup.t() @ x).to(dtype)}


# ------------------------------------------------------- the library's calls

def _run_own(state):
    import collective_reduction_virtual_gb300 as vc
    case = state["case"]
    op = case["op"]
    if op == "loss":
        loss, lse = vc.cross_entropy(state["x"], state["table"], state["targets"])
        return {"loss": loss, "lse": lse}
    if op == "loss_grad":
        gx, gtable = vc.cross_entropy_backward(state["gloss"], state["x"], state["table"], state["targets"], state["lse"], base=state.get("base"))
        return {"x": gx, "table": gtable}
    if op == "ff":
        if case["keep"]:
            h, gate, up = vc.gated_ff(state["x"], state["w_gate"], state["w_up"], activation=case["act"], keep=True)
            return {"h": h, "gate": gate, "up": up}
        return {"h": vc.gated_ff(state["x"], state["w_gate"], state["w_up"], activation=case["act"])}
    gx, gg, gu = vc.gated_ff_backward(state["gh"], state["x"], state["w_gate"], state["w_up"], state["gate"], state["up"], activation=case["act"])
    return {"x": gx, "w_gate": gg, "w_up": gu}


# ------------------------------------------- the definitions, in 64 bits

MOST_FLOPS = 1.4e13  # products in 64 bits of at most some ten seconds


def _exact_loss(case, state):
    n, v = case["n"], case["vocab"]
    table = state["table"].double()
    loss, lse = torch.empty(n, dtype=torch.float64, device="cuda"), torch.empty(n, dtype=torch.float64, device="cuda")
    for a in range(0, n, 1024):
        z = torch.nn.functional.linear(state["x"][a:a + 1024].double(), table)
        lse[a:a + 1024] = torch.logsumexp(z, 1)
        t = state["targets"][a:a + 1024].long()
        picked = torch.take_along_dim(z, torch.where((t >= 0) & (t < v), t, 0)[:, None], 1)[:, 0]
        loss[a:a + 1024] = torch.where((t >= 0) & (t < v), lse[a:a + 1024] - picked, 0.0)
    return {"loss": loss, "lse": lse}


def _exact_loss_grad(case, state):
    n, v, d = case["n"], case["vocab"], case["width"]
    table = state["table"].double()
    gx = torch.empty(n, d, dtype=torch.float64, device="cuda")
    gtable = state["base"].double() if case["base"] else torch.zeros(v, d, dtype=torch.float64, device="cuda")
    for a in range(0, n, 1024):
        x, t = state["x"][a:a + 1024].double(), state["targets"][a:a + 1024].long()
        p = torch.nn.functional.linear(x, table).sub_(state["lse"][a:a + 1024, None].double()).exp_()
        rows = torch.nonzero((t >= 0) & (t < v)).flatten()
        p[rows, t[rows]] -= 1.0
        weight = torch.zeros(len(t), dtype=torch.float64, device="cuda")
        weight[rows] = state["gloss"][a:a + 1024].double()[rows]
        p.mul_(weight[:, None])
        gx[a:a + 1024] = torch.mm(p, table)
        gtable.addmm_(p.t(), x)
    return {"x": gx, "table": gtable}


def _exact_act(gate, kind):
    """The activation and its derivative, from functions that give them otherwise than the plain form does."""
    if kind == "silu":
        s = torch.sigmoid(gate)
        return gate * s, s + gate * s * torch.sigmoid(-gate)
    if kind == "gelu":
        phi = torch.special.ndtr(gate)
        return gate * phi, phi + gate * torch.exp(-gate.square() / 2.0) / math.sqrt(2.0 * math.pi)
    inner = math.sqrt(2.0 / math.pi) * (gate + 0.044715 * gate ** 3)
    s = torch.sigmoid(2.0 * inner)  # (1 + tanh(inner)) / 2
    return gate * s, s + gate * s * (1.0 - s) * 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * gate.square())


def exact(case, seed):
    if work(case)["flops"] > MOST_FLOPS:
        return None
    state = prepare(case, seed)
    op = case["op"]
    if op == "loss":
        return _exact_loss(case, state)
    if op == "loss_grad":
        return _exact_loss_grad(case, state)
    x, w_gate, w_up = state["x"].double(), state["w_gate"].double(), state["w_up"].double()
    if op == "ff":
        gate, up = torch.nn.functional.linear(x, w_gate), torch.nn.functional.linear(x, w_up)
        h = _exact_act(gate, case["act"])[0].mul_(up)
        return {"h": h, "gate": gate, "up": up} if case["keep"] else {"h": h}
    gh = state["gh"].double()
    a, slope = _exact_act(state["gate"].double(), case["act"])
    ggate, gup = slope.mul_(state["up"].double()).mul_(gh), a.mul_(gh)
    return {"x": torch.mm(ggate, w_gate).addmm_(gup, w_up), "w_gate": torch.einsum("nf,nd->fd", ggate, x), "w_up": torch.einsum("nf,nd->fd", gup, x)}
