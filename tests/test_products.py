"""The loss against a vocabulary and the gated feed-forward block, with their
gradients, against 64-bit definitions (products_ref.py): types, strides, sizes
from nothing to several tiles, masks, pieces of the vocabulary, captured calls
and other streams; and their refusals.  Every tolerance is the bound that
products_ref.py derives for the inputs."""
import math

import numpy as np
import pytest
import torch

import products_ref as R
from test_layers import gen, like, matrix

TYPES = [torch.float32, torch.bfloat16]
LAYOUTS = ["dense", "slice", "odd"]


@pytest.fixture(scope="module")
def v():
    from collective_reduction_virtual_gb300 import build
    build.build()
    import collective_reduction_virtual_gb300 as vc
    return vc


def near(got, want, bound, dtype=torch.float32):
    """got is within the bound and its type's rounding of want, and NaN where want is."""
    assert got.dtype == dtype and got.shape == want.shape
    got = got.double()
    tol = bound * 1.01 + R.unit(dtype) * (want.abs() + bound) + 2.0 ** -126
    bad = ~(((got - want).abs() <= tol) | (got.isnan() & want.isnan()) | (got == want))
    assert not bad.any(), (torch.nonzero(bad)[:4].tolist(), got[bad][:4].tolist(),
                           want[bad][:4].tolist(), tol.expand_as(want)[bad][:4].tolist())


def targets_of(g, n, V, kind="some", dtype=torch.int64):
    if kind == "none" or not V:  # every row masked
        t = torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, -1, V)
    else:
        t = torch.randint(0, V, (n,), generator=g, device="cuda")
        if kind == "some":
            t[torch.rand(n, generator=g, device="cuda") < 0.2] = -100
        if n > 2:
            t[0], t[-1] = V - 1, 0
    return t.to(dtype)


def filled(t):
    return t.fill_(float("nan"))


def loss_case(g, n, V, D, dtype, layout="dense", kind="some", index=torch.int64):
    x = matrix(g, n, D, dtype, layout)
    table = matrix(g, V, D, dtype, layout, 2.0 / max(1, D) ** 0.5)
    return x, table, targets_of(g, n, V, kind, index)


# ------------------------------------------------------------- cross entropy

LOSS_SHAPES = [(1, 1, 1, "dense"), (1, 7, 8, "dense"), (3, 100, 33, "odd"), (130, 300, 64, "dense"),
               (5, 1000, 129, "slice"), (257, 513, 200, "dense"), (128, 256, 128, "slice"),
               (33, 65, 72, "odd"), (7, 3001, 512, "dense"), (300, 40, 1001, "dense"),
               (1, 5003, 320, "dense"), (64, 2048, 96, "dense"), (200, 129, 16, "odd"),
               (129, 1, 40, "dense"), (1000, 777, 24, "slice"), (2, 70000, 8, "dense")]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,V,D,layout", LOSS_SHAPES)
def test_cross_entropy(v, dtype, n, V, D, layout):
    g = gen(n + V + D)
    x, table, t = loss_case(g, n, V, D, dtype, layout, index=torch.int32 if n % 2 else torch.int64)
    loss, lse = v.cross_entropy(x, table, t)
    want, wlse, bound, blse = R.loss(x, table, t)
    near(loss, want, bound)
    near(lse, wlse, blse)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,V,D,layout", LOSS_SHAPES)
@pytest.mark.parametrize("kind", ["all", "some", "none"])
def test_cross_entropy_backward(v, dtype, n, V, D, layout, kind):
    g = gen(n + V + D + 1)
    x, table, t = loss_case(g, n, V, D, dtype, layout, kind, torch.int32 if n % 2 else torch.int64)
    lse = R.loss(x, table, t)[1].float()
    gloss = torch.randn(n, generator=g, device="cuda") * 1e-3
    base = matrix(g, V, D, dtype, layout, 1e-3)
    dx, dt = v.cross_entropy_backward(gloss, x, table, t, lse, dx=filled(like(x, layout)),
                                      dtable=filled(like(table, layout)))
    want = R.loss_grad(gloss, x, table, t, lse, None, dtype)
    near(dx, want[0], want[2], dtype)
    near(dt, want[1], want[3], dtype)
    # one value for all rows, added in place to what is there, dx over x
    one = torch.full((1,), 0.37, device="cuda")
    want = R.loss_grad(one, x, table, t, lse, base, dtype)
    dx, dt = v.cross_entropy_backward(one, x, table, t, lse, base=base, dtable=base, dx=x)
    assert dt is base and dx is x
    near(dx, want[0], want[2], dtype)
    near(dt, want[1], want[3], dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_cross_entropy_of_nothing(v, dtype):
    x, table, t = loss_case(gen(1), 5, 9, 16, dtype)
    loss, lse = v.cross_entropy(x[:0], table, t[:0])
    assert loss.shape == lse.shape == (0,)
    base = torch.randn(9, 16, device="cuda").to(dtype)
    g = torch.ones(5, device="cuda")
    dx, dt = v.cross_entropy_backward(g[:0], x[:0], table, t[:0], lse, dtable=filled(torch.empty_like(table)))
    assert dx.shape == (0, 16) and not dt.any()
    kept = base.clone()
    v.cross_entropy_backward(g[:0], x[:0], table, t[:0], lse, base=base, dtable=base)
    assert torch.equal(base, kept)
    dt = v.cross_entropy_backward(g[:0], x[:0], table, t[:0], lse, base=base, dtable=filled(torch.empty_like(table)))[1]
    assert torch.equal(dt, base)
    # no token at all
    loss, lse = v.cross_entropy(x, table[:0], t)
    assert not loss.any() and (lse == -float("inf")).all()
    dx, dt = v.cross_entropy_backward(g, x, table[:0], t, lse, dx=filled(torch.empty_like(x)))
    assert not dx.any() and dt.shape == (0, 16)
    # no column: every logit is zero
    t = t.clamp(min=0)
    loss, lse = v.cross_entropy(x[:, :0], table[:, :0], t)
    assert torch.allclose(lse, torch.full_like(lse, 9.0).log()) and torch.allclose(loss, lse)
    dx, dt = v.cross_entropy_backward(g, x[:, :0], table[:, :0], t, lse)
    assert dx.shape == (5, 0) and dt.shape == (9, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_masked_rows_may_hold_anything(v, dtype):
    g = gen(2)
    x, table, t = loss_case(g, 150, 300, 72, dtype, kind="all")
    bad = torch.tensor([0, 31, 32, 127, 128, 149], device="cuda")
    x[bad] = float("nan")
    x[bad[1], 3] = float("inf")
    t[bad] = torch.tensor([-1, 300, 2 ** 40, -2 ** 40, 301, -100], device="cuda")
    loss, lse = v.cross_entropy(x, table, t)
    keep = torch.ones(150, dtype=torch.bool, device="cuda")
    keep[bad] = False
    want, wlse, bound, blse = R.loss(x[keep], table, t[keep])
    near(loss[keep], want, bound)
    near(lse[keep], wlse, blse)
    assert not loss[bad].any()
    gloss = torch.randn(150, generator=g, device="cuda")
    gloss[bad] = float("inf")
    lse[bad] = float("nan")
    dx, dt = v.cross_entropy_backward(gloss, x, table, t, lse)
    want = R.loss_grad(gloss, x, table, t, lse, None, dtype)
    near(dx, want[0], want[2], dtype)
    near(dt, want[1], want[3], dtype)
    assert not dx[bad].any()


@pytest.mark.gpu
def test_a_row_of_nan_touches_no_other(v):
    g = gen(3)
    for dtype in TYPES:
        x, table, t = loss_case(g, 140, 500, 40, dtype, kind="all")
        x[7, 2] = float("nan")
        loss, lse = v.cross_entropy(x, table, t)
        bad = torch.isnan(loss)
        assert bad.sum() == 1 and bad[7] and torch.isnan(lse[7])
        dx, _ = v.cross_entropy_backward(torch.ones(1, device="cuda"), x, table, t, lse, table_grad=False)
        assert torch.isnan(dx[7]).all() and torch.isfinite(dx[torch.arange(140, device="cuda") != 7]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_logits_far_apart(v, dtype):
    # rows whose largest logit is far above or below zero
    g = gen(4)
    x, table, t = loss_case(g, 70, 600, 64, dtype, kind="all")
    x *= torch.logspace(-3, 2.5, 70, device="cuda").to(dtype)[:, None]
    table[5] = -30.0
    loss, lse = v.cross_entropy(x, table, t)
    want, wlse, bound, blse = R.loss(x, table, t)
    near(loss, want, bound)
    near(lse, wlse, blse)
    want = R.loss_grad(torch.ones(1, device="cuda"), x, table, t, lse, None, dtype)
    dx, dt = v.cross_entropy_backward(torch.ones(1, device="cuda"), x, table, t, lse)
    near(dx, want[0], want[2], dtype)
    near(dt, want[1], want[3], dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,n,V,D,layout", [
    (torch.float32, 3, 5001, 65536, "dense"), (torch.bfloat16, 3, 5001, 65537, "odd"),
    (torch.float32, 40000, 5001, 24, "dense"), (torch.bfloat16, 70001, 5001, 16, "dense"),
])
def test_a_vocabulary_in_pieces(v, dtype, n, V, D, layout):
    g = gen(5)
    x, table, t = loss_case(g, n, V, D, dtype, layout)
    loss, lse = v.cross_entropy(x, table, t)
    gloss = torch.randn(n, generator=g, device="cuda")
    base = matrix(g, V, D, dtype)
    dx, dt = v.cross_entropy_backward(gloss, x, table, t, lse, base=base)
    want = [[], []]
    total = bound = 0.0
    for a in range(0, n, 8192):
        part = slice(a, a + 8192)
        w = R.loss(x[part], table, t[part])
        near(loss[part], w[0], w[2])
        near(lse[part], w[1], w[3])
        w = R.loss_grad(gloss[part], x[part], table, t[part], lse[part], None, dtype)
        near(dx[part], w[0], w[2], dtype)
        total, bound = total + w[1], bound + w[3]
    # the bound of a sum of n terms, from that of its parts
    bound = bound * max(1, n // 4096) + 2 * R.U * (total + base.double()).abs()
    near(dt, total + base.double(), bound, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,n,V,D", [(torch.float32, 30011, 4801, 9), (torch.bfloat16, 70001, 5001, 15)])
def test_one_gradient_of_a_vocabulary_in_pieces(v, dtype, n, V, D):
    g = gen(6)
    x, table, t = loss_case(g, n, V, D, dtype, "odd", index=torch.int32)
    lse = v.cross_entropy(x, table, t)[1]
    one = torch.full((1,), 1.0 / n, device="cuda")
    base = matrix(g, V, D, dtype)
    dx, none = v.cross_entropy_backward(one, x, table, t, lse, table_grad=False)
    assert none is None
    none, dt = v.cross_entropy_backward(one, x, table, t, lse, base=base, x_grad=False)
    assert none is None
    total = bound = 0.0
    for a in range(0, n, 8192):
        part = slice(a, a + 8192)
        w = R.loss_grad(one, x[part], table, t[part], lse[part], None, dtype)
        near(dx[part], w[0], w[2], dtype)
        total, bound = total + w[1], bound + w[3]
    bound = bound * max(1, n // 4096) + 2 * R.U * (total + base.double()).abs()
    near(dt, total + base.double(), bound, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_a_long_batch_of_narrow_rows(v, dtype):
    n, V, D = 300007, 37, 8
    g = gen(8)
    x, table, t = loss_case(g, n, V, D, dtype)
    loss, lse = v.cross_entropy(x, table, t)
    w = R.loss(x, table, t)
    near(loss, w[0], w[2])
    near(lse, w[1], w[3])
    h, gate, up = v.gated_ff(x, table, table, "gelu", keep=True)
    want = R.gated(x, table, table, "gelu")
    for got, exact, bound in zip((h, gate, up), want[:3], want[3:]):
        near(got, exact, bound, dtype)


@pytest.mark.gpu
def test_cross_entropy_gradient_against_differences(v):
    g = gen(6)
    n, V, D = 40, 90, 48
    x, table, t = loss_case(g, n, V, D, torch.float32)
    gloss = torch.randn(n, generator=g, device="cuda")
    lse = v.cross_entropy(x, table, t)[1]
    dx, dt = v.cross_entropy_backward(gloss, x, table, t, lse)

    def total(x, table):
        loss, _, bound, _ = R.loss(x, table, t)  # in 64 bits
        mine = v.cross_entropy(x.float(), table.float(), t)[0]
        near(mine, loss, bound)
        return (gloss.double() * loss).sum().item()

    for which, grad in ((0, dx), (1, dt)):
        step = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        h = 2.0 ** -12
        # fp32 holds these inputs only roughly: what it holds is what is moved
        a, b = [(y.double() + s * h * step).float() for y in ((x, table)[which],) for s in (1, -1)]
        up, down = (total(*((y, table) if which == 0 else (x, y))) for y in (a, b))
        moved = (grad.double() * (a.double() - b.double())).sum().item()
        # third differences: |f'''| of a log of exponentials is below 2 |direction|^3 per row
        far = ((a.double() - b.double()).abs().sum(1).amax() / 2).item() * 4
        size = (gloss.abs().double().sum() * 2 * far ** 3).item()
        rounding = (grad.double().abs() * (a.double() - b.double()).abs()).sum().item() * 1e-5
        assert abs(up - down - moved) <= size + rounding + 1e-9, (which, up - down, moved)


# ---------------------------------------------------------------- gated block

GATED_SHAPES = [(1, 1, 1, "dense"), (1, 64, 128, "dense"), (3, 33, 100, "odd"), (130, 64, 96, "dense"),
                (5, 129, 1000, "slice"), (257, 200, 129, "dense"), (128, 128, 256, "slice"),
                (33, 72, 65, "odd"), (48, 512, 640, "dense"), (300, 1001, 40, "dense"),
                (1, 320, 5003, "dense"), (1000, 24, 31, "slice"), (129, 40, 32, "dense"),
                (2, 8, 3000, "dense"), (700, 256, 260, "dense")]


def gated_case(g, n, D, F, dtype, layout):
    x = matrix(g, n, D, dtype, layout)
    wg, wu = (matrix(g, F, D, dtype, layout, 1.5 / max(1, D) ** 0.5) for _ in range(2))
    return x, wg, wu


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,D,F,layout", GATED_SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_ff(v, dtype, n, D, F, layout, act):
    g = gen(n + D + F)
    x, wg, wu = gated_case(g, n, D, F, dtype, layout)
    out = filled(like(torch.empty(n, F, dtype=dtype, device="cuda"), layout))
    h, gate, up = v.gated_ff(x, wg, wu, activation=act, keep=True, out=out)
    want = R.gated(x, wg, wu, act)
    assert h is out
    for got, w, b in zip((h, gate, up), want[:3], want[3:]):
        near(got, w, b, dtype)
    assert torch.equal(v.gated_ff(x, wg, wu, activation=act), h)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,D,F,layout", GATED_SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_ff_backward(v, dtype, n, D, F, layout, act):
    g = gen(n + D + F + 1)
    x, wg, wu = gated_case(g, n, D, F, dtype, layout)
    gate, up, dh = (matrix(g, n, F, dtype, layout, s) for s in (2.0, 1.0, 1e-2))
    got = v.gated_ff_backward(dh, x, wg, wu, gate, up, activation=act, dx=filled(like(x, layout)),
                              dw_gate=filled(like(wg, layout)), dw_up=filled(like(wu, layout)))
    want = R.gated_grad(dh, x, wg, wu, gate, up, act, dtype)
    for t, w, b in zip(got, want[:3], want[3:]):
        near(t, w, b, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 7])
@pytest.mark.parametrize("D,F,layout", [(72, 200, "dense"), (129, 67, "odd"), (640, 1030, "slice")])
def test_gradients_of_a_few_bf16_rows_round_once(v, n, D, F, layout):
    # dgate and dup hold 16 bits: what they lose is 2^-8 of a rounding to bf16
    bf = torch.bfloat16
    g = gen(n + D)
    x, wg, wu = gated_case(g, n, D, F, bf, layout)
    dh, gate, up = (matrix(g, n, F, bf, layout) for _ in range(3))
    got = v.gated_ff_backward(dh, x, wg, wu, gate, up, "silu")
    exact = R.gated_grad(dh, x, wg, wu, gate, up, "silu", torch.float32)
    rounded = R.gated_grad(dh, x, wg, wu, gate, up, "silu", bf)
    for one, want, fine, coarse in zip(got, exact[:3], exact[3:], rounded[3:]):
        near(one, want, fine + (coarse - fine) * 2.0 ** -8, bf)
    for skip in ({"x_grad": False}, {"weight_grads": False}):
        for one, want, fine, coarse in zip(v.gated_ff_backward(dh, x, wg, wu, gate, up, "silu", **skip),
                                           exact[:3], exact[3:], rounded[3:]):
            if one is not None:
                near(one, want, fine + (coarse - fine) * 2.0 ** -8, bf)


@pytest.mark.gpu
def test_gated_ff_of_nothing(v):
    for dtype in TYPES:
        x, wg, wu = gated_case(gen(7), 6, 40, 50, dtype, "dense")
        h, gate, up = v.gated_ff(x[:0], wg, wu, keep=True)
        assert h.shape == gate.shape == up.shape == (0, 50)
        dx, dg, du = v.gated_ff_backward(h, x[:0], wg, wu, gate, up, dw_gate=filled(torch.empty_like(wg)),
                                         dw_up=filled(torch.empty_like(wu)))
        assert dx.shape == (0, 40) and not dg.any() and not du.any()
        h, gate, up = v.gated_ff(x, wg[:0], wu[:0], keep=True)
        assert h.shape == (6, 0)
        dx, dg, du = v.gated_ff_backward(h, x, wg[:0], wu[:0], gate, up, dx=filled(torch.empty_like(x)))
        assert not dx.any() and dg.shape == (0, 40)
        h, gate, up = v.gated_ff(x[:, :0], wg[:, :0], wu[:, :0], keep=True, out=filled(torch.empty(6, 50, dtype=dtype, device="cuda")))
        assert not h.any() and not gate.any() and not up.any()


@pytest.mark.gpu
def test_activations_at_their_ends(v):
    # gate takes each value through a weight of one: far tails, zeros, infinities
    ends = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 12.0, -12.0, 30.0, -30.0, 90.0, -90.0,
                         200.0, -200.0, 1e4, -1e4], device="cuda")
    for act in ("silu", "gelu", "gelu_tanh"):
        x = ends[:, None].clone()
        one = torch.ones(1, 1, device="cuda")
        h = v.gated_ff(x, one, torch.zeros(1, 1, device="cuda"), activation=act)
        assert not h.any()  # a zero up
        a, slope = R.act(ends.double(), act)
        gate, up = x, torch.ones_like(x)
        dx, dg, _ = v.gated_ff_backward(up, torch.ones_like(x), one, one, gate, up, activation=act)
        both = a + slope
        tol = R.act_rel(ends.double()) * (a.abs() + 1 + (slope - a).abs()) + 2.0 ** -100
        assert ((dx[:, 0].double() - both).abs() <= tol).all(), (act, dx[:, 0], both)


@pytest.mark.gpu
def test_gated_gradient_against_differences(v):
    g = gen(8)
    for act in ("silu", "gelu", "gelu_tanh"):
        x, wg, wu = gated_case(g, 30, 40, 50, torch.float32, "dense")
        dh = torch.randn(30, 50, generator=g, device="cuda")
        _, gate, up = v.gated_ff(x, wg, wu, activation=act, keep=True)
        grads = v.gated_ff_backward(dh, x, wg, wu, gate, up, activation=act)
        for which in range(3):
            args = [x, wg, wu]
            step = torch.randn(args[which].shape, generator=g, device="cuda", dtype=torch.float64)
            h = 2.0 ** -10
            ends = []
            for s in (1, -1):
                args[which] = ((x, wg, wu)[which].double() + s * h * step).float()
                ends.append(((dh.double() * R.gated(*args, act)[0]).sum().item(), args[which].double()))
            delta = ends[0][1] - ends[1][1]
            moved = (grads[which].double() * delta).sum().item()
            # |third derivative| of h along a unit move of gate or up is below 4 (1 + |up| + |gate|);
            # gate and up move by at most |delta| . |other| / 2
            other = (wg.abs().amax() + wu.abs().amax()) if which == 0 else x.abs().amax()
            far = (delta.abs().sum(1).amax() * other / 2).item()
            size = (dh.abs().sum() * 4 * (1 + up.abs().amax() + gate.abs().amax()) * far ** 3).item()
            rounding = (grads[which].double().abs() * delta.abs()).sum().item() * 1e-5
            assert abs(ends[0][0] - ends[1][0] - moved) <= size + rounding, (act, which)


# ------------------------------------------------------------- how it is used

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_a_step_of_lookup_block_norm_and_loss(v, dtype):
    """The operators in the order of a training step, against autograd in 64
    bits on the same roundings' neighbourhood."""
    g = gen(9)
    V, D, F, n = 301, 96, 224, 260
    table = (torch.randn(V, D, generator=g, device="cuda") * 0.3).to(dtype)
    wg, wu, wd = ((torch.randn(*s, generator=g, device="cuda") * 0.15).to(dtype) for s in ((F, D), (F, D), (D, F)))
    tokens = torch.randint(0, V, (4, n // 4), generator=g, device="cuda")
    targets = torch.roll(tokens, -1, 1)
    targets[:, -1] = -1
    x = v.embedding(tokens, table)
    h, gate, up = v.gated_ff(x, wg, wu, keep=True)
    r = h @ wd.t() + x
    y, mean, rstd = v.layer_norm(r)
    loss, lse = v.cross_entropy(y, table, targets)
    one = torch.full((1,), 1.0 / int((targets >= 0).sum()), device="cuda")
    dy, dtable = v.cross_entropy_backward(one, y, table, targets, lse)
    dr, _, _ = v.layer_norm_backward(dy, r, mean, rstd, weight_grads=False)
    dx, dwg, dwu = v.gated_ff_backward(dr @ wd, x, wg, wu, gate, up)
    v.embedding_backward(dx + dr, tokens, V, base=dtable, out=dtable)

    params = [p.double().requires_grad_() for p in (table, wg, wu)]
    T, G, Up = params
    x64 = T[tokens]
    h64 = torch.nn.functional.silu(x64 @ G.t()) * (x64 @ Up.t())
    r64 = h64 @ wd.double().t() + x64
    z = torch.nn.functional.layer_norm(r64, (D,)) @ T.t()
    want = torch.nn.functional.cross_entropy(z.flatten(0, 1), targets.flatten(), ignore_index=-1, reduction="none")
    (want.sum() * one.double()).backward()
    # ten roundings in a row between the table and its gradient, each of half a unit of its value,
    # in sums of terms of both signs: compared as norms
    rel = 10 * R.unit(dtype) if dtype == torch.bfloat16 else 1e-5
    for got, p in zip((dtable, dwg, dwu), params):
        assert (got.double() - p.grad).norm() <= rel * p.grad.norm()
    assert (loss.double().flatten() - want.detach()).norm() <= rel * want.detach().norm()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_captured_calls_replay_on_new_inputs(v, dtype):
    g = gen(10)
    x, table, t = loss_case(g, 200, 700, 96, dtype)
    a, wg, wu = gated_case(g, 200, 96, 160, dtype, "dense")
    gloss = torch.randn(200, generator=g, device="cuda")
    dh = matrix(g, 200, 160, dtype)

    def calls():
        loss, lse = v.cross_entropy(x, table, t)
        h, gate, up = v.gated_ff(a, wg, wu, keep=True)
        return (loss, lse, *v.cross_entropy_backward(gloss, x, table, t, lse), h, gate, up,
                *v.gated_ff_backward(dh, a, wg, wu, gate, up))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for _ in range(2):
        for u in (x, table, a, wg, wu, dh):
            u.copy_(torch.randn(u.shape, generator=g, device="cuda").to(dtype) * 0.2)
        t.copy_(targets_of(g, 200, 700))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, calls()):
            assert torch.equal(got, want)


@pytest.mark.gpu
def test_a_process_may_capture_its_first_calls():
    import os
    import subprocess
    import sys
    code = """
import torch
import collective_reduction_virtual_gb300 as vc
x, w = torch.randn(200, 256, device="cuda").bfloat16(), torch.randn(512, 256, device="cuda").bfloat16()
t = torch.randint(0, 512, (200,), device="cuda")
one = torch.ones(1, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    loss, lse = vc.cross_entropy(x, w, t)
    grads = vc.cross_entropy_backward(one, x, w, t, lse)
    h, gate, up = vc.gated_ff(x, w, w, keep=True)
    more = vc.gated_ff_backward(h, x, w, w, gate, up)
graph.replay()
torch.cuda.synchronize()
again = vc.cross_entropy(x, w, t)
assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
for a, b in zip((*grads, *more), (*vc.cross_entropy_backward(one, x, w, t, lse), *vc.gated_ff_backward(h, x, w, w, gate, up))):
    assert torch.equal(a, b)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.gpu
def test_calls_on_two_streams_at_once(v):
    g = gen(11)
    cases = [loss_case(g, 400, 3000, 256, torch.bfloat16) for _ in range(2)]
    one = torch.ones(1, device="cuda")
    want = []
    for x, table, t in cases:
        loss, lse = v.cross_entropy(x, table, t)
        want.append((loss, lse, *v.cross_entropy_backward(one, x, table, t, lse)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, (x, table, t) in zip(streams, cases):
            loss, lse = v.cross_entropy(x, table, t, stream=s)
            got.append((loss, lse, *v.cross_entropy_backward(one, x, table, t, lse, stream=s)))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.gpu
def test_repeated_calls_give_the_same_bits(v):
    g = gen(12)
    for n, V, D in ((900, 4000, 128), (3, 9000, 1024)):
        x, table, t = loss_case(g, n, V, D, torch.bfloat16)
        one = torch.ones(1, device="cuda")
        loss, lse = v.cross_entropy(x, table, t)
        grads = v.cross_entropy_backward(one, x, table, t, lse)
        for _ in range(4):
            again = v.cross_entropy(x, table, t)
            assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
            for a, b in zip(grads, v.cross_entropy_backward(one, x, table, t, lse)):
                assert torch.equal(a, b)


def spot(r, t):
    """A copy of a matrix at a random alignment and row stride."""
    n, d = t.shape
    pad, at = int(r.choice([0, 0, 0, 1, 2, 8, 24])), int(r.choice([0, 0, 1, 2, 3, 4, 8]))
    flat = torch.empty(n * (d + pad) + at, dtype=t.dtype, device="cuda")
    return flat[at:].view(n, d + pad)[:, :d].copy_(t)


def size(r, lo, hi):
    return int(round(np.exp(r.uniform(np.log(lo), np.log(hi)))))


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(60))
def test_random_losses(v, seed):
    r, g = np.random.default_rng(seed), gen(seed)
    n, V, D = size(r, 1, 1500), size(r, 1, 6000), size(r, 1, 1500)
    dtype = TYPES[r.integers(2)]
    x, table, t = loss_case(g, n, V, D, dtype, kind=["all", "some", "some", "none"][r.integers(4)],
                            index=[torch.int32, torch.int64][r.integers(2)])
    x, table = spot(r, x), spot(r, table)
    loss, lse = v.cross_entropy(x, table, t)
    want, wlse, bound, blse = R.loss(x, table, t)
    near(loss, want, bound)
    near(lse, wlse, blse)
    gloss = torch.randn(n if r.integers(2) else 1, generator=g, device="cuda")
    base = spot(r, matrix(g, V, D, dtype)) if r.integers(2) else None
    want = R.loss_grad(gloss, x, table, t, lse, base, dtype)
    which = r.integers(4)  # both, or one alone
    dx, dt = v.cross_entropy_backward(gloss, x, table, t, lse, base=base,
                                      dx=filled(spot(r, x)) if which != 1 else None,
                                      dtable=filled(spot(r, table)) if which != 2 else None,
                                      x_grad=which != 1, table_grad=which != 2)
    if which != 1:
        near(dx, want[0], want[2], dtype)
    if which != 2:
        near(dt, want[1], want[3], dtype)
    assert v.device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(60))
def test_random_gated_blocks(v, seed):
    r, g = np.random.default_rng(seed + 1000), gen(seed + 1000)
    n, D, F = size(r, 1, 1500), size(r, 1, 1500), size(r, 1, 3000)
    dtype, act = TYPES[r.integers(2)], ["silu", "gelu", "gelu_tanh"][r.integers(3)]
    x, wg, wu = (spot(r, t) for t in gated_case(g, n, D, F, dtype, "dense"))
    keep = bool(r.integers(2))
    h = v.gated_ff(x, wg, wu, activation=act, keep=keep, out=filled(spot(r, torch.empty(n, F, dtype=dtype, device="cuda"))))
    want = R.gated(x, wg, wu, act)
    for got, w, b in zip(h if keep else (h,), want[:3], want[3:]):
        near(got, w, b, dtype)
    gate, up, dh = (spot(r, matrix(g, n, F, dtype, "dense", s)) for s in (2.0, 1.0, 1e-2))
    which = r.integers(4)
    got = v.gated_ff_backward(dh, x, wg, wu, gate, up, activation=act, x_grad=which != 1, weight_grads=which != 2,
                              dw_gate=filled(spot(r, wg)) if which == 3 else None)
    want = R.gated_grad(dh, x, wg, wu, gate, up, act, dtype)
    assert (got[0] is None) == (which == 1) and (got[2] is None) == (which == 2)
    for t, w, b in zip(got, want[:3], want[3:]):
        if t is not None:
            near(t, w, b, dtype)
    assert v.device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 4, 5, 8, 9, 15, 16, 17, 33])
@pytest.mark.parametrize("D,V", [(512, 1000), (1028, 333), (4099, 66), (130, 2049), (2, 9)])
def test_few_rows_in_full_precision(v, n, D, V):
    # up to 16 rows go another way than more, and rows of whole 16 bytes another than others
    g = gen(n * D + V)
    x, table, t = loss_case(g, n, V, D, torch.float32, kind="some")
    loss, lse = v.cross_entropy(x, table, t)
    want, wlse, bound, blse = R.loss(x, table, t)
    near(loss, want, bound)
    near(lse, wlse, blse)
    gloss = torch.randn(n, generator=g, device="cuda")
    base = matrix(g, V, D, torch.float32)
    want = R.loss_grad(gloss, x, table, t, lse, base, torch.float32)
    dx, dt = v.cross_entropy_backward(gloss, x, table, t, lse, base=base)
    near(dx, want[0], want[2])
    near(dt, want[1], want[3])
    _, wg, wu = gated_case(g, 1, D, V, torch.float32, "dense")
    h, gate, up = v.gated_ff(x, wg, wu, activation="gelu", keep=True)
    want = R.gated(x, wg, wu, "gelu")
    for got, w, b in zip((h, gate, up), want[:3], want[3:]):
        near(got, w, b)
    got = v.gated_ff_backward(h, x, wg, wu, gate, up, activation="gelu")
    want = R.gated_grad(h, x, wg, wu, gate, up, "gelu", torch.float32)
    for a, w, b in zip(got, want[:3], want[3:]):
        near(a, w, b)


@pytest.mark.gpu
def test_a_table_past_32_bit_offsets(v):
    g = gen(16)
    V, D, n = 2_100_013, 2048, 5
    assert V * D > 2 ** 32
    table = torch.randn(V, D, generator=g, device="cuda", dtype=torch.bfloat16).mul_(0.02)
    x = matrix(g, n, D, torch.bfloat16)
    t = torch.tensor([0, V - 1, V - 2, V // 2, V], device="cuda")
    loss, lse = v.cross_entropy(x, table, t)
    parts = [R.product(x.double(), table[a:a + 65536].double().t()) for a in range(0, V, 65536)]
    z, dz = (torch.cat([p[k] for p in parts], 1) for k in range(2))
    wlse = torch.logsumexp(z, 1)
    # the bound of a vocabulary that products_ref.loss has, written for rows already multiplied
    p = torch.exp(z - wlse[:, None])
    blse = (p * (dz + 4 * R.U * (2 + 2 * (z - z.amax(1, keepdim=True)).abs()))).sum(1) + (320 + V / 256) * R.U
    blse = blse + 4 * R.U * (wlse.abs() + z.amax(1).abs() + math.log(V) + 1)
    near(lse, wlse, blse)
    at = t[:4, None]
    near(loss[:4], wlse[:4] - z[:4].gather(1, at)[:, 0], blse[:4] + dz[:4].gather(1, at)[:, 0] + 8 * R.U * wlse[:4])
    assert loss[4] == 0
    dx, dt = v.cross_entropy_backward(torch.ones(1, device="cuda"), x, table, t, lse)
    # the rows at both ends of the table's gradient, and between
    for a in (0, V // 2 - 32, V - 64):
        rows = slice(a, a + 64)
        e = torch.exp(z[:4, rows] - lse[:4, None].double())
        size_e = e.clone()
        for i in range(4):
            if a <= int(t[i]) < a + 64:
                e[i, int(t[i]) - a] -= 1.0
                size_e[i, int(t[i]) - a] += 1.0
        want = e.t() @ x[:4].double()
        bound = (size_e * (dz[:4, rows] + 2.0 ** -20 * (2 + z[:4, rows].abs())) + R.BF16 * 1.01 * e.abs()).t() @ x[:4].double().abs()
        near(dt[rows], want, bound + 64 * R.U * (e.abs().t() @ x[:4].double().abs()), torch.bfloat16)
    want = sum(p[:4, a:a + 65536] @ table[a:a + 65536].double() for a in range(0, V, 65536))
    want = want - table[t[:4]].double()
    size_w = sum(p[:4, a:a + 65536] @ table[a:a + 65536].double().abs() for a in range(0, V, 65536)) + table[t[:4]].double().abs()
    near(dx[:4], want, size_w * (R.BF16 * 1.01 + 1e-3), torch.bfloat16)
    assert not dx[4].any()


@pytest.mark.gpu
def test_two_graphs_in_turn(v):
    g = gen(17)
    cases = [loss_case(g, n, V, 64, torch.bfloat16) for n, V in ((300, 900), (40, 5000))]
    one = torch.ones(1, device="cuda")
    graphs, outs = [], []
    for x, table, t in cases:
        lse = v.cross_entropy(x, table, t)[1]
        v.cross_entropy_backward(one, x, table, t, lse)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            loss, lse = v.cross_entropy(x, table, t)
            outs.append((loss, lse, *v.cross_entropy_backward(one, x, table, t, lse)))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (x, table, t), out in zip(cases, outs):
        loss, lse = v.cross_entropy(x, table, t)
        for a, b in zip(out, (loss, lse, *v.cross_entropy_backward(one, x, table, t, lse))):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_pinned_host_operands_and_rows_around_the_result(v):
    g = gen(13)
    x, table, t = loss_case(g, 20, 60, 32, torch.bfloat16)
    host = [u.cpu().pin_memory() for u in (x, table, t)]
    for a, b in zip(v.cross_entropy(*host), v.cross_entropy(x, table, t)):
        assert torch.equal(a, b)
    wide = torch.full((24, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    a, wg, wu = gated_case(g, 20, 32, 30, torch.bfloat16, "dense")
    v.gated_ff(a, wg, wu, out=wide[2:22, 8:38])
    keep = wide.clone()
    keep[2:22, 8:38] = 7.0
    assert (keep == 7.0).all() and torch.equal(wide[2:22, 8:38], v.gated_ff(a, wg, wu))


@pytest.mark.gpu
def test_own_workspaces_and_shapes(v):
    g = gen(14)
    x, table, t = loss_case(g, 60, 90, 64, torch.bfloat16)
    ws = torch.empty(v.cross_entropy_workspace_bytes(60, 90, 64), dtype=torch.uint8, device="cuda").fill_(255)
    loss, lse = v.cross_entropy(x.view(3, 20, 64), table, t.view(3, 20), workspace=ws)
    assert loss.shape == lse.shape == (3, 20)
    assert torch.equal(loss.flatten(), v.cross_entropy(x, table, t)[0])
    ws = torch.empty(v.cross_entropy_backward_workspace_bytes(60, 90, 64), dtype=torch.uint8, device="cuda").fill_(255)
    one = torch.ones((), device="cuda")
    dx, dt = v.cross_entropy_backward(one, x.view(3, 20, 64), table, t.view(3, 20), lse, workspace=ws)
    assert dx.shape == (3, 20, 64)
    assert v.cross_entropy_backward(one, x, table, t, lse.flatten(), x_grad=False)[0] is None
    assert torch.equal(v.cross_entropy_backward(one, x, table, t, lse.flatten(), x_grad=False)[1], dt)
    only = v.cross_entropy_backward(one, x, table, t, lse.flatten(), table_grad=False)
    assert only[1] is None and torch.equal(only[0], dx.view(60, 64))
    a, wg, wu = gated_case(g, 60, 64, 72, torch.bfloat16, "dense")
    ws = torch.empty(v.gated_ff_workspace_bytes(60, 64, 72), dtype=torch.uint8, device="cuda").fill_(255)
    h, gate, up = v.gated_ff(a.view(3, 20, 64), wg, wu, keep=True, workspace=ws)
    assert h.shape == gate.shape == (3, 20, 72)
    ws = torch.empty(v.gated_ff_backward_workspace_bytes(60, 64, 72), dtype=torch.uint8, device="cuda").fill_(255)
    d = v.gated_ff_backward(h, a.view(3, 20, 64), wg, wu, gate, up, workspace=ws)
    e = v.gated_ff_backward(h, a.view(3, 20, 64), wg, wu, gate, up, weight_grads=False)
    assert torch.equal(d[0], e[0]) and e[1] is None and e[2] is None
    e = v.gated_ff_backward(h, a.view(3, 20, 64), wg, wu, gate, up, x_grad=False)
    assert e[0] is None and torch.equal(d[1], e[1]) and torch.equal(d[2], e[2])


@pytest.mark.gpu
def test_tensor_refusals(v):
    g = gen(15)
    x, table, t = loss_case(g, 8, 20, 64, torch.bfloat16)
    loss, lse = v.cross_entropy(x, table, t)
    one = torch.ones(1, device="cuda")
    w = table
    h, gate, up = v.gated_ff(x, w, w, keep=True)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    back = v.cross_entropy_backward
    bad = [
        lambda: v.cross_entropy(x.half(), table.half(), t), lambda: v.cross_entropy(x.float(), table, t),
        lambda: v.cross_entropy(x, table[:, :32], t), lambda: v.cross_entropy(x, table, t[:4]),
        lambda: v.cross_entropy(x, table, t.float()), lambda: v.cross_entropy(x, table[0], t),
        lambda: v.cross_entropy(x.t(), table, t), lambda: v.cross_entropy(x.cpu(), table, t),
        lambda: v.cross_entropy(x, table, t, loss=loss, lse=loss), lambda: v.cross_entropy(x, table, t, lse=lse.double()),
        lambda: v.cross_entropy(x, table, t, workspace=small),
        lambda: v.cross_entropy(x, table, t, workspace=torch.empty(1 << 20, dtype=torch.uint8).pin_memory()),
        lambda: back(one.double(), x, table, t, lse), lambda: back(torch.ones(3, device="cuda"), x, table, t, lse),
        lambda: back(one, x, table, t, lse[:4]), lambda: back(one, x, table, t, lse, dtable=table),
        lambda: back(one, x, table, t, lse, dx=x.float()), lambda: back(one, x, table, t, lse, base=table[:10]),
        lambda: back(one, x, table, t, lse, base=table.float()), lambda: back(one, x, table, t, lse, workspace=small),
        lambda: v.gated_ff(x, w, w[:10]), lambda: v.gated_ff(x, w, w.float()), lambda: v.gated_ff(x, w, w, activation="relu"),
        lambda: v.gated_ff(x, w, w, out=h[:, :10]), lambda: v.gated_ff(x, w, w, out=h.float()),
        lambda: v.gated_ff(x, w, w, out=x.view(-1)[: 8 * 20].view(8, 20)), lambda: v.gated_ff(x[:, ::2], w[:, :32], w[:, :32]),
        lambda: v.gated_ff_backward(h[:4], x, w, w, gate, up), lambda: v.gated_ff_backward(h, x, w, w, gate.float(), up),
        lambda: v.gated_ff_backward(h, x, w, w, gate, up, dx=x), lambda: v.gated_ff_backward(h, x, w, w, gate, up, dw_gate=w),
        lambda: v.gated_ff_backward(h, x, w, w, gate, up, workspace=small),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((v.VcollError, RuntimeError)) as e:
            f()
        assert not isinstance(e.value, torch.cuda.OutOfMemoryError), i
    torch.cuda.synchronize()


# -------------------------------------- refusals of the C entries (host only)

A, B, C, D_, E, G_ = (0x10000000 * i for i in range(1, 7))
WS = 0x7000000000


def refused(v, f, ok, bad):
    for at, value, want in bad:
        args = list(ok)
        args[at] = value
        assert f(*args) == want, (at, value, v.last_error())


def test_cross_entropy_refusals(v):
    need = v.vcoll_cross_entropy_workspace_bytes(4, 10, 64, v.F32, 0)
    assert need > 0 and v.vcoll_cross_entropy_workspace_bytes(0, 10, 64, v.F32, 0) == 0
    assert v.vcoll_cross_entropy_workspace_bytes(4, 10, 64, 7, 0) == 0
    assert v.vcoll_cross_entropy_workspace_bytes(-4, 10, 64, v.F32, 0) == 0
    ok = [A, 64, B, 64, C, v.I64, 4, 10, 64, D_, E, v.F32, WS, need]
    T, I, X = v.ERR_INVALID_TYPE, v.ERR_INVALID_ARG, v.ERR_UNSUPPORTED
    refused(v, v.vcoll_cross_entropy, ok, [
        (11, 3, T), (5, 2, T), (6, -1, I), (7, -1, I), (8, -1, I), (6, 1 << 31, X), (7, 1 << 31, X), (8, 1 << 31, X),
        (0, 0, I), (2, 0, I), (4, 0, I), (9, 0, I), (10, 0, I), (0, A + 2, I), (4, C + 4, I), (1, 63, I), (3, 63, I),
        (9, A, I), (10, D_, I), (10, D_ + 12, I), (9, C, I), (12, 0, I), (12, WS + 16, I), (13, need - 1, I), (12, A, I),
        (12, D_, I), (3, 1 << 61, I)])
    assert v.vcoll_cross_entropy(0, 64, 0, 64, 0, v.I64, 0, 10, 64, 0, 0, v.F32) == v.OK


def test_cross_entropy_backward_refusals(v):
    need = v.vcoll_cross_entropy_backward_workspace_bytes(4, 10, 64, v.F32, 0)
    assert need > 0
    ok = [A, 4, B, 64, C, 64, D_, v.I64, E, 4, 10, 64, G_, 64, 0, 64, G_ + 65536, 64, v.F32, WS, need]
    T, I, X = v.ERR_INVALID_TYPE, v.ERR_INVALID_ARG, v.ERR_UNSUPPORTED
    refused(v, v.vcoll_cross_entropy_backward, ok, [
        (18, 2, T), (7, 5, T), (1, 3, I), (1, 0, I), (9, -1, I), (10, -2, I), (11, 1 << 31, X), (0, 0, I), (2, 0, I), (4, 0, I),
        (6, 0, I), (8, 0, I), (12, C, I), (16, C, I), (16, G_, I), (14, G_, I), (14, G_ + 65536 + 4, I), (13, 63, I), (17, 60, I),
        (19, 0, I), (20, need - 1, I), (19, B, I), (19, G_, I), (12, B + 16, I)])
    args = list(ok)
    args[12] = args[16] = 0  # nothing wanted
    assert v.vcoll_cross_entropy_backward(*args) == v.OK
    args = list(ok)
    args[14], args[15], args[17] = args[16], 72, 64  # base over dtable with another row stride
    assert v.vcoll_cross_entropy_backward(*args) == I
    args = list(ok)
    args[12], args[13] = B, 72  # dx over x with another row stride
    assert v.vcoll_cross_entropy_backward(*args) == I


def test_gated_ff_refusals(v):
    need = v.vcoll_gated_ff_workspace_bytes(4, 64, 48, v.F32, 0)
    assert need > 0
    ok = [A, 64, B, 64, C, 64, v.GELU, 4, 64, 48, D_, 48, E, 48, G_, 48, v.F32, WS, need]
    T, I, X, O = v.ERR_INVALID_TYPE, v.ERR_INVALID_ARG, v.ERR_UNSUPPORTED, v.ERR_INVALID_OP
    refused(v, v.vcoll_gated_ff, ok, [
        (16, 2, T), (6, 3, O), (6, -1, O), (7, -1, I), (8, -1, I), (9, -1, I), (7, 1 << 31, X), (9, 1 << 31, X), (0, 0, I),
        (2, 0, I), (4, 0, I), (10, 0, I), (1, 63, I), (11, 47, I), (10, A, I), (12, D_, I), (14, E + 16, I), (10, C, I),
        (17, 0, I), (18, need - 1, I), (17, D_, I), (17, WS + 8, I)])
    assert v.vcoll_gated_ff(0, 64, 0, 64, 0, 64, v.SILU, 0, 64, 48, 0, 48, 0, 48, 0, 48, v.F32) == v.OK
    assert v.vcoll_gated_ff(0, 64, 0, 64, 0, 64, v.SILU, 4, 64, 0, 0, 0, 0, 0, 0, 0, v.F32) == v.OK
    # the same weight twice is allowed, and sizes whose bytes fit no memory are not
    args = list(ok)
    args[7], args[8], args[1], args[3], args[5] = (1 << 31) - 2, 1 << 30, 1 << 30, 1 << 30, 1 << 30
    assert v.vcoll_gated_ff(*args) == X


def test_gated_ff_backward_refusals(v):
    need = v.vcoll_gated_ff_backward_workspace_bytes(4, 64, 48, v.F32, 0)
    assert need > 0
    o = 0x90000000
    ok = [A, 48, B, 64, C, 64, D_, 64, E, 48, G_, 48, v.SILU, 4, 64, 48, o, 64, o + 65536, 64, o + 131072, 64, v.F32, WS, need]
    T, I, X, O = v.ERR_INVALID_TYPE, v.ERR_INVALID_ARG, v.ERR_UNSUPPORTED, v.ERR_INVALID_OP
    refused(v, v.vcoll_gated_ff_backward, ok, [
        (22, 9, T), (12, 9, O), (13, -1, I), (14, -1, I), (15, -1, I), (15, 1 << 31, X), (0, 0, I), (2, 0, I), (4, 0, I), (6, 0, I),
        (8, 0, I), (10, 0, I), (1, 47, I), (17, 63, I), (16, B, I), (18, C, I), (20, D_, I), (18, o, I), (20, o + 65536, I),
        (16, A, I), (23, 0, I), (24, need - 1, I), (23, o, I), (23, A, I)])
    args = list(ok)
    args[16] = args[18] = args[20] = 0
    assert v.vcoll_gated_ff_backward(*args) == v.OK
