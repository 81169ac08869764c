"""The layer operators against 64-bit definitions (layers_ref.py), at the
sizes, types, strides and values where they can go wrong, and their refusals.
Every tolerance is the bound that layers_ref.py derives for the inputs."""
import numpy as np
import pytest
import torch

import layers_ref as R

TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def v():
    from collective_reduction_virtual_gb300 import build
    build.build()
    import collective_reduction_virtual_gb300 as vc
    return vc


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def near(got, want, bound, dtype=None):
    """got (a tensor) is within the bound of want, and NaN where want is."""
    got = R.f64(got)
    unit = R.out_unit(dtype) if dtype is not None else 0.0
    tol = bound * 1.01 + unit * (np.abs(want) + bound)
    bad = ~((np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want)) | (got == want))
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4],
                           np.broadcast_to(tol, want.shape)[bad][:4])


def matrix(g, n, d, dtype, layout="dense", scale=1.0, offset=0.0):
    """Random rows: dense, a column slice of wider rows, or starting off any
    16-byte boundary."""
    def fill(t):
        return t.copy_((torch.randn(t.shape, generator=g, device="cuda") * scale + offset).to(dtype))
    if layout == "slice":
        return fill(torch.empty(n, d + 24, dtype=dtype, device="cuda")[:, 8:8 + d])
    if layout == "odd":
        return fill(torch.empty(n * d + 1, dtype=dtype, device="cuda")[1:].view(n, d))
    return fill(torch.empty(n, d, dtype=dtype, device="cuda"))


def like(t, layout):
    if layout == "odd":
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
    if layout == "slice":
        return torch.empty(*t.shape[:-1], t.shape[-1] + 8, dtype=t.dtype, device="cuda")[..., :t.shape[-1]]
    return torch.empty_like(t)


# ---------------------------------------------------------------- embedding

def tokens_of(g, n, V, kind, dtype=torch.int64):
    if kind == "one":  # every token the same
        t = torch.full((n,), min(3, V - 1), device="cuda")
    elif kind == "none":  # nothing inside the table
        t = torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, -1, V)
    elif kind == "skewed":
        t = (V * torch.rand(n, generator=g, device="cuda") ** 6).long().clamp_(max=V - 1)
        t[torch.rand(n, generator=g, device="cuda") < 0.1] = -100
    else:
        t = torch.randint(0, V, (n,), generator=g, device="cuda")
        if n > 2:
            t[0], t[-1] = V - 1, 0
    return t.to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,V,d,layout,index", [
    (1, 7, 1, "dense", torch.int64), (5, 100, 8, "dense", torch.int32),
    (300, 50, 333, "dense", torch.int64), (37, 1000, 256, "slice", torch.int32),
    (1025, 500, 1024, "dense", torch.int64), (64, 90, 514, "odd", torch.int64),
    (3, 11, 20000, "dense", torch.int32), (0, 11, 64, "dense", torch.int64),
])
def test_embedding(v, dtype, n, V, d, layout, index):
    g = gen(n + V + d)
    table = matrix(g, V, d, dtype, layout, 0.5)
    tokens = tokens_of(g, n, V, "skewed", index)
    for scale in (1.0, 7.3):
        out = v.embedding(tokens, table, scale=scale, out=like(torch.empty(n, d, dtype=dtype, device="cuda"), layout))
        t = tokens.long()
        want = table.double()[t.clamp(0, V - 1)] * float(np.float32(scale))  # exact: 24 + 24 bits
        want[(t < 0) | (t >= V)] = 0.0
        assert torch.equal(out, want.float().to(dtype))


@pytest.mark.gpu
def test_embedding_shapes_extreme_tokens_and_an_empty_table(v):
    g = gen(1)
    table = matrix(g, 10, 64, torch.float32)
    tokens = torch.tensor([[0, 9, 10], [-1, 2 ** 40, -2 ** 40]], device="cuda")
    out = v.embedding(tokens, table)
    assert out.shape == (2, 3, 64)
    assert torch.equal(out[0, 1], table[9]) and not out[0, 2].any() and not out[1].any()
    small = torch.tensor([2 ** 31 - 1, -2 ** 31, 4], device="cuda", dtype=torch.int32)
    out = v.embedding(small, table)
    assert not out[:2].any() and torch.equal(out[2], table[4])
    assert not v.embedding(tokens, table[:0]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,table_dtype", [(a, b) for a in TYPES for b in TYPES])
@pytest.mark.parametrize("n,V,d,kind,layout", [
    (1, 1, 1, "any", "dense"), (33, 5, 40, "any", "dense"), (1000, 700, 96, "any", "slice"),
    (2500, 40, 129, "skewed", "dense"), (4100, 3000, 64, "skewed", "odd"),
    (700, 30, 515, "one", "dense"), (300, 20, 64, "none", "dense"), (0, 9, 64, "any", "dense"),
    (9000, 70000, 16, "skewed", "dense"), (20000, 17, 8, "skewed", "dense"),
    (513, 600000, 2, "any", "dense"), (200, 50, 2500, "skewed", "slice"),
    (512, 300, 72, "one", "odd"), (512, 2000, 258, "skewed", "dense"), (513, 2000, 258, "one", "dense"),
    (4096, 9000, 24, "skewed", "dense"), (4097, 65, 24, "any", "slice"), (6000, 3, 1000, "any", "dense"),
    (5000, 40, 129, "none", "dense"), (70000, 513, 16, "skewed", "dense"),
    (2048, 30, 256, "one", "dense"), (2048, 9000, 200, "skewed", "odd"), (2049, 300, 40, "any", "dense"),
    (1500, 70000, 12, "skewed", "dense"), (1800, 500, 1030, "skewed", "dense"), (900, 12, 700, "skewed", "slice"),
])
def test_embedding_backward(v, dtype, table_dtype, n, V, d, kind, layout):
    g = gen(n + V + d)
    tokens = tokens_of(g, n, V, kind, torch.int32 if n % 2 else torch.int64)
    grad = matrix(g, n, d, dtype, layout)
    base = matrix(g, V, d, table_dtype, layout, 3.0)
    host, t = R.f64(grad), tokens.cpu().numpy()
    for scale in (1.0, 0.37):
        s = float(np.float32(scale))
        got = v.embedding_backward(grad, tokens, V, scale=scale, dtype=table_dtype,
                                   out=like(base, layout))
        near(got, *R.lookup_grad(host, t, V, s, None), table_dtype)
    want = R.lookup_grad(host, t, V, s, R.f64(base))
    got = v.embedding_backward(grad, tokens, V, scale=scale, base=base)
    near(got, *want, table_dtype)
    kept = base.clone()
    assert v.embedding_backward(grad, tokens, V, scale=scale, base=base, out=base) is base
    near(base, *want, table_dtype)
    # in place, rows of tokens that do not occur are not written
    untouched = np.setdiff1d(np.arange(V), t)
    assert torch.equal(base[untouched], kept[untouched])
    assert torch.equal(base, got)


@pytest.mark.gpu
def test_embedding_backward_repeats_its_bits_and_sums_in_token_order(v):
    g = gen(5)
    tokens = tokens_of(g, 50000, 300, "skewed")
    grad = matrix(g, 50000, 70, torch.float32)
    a = v.embedding_backward(grad, tokens, 300)
    for _ in range(3):
        assert torch.equal(a, v.embedding_backward(grad, tokens, 300))
    # few rows of each token: their order alone decides the bits
    tokens = torch.tensor([2, 1, 2, 0, 2], device="cuda")
    grad = torch.tensor([[2.0 ** 24], [1.0], [1.0], [5.0], [-2.0 ** 24]], device="cuda")
    assert v.embedding_backward(grad, tokens, 3).flatten().tolist() == [5.0, 1.0, 0.0]


@pytest.mark.gpu
def test_embedding_backward_keeps_nan_and_infinity_in_their_rows(v):
    g = gen(6)
    grad = matrix(g, 64, 40, torch.float32)
    tokens = torch.arange(64, device="cuda") % 7
    tokens[10] = -1  # an ignored row holds anything
    grad[10] = float("nan")
    grad[20, 3] = float("inf")
    grad[21, 5] = float("nan")
    out = v.embedding_backward(grad, tokens, 7)
    bad = ~torch.isfinite(out)
    assert bad.sum() == 2 and out[20 % 7, 3] == float("inf") and torch.isnan(out[21 % 7, 5])


@pytest.mark.gpu
def test_embedding_is_the_adjoint_of_its_gradient(v):
    # <grad, embedding(T + dT) - embedding(T)> / eps = <table gradient, dT>: the lookup is linear,
    # so its differences are exact up to rounding
    g = gen(7)
    V, d, n = 37, 48, 301
    table, dt = matrix(g, V, d, torch.float32), matrix(g, V, d, torch.float32)
    grad = matrix(g, n, d, torch.float32)
    tokens = tokens_of(g, n, V, "skewed")
    moved = v.embedding(tokens, table + dt, 0.5).double() - v.embedding(tokens, table, 0.5).double()
    left = (grad.double() * moved).sum().item()
    right = (v.embedding_backward(grad, tokens, V, 0.5).double() * dt.double()).sum().item()
    size = (grad.double().abs() * (table.double().abs().amax() + dt.double().abs().amax())).sum().item()
    assert abs(left - right) <= 8 * R.U * size + n * R.U * size


# --------------------------------------------------------------- layer norm

SHAPES = [(1, 1), (3, 2), (2, 31), (5, 128), (17, 129), (9, 1000), (130, 256), (4, 1001), (33, 4096),
          (2, 8200), (3, 16384), (2, 70001), (1200, 72), (7, 130), (6, 514), (5, 1026), (4, 4098),
          (3, 8202), (2, 16382)]


def weights(g, d, wtype, which="both"):
    w = (torch.randn(d, generator=g, device="cuda") * 0.3 + 1.0).to(wtype)
    b = (torch.randn(d, generator=g, device="cuda") * 0.3).to(wtype)
    return (w if which != "none" and which != "bias" else None,
            b if which != "none" and which != "weight" else None)


def host_weights(w, b, d):
    return (R.f64(w) if w is not None else np.ones(d), R.f64(b) if b is not None else np.zeros(d))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d", SHAPES)
@pytest.mark.parametrize("layout", ["dense", "slice", "odd"])
def test_layer_norm(v, dtype, n, d, layout):
    g = gen(n * 7 + d)
    x = matrix(g, n, d, dtype, layout, 2.0, 1.0)
    wtype = TYPES[(n + d) % 2]
    w, b = weights(g, d, wtype, ["both", "weight", "bias", "none"][(n + d) % 4])
    y, mean, rstd = v.layer_norm(x, w, b, eps=1e-4, out=like(x, layout))
    wy, wm, wr, _, bm, br, _, by = R.norm(R.f64(x), *host_weights(w, b, d), float(np.float32(1e-4)))
    near(mean, wm, bm + R.U * np.abs(wm))
    near(rstd, wr, wr * br)
    near(y, wy, by, dtype)
    # in place
    assert v.layer_norm(x, w, b, eps=1e-4, out=x)[0] is x
    assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wtype", [(a, b) for a in TYPES for b in TYPES])
@pytest.mark.parametrize("at", [1, 2, 4])
def test_weights_at_any_alignment(v, dtype, wtype, at):
    # weight and bias off the 16-byte boundary beside aligned rows
    g = gen(at)
    n, d = 70, 1024
    x, grad = matrix(g, n, d, dtype), matrix(g, n, d, dtype)
    aligned = weights(g, d, wtype)
    flat = torch.empty(2 * d + 16, dtype=wtype, device="cuda")
    w, b = flat[at:at + d].copy_(aligned[0]), flat[d + 8 + at:2 * d + 8 + at].copy_(aligned[1])
    wy, _, _, _, _, _, _, by = R.norm(R.f64(x), *host_weights(w, b, d), float(np.float32(1e-5)))
    y, mean, rstd = v.layer_norm(x, w, b)
    near(y, wy, by, dtype)
    wy, _, _, _, _, _, _, by = R.norm(R.f64(x), np.ones(d), R.f64(b), float(np.float32(1e-5)))
    near(v.layer_norm(x, None, b)[0], wy, by, dtype)
    h = (R.f64(x) - R.f64(mean)[:, None]) * R.f64(rstd)[:, None]
    wx, ww, wb, bx, bw, bb = R.norm_grad(R.f64(grad), h, R.f64(rstd), R.f64(w))
    dx, dw, db = v.layer_norm_backward(grad, x, mean, rstd, w)
    near(dx, wx, bx, dtype)
    near(dw, ww, bw, wtype)
    y2, rstd, k = v.layer_norm_checkpoint8(x, w, b)
    assert torch.equal(y2, y)
    # no sums: the same bits whatever the alignment
    assert torch.equal(v.checkpoint8_restore(k, w, b, dtype=dtype),
                       v.checkpoint8_restore(k, *aligned, dtype=dtype))
    assert torch.equal(v.checkpoint8_restore(k, None, b, dtype=dtype),
                       v.checkpoint8_restore(k, None, aligned[1], dtype=dtype))
    kept = R.unpack8(k.codes.cpu().numpy(), k.scales.cpu().numpy())
    wx, ww, wb, bx, bw, bb = R.norm_grad(R.f64(grad), kept, R.f64(rstd), R.f64(w))
    dx, dw, db = v.layer_norm_backward_checkpoint8(grad, k, rstd, w)
    near(dx, wx, bx, dtype)
    near(dw, ww, bw, wtype)
    near(db, wb, bb, wtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_layer_norm_constant_rows_offsets_and_special_values(v, dtype):
    g = gen(3)
    d = 384
    x = torch.randn(8, d, generator=g, device="cuda")
    x[0] = 0.0
    x[1] = 5.0  # no deviation at all: y is the bias
    x[2] = x[2] * 0.5 + 4096.0  # a large offset
    x[3, 7] = float("nan")
    x[4, 9] = float("inf")
    x[5] *= 1e-20  # far below eps
    x = x.to(dtype)
    b = torch.randn(d, generator=g, device="cuda").to(dtype)
    y, mean, rstd = v.layer_norm(x, None, b, eps=1e-5)
    assert torch.equal(y[0], b) and torch.equal(y[1], b)
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    rows = [0, 1, 2, 5, 6, 7]
    wy, _, _, _, _, _, _, by = R.norm(R.f64(x)[rows], np.ones(d), R.f64(b), float(np.float32(1e-5)))
    near(y[rows], wy, by, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d", SHAPES + [(1, 640), (5000, 40)])
@pytest.mark.parametrize("layout", ["dense", "slice", "odd"])
def test_layer_norm_backward(v, dtype, n, d, layout):
    g = gen(n * 3 + d)
    x = matrix(g, n, d, dtype, layout, 2.0, 0.5)
    grad = matrix(g, n, d, dtype, layout)
    wtype = TYPES[(n + d) % 2]
    w, _ = weights(g, d, wtype, "none" if n % 5 == 3 else "both")
    _, mean, rstd = v.layer_norm(x, w)
    h = (R.f64(x) - R.f64(mean)[:, None]) * R.f64(rstd)[:, None]
    wx, ww, wb, bx, bw, bb = R.norm_grad(R.f64(grad), h, R.f64(rstd), host_weights(w, None, d)[0])
    out = like(x, layout)
    flat = torch.empty(2 * d + 1, dtype=w.dtype if w is not None else torch.float32, device="cuda")
    dx, dw, db = v.layer_norm_backward(grad, x, mean, rstd, w, dx=out, dweight=flat[1:d + 1],
                                       dbias=flat[d + 1:])
    assert dx is out
    near(dx, wx, bx, dtype)
    near(dw, ww, bw, dw.dtype)
    near(db, wb, bb, db.dtype)
    # parts of it give the same bits, in place too
    only, a, b = v.layer_norm_backward(grad, x, mean, rstd, w, weight_grads=False)
    assert a is None and b is None and torch.equal(only, dx)
    _, a, b = v.layer_norm_backward(grad, x, mean, rstd, w, dbias=torch.empty_like(db),
                                    weight_grads=False)
    assert a is None and torch.equal(b, db)
    v.layer_norm_backward(grad, x, mean, rstd, w, dx=grad, weight_grads=False)
    assert torch.equal(grad, dx)


def close(got, want, bound, dtype):
    """near(), on the GPU"""
    tol = bound * 1.01 + R.out_unit(dtype) * (want.abs() + bound)
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d", [(20011, 16), (20000, 40), (30001, 64), (3000, 200), (5000, 128), (5000, 256), (5000, 512), (3000, 1024), (2500, 1536),
                                 (1500, 4096), (700, 8192), (700, 12288), (700, 16384), (100, 32768)])
@pytest.mark.parametrize("at", [0, 2, 1])
def test_layer_norm_every_width_and_alignment_over_many_rows(v, dtype, n, d, at):
    # rows enough for every CTA to take several, and the accesses that 16-, 4- and 2- (4-) byte
    # alignment allow, at widths on each side of how a row is shared out
    g = gen(n + d + at)

    def place(t):
        return torch.empty(t.numel() + at, dtype=t.dtype, device="cuda")[at:].view(t.shape).copy_(t)

    x, grad = (place(matrix(g, n, d, dtype, "dense", 2.0, 0.3)) for _ in range(2))
    w, b = (place(t) for t in weights(g, d, dtype))
    w64, b64, g64 = w.double(), b.double(), grad.double()
    wy, wm, wr, h, bm, br, dh, by = R.norm(x.double(), w64, b64, float(np.float32(1e-5)))
    y, mean, rstd = v.layer_norm(x, w, b, out=place(x))
    close(mean, wm, bm + R.U * wm.abs(), torch.float32)
    close(rstd, wr, wr * br, torch.float32)
    close(y, wy, by, dtype)
    y2, rstd, k = v.layer_norm_checkpoint8(x, w, b, out=place(x))
    assert torch.equal(y, y2)
    step = k.scales.double().repeat_interleave(128, 1)[:, :d]
    kept = k.codes[:, :d].double() * step
    assert ((kept - h).abs() <= 0.5 * step * (1 + 300 * R.U) + dh).all()
    back = v.checkpoint8_restore(k, w, b, dtype=dtype, out=place(x))
    close(back, kept * w64 + b64, 3 * R.U * ((kept * w64).abs() + b64.abs()), dtype)
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for form, hh in ((0, h), (1, kept)):
        wx, ww, wb, bx, bw, bb = R.norm_grad(g64, hh, rstd.double(), w64)
        if form:
            dx, dw, db = v.layer_norm_backward_checkpoint8(grad, k, rstd, w, dx=place(x))
        else:
            dx, dw, db = v.layer_norm_backward(grad, x, mean, rstd, w, dx=place(x))
        close(dx, wx, bx, dtype)
        close(dw, ww, bw, dtype)
        close(db, wb, bb, dtype)


@pytest.mark.gpu
def test_layer_norm_backward_in_place_over_both_inputs(v):
    g = gen(11)
    for d in (96, 1001, 4096):
        x, grad = matrix(g, 50, d, torch.bfloat16), matrix(g, 50, d, torch.bfloat16)
        _, mean, rstd = v.layer_norm(x)
        want = v.layer_norm_backward(grad, x, mean, rstd)
        for over in ("grad", "x"):
            xs, gs = x.clone(), grad.clone()
            got = v.layer_norm_backward(gs, xs, mean, rstd, dx=gs if over == "grad" else xs)
            for a, b in zip(got, want):
                assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [False, True])
def test_layer_norm_of_no_rows(v, kept):
    x = torch.empty(0, 96, device="cuda")
    w = torch.ones(96, device="cuda")
    if kept:
        y, rstd, c = v.layer_norm_checkpoint8(x, w)
        dx, dw, db = v.layer_norm_backward_checkpoint8(x, c, rstd, w)
    else:
        y, mean, rstd = v.layer_norm(x, w)
        dx, dw, db = v.layer_norm_backward(x, x, mean, rstd, w)
    assert y.shape == dx.shape == (0, 96)
    assert not dw.any() and not db.any()  # the gradient of nothing is zero, and is written
    assert v.layer_norm(torch.empty(4, 0, device="cuda"))[0].shape == (4, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [False, True])
def test_layer_norm_gradient_against_differences(v, kept):
    # central differences, in 64 bits, of sum(c * layer norm): e^2 times the third derivative, and
    # the rounding of the 64-bit sums over e, stay below 1e-6 here; the kept form is off by half a
    # step of its codes instead, 1/254 of a block's largest value, in each h
    g = gen(13)
    n, d, e = 4, 24, 1e-5
    x = matrix(g, n, d, torch.float32)
    c = matrix(g, n, d, torch.float32)
    w, b = weights(g, d, torch.float32)
    hx, hc, (hw, hb) = R.f64(x), R.f64(c), host_weights(w, b, d)

    def loss(x, w, b):
        return (hc * R.norm(x, w, b, 1e-5)[0]).sum()

    def slope(i, a):
        up, dn = [hx.copy(), hw.copy(), hb.copy()], [hx.copy(), hw.copy(), hb.copy()]
        up[a].flat[i] += e
        dn[a].flat[i] -= e
        return (loss(*up) - loss(*dn)) / (2 * e)

    if kept:
        _, rstd, k = v.layer_norm_checkpoint8(x, w, b, eps=1e-5)
        got = v.layer_norm_backward_checkpoint8(c, k, rstd, w)
    else:
        _, mean, rstd = v.layer_norm(x, w, b, eps=1e-5)
        got = v.layer_norm_backward(c, x, mean, rstd, w)
    h = R.norm(hx, hw, hb, 1e-5)[3]
    step = np.abs(h).max() / 254 if kept else 0.0
    gs = np.abs(hc * hw)
    tol = [np.max(R.f64(rstd)) * step * (2 * np.abs(h).max() * gs.max() + gs.max()) + 2e-5,
           step * np.abs(hc).sum(0).max() + 2e-5, 2e-5]
    for a, t in enumerate(got):
        want = np.array([slope(i, a) for i in range(t.numel())])
        assert np.abs(R.f64(t).ravel() - want).max() <= tol[a]


# ------------------------------------------------------- 8-bit activations

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d", SHAPES)
@pytest.mark.parametrize("layout", ["dense", "slice", "odd"])
def test_checkpoint8(v, dtype, n, d, layout):
    g = gen(n + d)
    x = matrix(g, n, d, dtype, layout, 3.0)
    x[0, :min(d, 130)] = 0.0
    k = v.checkpoint8(x)
    codes, scales = R.pack8(R.f64(x))
    assert k.codes.shape[-1] % 16 == 0 and k.shape == x.shape
    assert np.array_equal(k.codes[:, :d].cpu().numpy(), codes)
    assert not k.codes[:, d:].any()
    assert np.array_equal(k.scales.cpu().numpy(), scales)
    want = R.unpack8(codes, scales)
    step = np.repeat(scales.astype(np.float64), R.BLOCK, 1)[:, :d]
    assert (np.abs(want - R.f64(x)) <= 0.5 * step * (1 + 300 * R.U)).all()
    near(v.checkpoint8_restore(k, dtype=dtype), want, 0.0 * want, dtype)
    w, b = weights(g, d, TYPES[n % 2], ["both", "weight", "bias"][n % 3])
    hw, hb = host_weights(w, b, d)
    out = like(x, layout)
    assert v.checkpoint8_restore(k, w, b, out=out) is out
    near(out, want * hw + hb, 3 * R.U * (np.abs(want * hw) + np.abs(hb)), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_checkpoint8_special_values(v, dtype):
    d = 5 * 128 + 40
    x = torch.randn(6, d, generator=gen(2), device="cuda")
    x[0, 130] = float("nan")
    x[1, 300] = float("-inf")
    x[2] *= 2.0 ** -126  # blocks of subnormals and below 2^-100: zeros
    x[3] *= 2.0 ** -99
    x[4] = 3e38 * torch.sign(x[4])
    x[5, :128] = 0.0
    x[5, 128] = -0.0
    x = x.to(dtype)
    k = v.checkpoint8(x)
    codes, scales = R.pack8(R.f64(x))
    assert np.array_equal(k.codes[:, :d].cpu().numpy(), codes)
    assert np.array_equal(k.scales.cpu().numpy(), scales, equal_nan=True)
    out = v.checkpoint8_restore(k, dtype=dtype)
    bad = torch.isnan(out)
    assert bad[0, 128:256].all() and bad[1, 256:384].all() and bad.sum() == 256
    assert not out[2].any() and torch.isfinite(out[4]).all() and not out[5, :128].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d", SHAPES)
@pytest.mark.parametrize("layout", ["dense", "slice", "odd"])
def test_layer_norm_checkpoint8(v, dtype, n, d, layout):
    g = gen(n * 5 + d)
    x = matrix(g, n, d, dtype, layout, 2.0, 0.5)
    grad = matrix(g, n, d, dtype, layout)
    w, b = weights(g, d, TYPES[n % 2], "both" if d % 3 else "none")
    y, rstd, k = v.layer_norm_checkpoint8(x, w, b, out=like(x, layout))
    hw, hb = host_weights(w, b, d)
    wy, _, wr, h, _, br, dh, by = R.norm(R.f64(x), hw, hb, float(np.float32(1e-5)))
    near(y, wy, by, dtype)
    near(rstd, wr, wr * br)
    assert torch.equal(y, v.layer_norm(x, w, b)[0])
    # each code is within half a step of h, which is off by at most dh itself
    kept = R.unpack8(k.codes[:, :d].cpu().numpy(), k.scales.cpu().numpy())
    step = np.repeat(R.f64(k.scales), R.BLOCK, 1)[:, :d]
    assert (np.abs(kept - h) <= 0.5 * step * (1 + 300 * R.U) + dh).all()
    top = np.abs(h).reshape(n, -1).max()
    assert (step <= (top + dh.max()) / 127 * (1 + 4 * R.U)).all()
    assert not k.codes[:, d:].any()
    # the backward pass, from what was kept
    wx, ww, wb, bx, bw, bb = R.norm_grad(R.f64(grad), kept, R.f64(rstd), hw)
    dx, dw, db = v.layer_norm_backward_checkpoint8(grad, k, rstd, w, dx=like(x, layout))
    near(dx, wx, bx, dtype)
    near(dw, ww, bw, dw.dtype)
    near(db, wb, bb, db.dtype)
    v.layer_norm_backward_checkpoint8(grad, k, rstd, w, dx=grad)
    assert torch.equal(grad, dx)


# ------------------------------------------- streams, offsets, other callers

@pytest.mark.gpu
def test_calls_on_another_stream_and_in_a_graph(v):
    g = gen(17)
    x, w = matrix(g, 513, 768, torch.bfloat16), torch.ones(768, device="cuda", dtype=torch.bfloat16)
    tokens = tokens_of(g, 513, 90, "skewed")

    def step(stream=None):
        y, rstd, k = v.layer_norm_checkpoint8(x, w, stream=stream)
        dx, dw, db = v.layer_norm_backward_checkpoint8(y, k, rstd, w, stream=stream)
        back = v.checkpoint8_restore(k, w, dtype=x.dtype, stream=stream)
        t = v.embedding_backward(dx, tokens, 90, 2.0, stream=stream)
        return [y, dx, dw, db, back, t, v.embedding(tokens, t, 0.5, stream=stream)]

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        got = step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_offsets_beyond_32_bits(v):
    # three rows 2^30 elements apart in one buffer
    big = torch.empty(2 * 2 ** 30 + 512, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(big, (3, 512), (2 ** 30, 1))
    dense = matrix(gen(19), 3, 512, torch.bfloat16)
    x.copy_(dense)
    tokens = torch.tensor([2, 0, 5], device="cuda")
    assert torch.equal(v.embedding(tokens[:2], x, 2.0), v.embedding(tokens[:2], dense, 2.0))
    want = v.layer_norm_checkpoint8(dense)
    got = v.layer_norm_checkpoint8(x)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2].codes, want[2].codes)
    y, mean, rstd = v.layer_norm(dense)
    assert torch.equal(v.layer_norm_backward(x, x, mean, rstd)[0],
                       v.layer_norm_backward(dense, dense, mean, rstd)[0])
    t = v.embedding_backward(x, tokens, 6)
    assert torch.equal(t, v.embedding_backward(dense, tokens, 6))
    v.embedding_backward(dense, tokens % 3, 3, out=x)
    assert torch.equal(x, v.embedding_backward(dense, tokens % 3, 3))
    assert torch.equal(v.checkpoint8(x).codes, v.checkpoint8(x.contiguous()).codes)


@pytest.mark.gpu
def test_pinned_host_tables_and_leading_axes(v):
    table = torch.randn(50, 96).pin_memory()
    tokens = torch.randint(0, 50, (4, 5), device="cuda")
    out = v.embedding(tokens, table)
    assert torch.equal(out.cpu(), table[tokens.cpu()])
    y, mean, rstd = v.layer_norm(out)
    assert y.shape == out.shape and mean.shape == rstd.shape == (4, 5)
    dx, dw, db = v.layer_norm_backward(out, out, mean, rstd)
    flat = v.layer_norm_backward(out.view(20, 96), out.view(20, 96), mean.view(-1), rstd.view(-1))
    assert torch.equal(dx.view(20, 96), flat[0]) and torch.equal(dw, flat[1])
    part = torch.randn(6, 7, 64, device="cuda")[:, :, 16:48]  # leading axes that fold into one stride
    assert torch.equal(v.layer_norm(part)[0], v.layer_norm(part.contiguous())[0])


@pytest.mark.gpu
def test_tensor_layer_refusals(v):
    x, w = torch.randn(8, 64, device="cuda"), torch.ones(64, device="cuda")
    y, mean, rstd = v.layer_norm(x, w)
    k = v.checkpoint8(x)
    t = torch.zeros(8, dtype=torch.int64, device="cuda")
    bad = [
        lambda: v.layer_norm(x.t()), lambda: v.layer_norm(x.half()), lambda: v.layer_norm(x.cpu()),
        lambda: v.layer_norm(x, w[:32]), lambda: v.layer_norm(x, w, w.bfloat16()),
        lambda: v.layer_norm(x, out=x.bfloat16()), lambda: v.layer_norm(x, out=x[:4]),
        lambda: v.layer_norm(x[:1].expand(8, 64)), lambda: v.layer_norm(x[:, ::2]),
        lambda: v.layer_norm(x, out=x.view(-1)[: 8 * 63].view(8, 63)),
        lambda: v.layer_norm_backward(x, x, mean[:4], rstd), lambda: v.layer_norm_backward(x, x.bfloat16(), mean, rstd),
        lambda: v.layer_norm_backward(x, x, mean.double(), rstd),
        lambda: v.layer_norm_backward(x, x, mean, rstd, w, dweight=w.bfloat16()),
        lambda: v.layer_norm_backward(x, x, mean, rstd, w, dweight=w),  # over the weight itself
        lambda: v.layer_norm_backward_checkpoint8(x[:4], k, rstd[:4]),
        lambda: v.checkpoint8(x.double()), lambda: v.checkpoint8_restore(k, out=x[:, :32]),
        lambda: v.checkpoint8_restore(k, dtype=torch.float16),
        lambda: v.embedding(t.float(), x), lambda: v.embedding(t, x.half()), lambda: v.embedding(t, x[0]),
        lambda: v.embedding(t, x, out=x), lambda: v.embedding(t.view(2, 4).t(), x),
        lambda: v.embedding_backward(x, t[:4], 10), lambda: v.embedding_backward(x, t, 10, out=x),
        lambda: v.embedding_backward(x, t, 10, base=torch.zeros(9, 64, device="cuda")),
        lambda: v.embedding_backward(x, t, 10, base=torch.zeros(10, 64, device="cuda"), dtype=torch.bfloat16),
        lambda: v.embedding_backward(x.repeat(500, 1), t.repeat(500), 10,
                                     workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: v.embedding_backward(x, t, -1),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((v.VcollError, RuntimeError)) as e:
            f()
        assert not isinstance(e.value, torch.cuda.OutOfMemoryError), i
    torch.cuda.synchronize()  # nothing was enqueued that fails


# -------------------------------------- refusals of the C entries (host only)

A, B, C, D_, E = (0x10000000 * i for i in range(1, 6))


def test_embedding_refusals(v):
    f = v.vcoll_embedding
    ok = [A, v.I64, 4, B, 64, 10, 64, 1.0, C, 64, v.F32]
    for at, value, want in [(1, 7, v.ERR_INVALID_TYPE), (10, 2, v.ERR_INVALID_TYPE),
                            (2, -1, v.ERR_INVALID_ARG), (5, -1, v.ERR_INVALID_ARG),
                            (6, -1, v.ERR_INVALID_ARG), (2, 1 << 31, v.ERR_UNSUPPORTED),
                            (0, 0, v.ERR_INVALID_ARG), (3, 0, v.ERR_INVALID_ARG),
                            (8, 0, v.ERR_INVALID_ARG), (0, A + 4, v.ERR_INVALID_ARG),
                            (3, B + 2, v.ERR_INVALID_ARG), (8, C + 1, v.ERR_INVALID_ARG),
                            (4, 63, v.ERR_INVALID_ARG), (9, 63, v.ERR_INVALID_ARG),
                            (9, 1 << 62, v.ERR_INVALID_ARG), (8, B + 256, v.ERR_INVALID_ARG),
                            (8, A, v.ERR_INVALID_ARG)]:
        args = list(ok)
        args[at] = value
        assert f(*args) == want, (at, value, v.last_error())
    assert f(0, v.I64, 0, 0, 64, 10, 64, 1.0, 0, 64, v.F32) == v.OK  # no tokens
    assert f(0, v.I64, 4, 0, 0, 10, 0, 1.0, 0, 0, v.F32) == v.OK  # no columns


def test_embedding_backward_refusals(v):
    f = v.vcoll_embedding_backward
    assert v.vcoll_embedding_backward_workspace_bytes(4, 10, 64) == 0  # short lists take none
    need = v.vcoll_embedding_backward_workspace_bytes(4000, 10, 64)
    assert need > 0
    ok = [A, 64, v.F32, B, v.I64, 4000, 10, 64, 1.0, 0, 64, C, 64, v.F32, D_, need]
    for at, value, want in [(2, 2, v.ERR_INVALID_TYPE), (13, 5, v.ERR_INVALID_TYPE),
                            (4, 2, v.ERR_INVALID_TYPE), (5, -1, v.ERR_INVALID_ARG),
                            (6, -1, v.ERR_INVALID_ARG), (7, 1 << 31, v.ERR_UNSUPPORTED),
                            (0, 0, v.ERR_INVALID_ARG), (3, 0, v.ERR_INVALID_ARG),
                            (11, 0, v.ERR_INVALID_ARG), (1, 10, v.ERR_INVALID_ARG),
                            (12, 10, v.ERR_INVALID_ARG), (9, C + 4, v.ERR_INVALID_ARG),
                            (11, A, v.ERR_INVALID_ARG), (14, 0, v.ERR_INVALID_ARG),
                            (15, need - 1, v.ERR_INVALID_ARG), (14, D_ + 16, v.ERR_INVALID_ARG),
                            (14, C, v.ERR_INVALID_ARG)]:
        args = list(ok)
        args[at] = value
        assert f(*args) == want, (at, value, v.last_error())
    # base over table_grad with another row stride
    args = list(ok)
    args[9], args[10], args[12] = C, 64, 72
    assert f(*args) == v.ERR_INVALID_ARG
    assert f(0, 64, v.F32, 0, v.I64, 4, 0, 64, 1.0, 0, 64, 0, 64, v.F32) == v.OK  # no table
    assert f(0, 64, v.F32, 0, v.I64, 0, 10, 64, 1.0, C, 64, C, 64, v.F32) == v.OK  # nothing to add


def test_layer_norm_refusals(v):
    f = v.vcoll_layer_norm
    ok = [A, 64, B, B + 4096, v.F32, 4, 64, 1e-5, C, 64, D_, D_ + 4096, v.F32]
    for at, value, want in [(12, 2, v.ERR_INVALID_TYPE), (4, 2, v.ERR_INVALID_TYPE),
                            (5, -1, v.ERR_INVALID_ARG), (6, -1, v.ERR_INVALID_ARG),
                            (0, 0, v.ERR_INVALID_ARG), (8, 0, v.ERR_INVALID_ARG),
                            (0, A + 2, v.ERR_INVALID_ARG), (1, 60, v.ERR_INVALID_ARG),
                            (8, A + 16, v.ERR_INVALID_ARG), (8, B, v.ERR_INVALID_ARG),
                            (11, D_ + 8, v.ERR_INVALID_ARG), (10, A, v.ERR_INVALID_ARG)]:
        args = list(ok)
        args[at] = value
        assert f(*args) == want, (at, value, v.last_error())
    args = list(ok)
    args[8], args[9] = A, 72  # over x with another row stride
    assert f(*args) == v.ERR_INVALID_ARG
    assert f(0, 64, 0, 0, v.F32, 0, 64, 1e-5, 0, 64, 0, 0, v.F32) == v.OK
    assert f(0, 0, 0, 0, v.F32, 4, 0, 1e-5, 0, 0, 0, 0, v.F32) == v.OK
    g = v.vcoll_layer_norm_checkpoint8
    ok = [A, 64, B, B + 4096, v.F32, 4, 64, 1e-5, C, 64, D_, E, 64, E + 4096, v.F32]
    for at, value in [(11, 0), (11, E + 8), (12, 72), (12, 48), (13, 0), (13, E), (13, E + 4098)]:
        args = list(ok)
        args[at] = value
        assert g(*args) == v.ERR_INVALID_ARG, (at, value)


def test_layer_norm_backward_refusals(v):
    f = v.vcoll_layer_norm_backward
    need = v.vcoll_layer_norm_workspace_bytes(4, 64)
    ws = 0x70000000
    ok = [A, 64, B, 64, D_, D_ + 4096, E, v.F32, 4, 64, C, 64, E + 4096, E + 8192, v.F32, ws, need]
    for at, value, want in [(14, 2, v.ERR_INVALID_TYPE), (7, 2, v.ERR_INVALID_TYPE),
                            (8, -1, v.ERR_INVALID_ARG), (9, -2, v.ERR_INVALID_ARG),
                            (0, 0, v.ERR_INVALID_ARG), (2, 0, v.ERR_INVALID_ARG),
                            (4, 0, v.ERR_INVALID_ARG), (5, 0, v.ERR_INVALID_ARG),
                            (10, A + 64, v.ERR_INVALID_ARG), (12, E, v.ERR_INVALID_ARG),
                            (13, E + 4096, v.ERR_INVALID_ARG), (11, 63, v.ERR_INVALID_ARG)]:
        args = list(ok)
        args[at] = value
        assert f(*args) == want, (at, value, v.last_error())
    if need:
        for at, value in [(15, 0), (15, ws + 128), (16, need - 1), (15, A)]:
            args = list(ok)
            args[at] = value
            assert f(*args) == v.ERR_INVALID_ARG, (at, value)
    g = v.vcoll_layer_norm_backward_checkpoint8
    ok = [A, 64, B, 64, B + 4096, D_, E, v.F32, 4, 64, C, 64, E + 4096, E + 8192, v.F32, ws, need]
    for at, value in [(2, 0), (2, B + 8), (3, 40), (4, 0), (5, 0), (10, B)]:
        args = list(ok)
        args[at] = value
        assert g(*args) == v.ERR_INVALID_ARG, (at, value)


def test_checkpoint8_refusals(v):
    f = v.vcoll_checkpoint8
    ok = [A, 64, 4, 64, B, 64, C, v.F32]
    for at, value, want in [(7, 2, v.ERR_INVALID_TYPE), (2, -1, v.ERR_INVALID_ARG),
                            (3, 1 << 31, v.ERR_UNSUPPORTED), (0, 0, v.ERR_INVALID_ARG),
                            (4, 0, v.ERR_INVALID_ARG), (6, 0, v.ERR_INVALID_ARG),
                            (4, B + 4, v.ERR_INVALID_ARG), (5, 72, v.ERR_INVALID_ARG),
                            (5, 48, v.ERR_INVALID_ARG), (4, A, v.ERR_INVALID_ARG),
                            (6, B + 16, v.ERR_INVALID_ARG), (1, 2, v.ERR_INVALID_ARG)]:
        args = list(ok)
        args[at] = value
        assert f(*args) == want, (at, value, v.last_error())
    # a row of 50 columns is written up to 64: the stride must hold it
    assert f(A, 64, 4, 50, B, 48, C, v.F32) == v.ERR_INVALID_ARG
    f = v.vcoll_checkpoint8_restore
    ok = [A, 64, B, 0, 0, v.F32, 4, 64, C, 64, v.F32]
    for at, value, want in [(10, 2, v.ERR_INVALID_TYPE), (5, 3, v.ERR_INVALID_TYPE),
                            (6, -1, v.ERR_INVALID_ARG), (0, 0, v.ERR_INVALID_ARG),
                            (2, 0, v.ERR_INVALID_ARG), (8, 0, v.ERR_INVALID_ARG),
                            (9, 63, v.ERR_INVALID_ARG), (8, A, v.ERR_INVALID_ARG),
                            (3, A + 2, v.ERR_INVALID_ARG), (3, C, v.ERR_INVALID_ARG)]:
        args = list(ok)
        args[at] = value
        assert f(*args) == want, (at, value, v.last_error())


def test_column_ranges_of_the_same_rows_do_not_overlap(v):
    # out in columns 64 .. 127 of rows whose first 64 columns are x: not an overlap (the call then
    # fails for want of a device, or runs), one column nearer: an overlap
    f = v.vcoll_layer_norm
    assert f(A, 128, 0, 0, v.F32, 4, 64, 1e-5, A + 4 * 63, 128, 0, 0, v.F32) == v.ERR_INVALID_ARG
    assert "overlaps" in v.last_error()
    assert f(A, 128, 0, 0, v.F32, 4, 64, 1e-5, A - 4 * 63, 128, 0, 0, v.F32) == v.ERR_INVALID_ARG
    assert f(A, 127, 0, 0, v.F32, 4, 64, 1e-5, A + 4 * 64, 127, 0, 0, v.F32) == v.ERR_INVALID_ARG


@pytest.mark.gpu
def test_data_parallel_example(v):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "data_parallel_step.py")
    spec = importlib.util.spec_from_file_location("data_parallel_step", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, grads = ex.train(steps=60)
    assert all(np.isfinite(losses))
    # it starts at an even guess among the tokens, or a little above, and learns the rule
    assert abs(losses[0] - np.log(ex.VOCAB)) < 0.5 and losses[-1] < 0.5 * losses[0]
    for u in range(1, ex.RANKS):
        for a, b in zip(grads[0], grads[u]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_example_gradients_against_autograd(v):
    # the whole backward pass of one rank beside autograd on the same formulas in 64 bits: what
    # separates them is the 8-bit form, half a step (a block's top / 254) in each normalised value
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "data_parallel_step.py")
    spec = importlib.util.spec_from_file_location("data_parallel_step", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    g = gen(20)
    tokens, targets = ex.batch(g)
    params = [torch.randn(ex.VOCAB, ex.WIDTH, generator=g, device="cuda") * 0.2,
              1 + 0.1 * torch.randn(ex.WIDTH, generator=g, device="cuda"),
              0.1 * torch.randn(ex.WIDTH, generator=g, device="cuda")]
    grads = [torch.empty_like(p) for p in params]
    loss = ex.gradients(params, grads, tokens, targets)
    table, weight, bias = (p.double().requires_grad_() for p in params)
    t = tokens.flatten()
    x = table[t.clamp(min=0)] * (t >= 0)[:, None] * float(np.float32(np.sqrt(ex.WIDTH)))
    mean = x.mean(1, keepdim=True)
    h = (x - mean) / ((x - mean).pow(2).mean(1, keepdim=True) + float(np.float32(1e-5))).sqrt()
    p = torch.log_softmax((h * weight + bias) @ table.t(), 1)
    valid = ((t >= 0) & (targets.flatten() >= 0))
    want = -(p.gather(1, targets.flatten().clamp(min=0)[:, None])[:, 0] * valid).sum() / valid.sum()
    want.backward()
    assert abs(float(loss) - float(want)) < 1e-4 * float(want)
    for a, b in zip(grads, (table.grad, weight.grad, bias.grad)):
        # rounding errors of half a step at most, about a third of that on average and unrelated
        # to one another: 1 / 254 of the top, 4 deviations, is 1.6 % of a typical value
        assert float((a.double() - b).norm() / b.norm()) < 0.016


def _spot(r, t):
    """A copy of a matrix at a random alignment and row stride."""
    n, d = t.shape
    pad, at = int(r.choice([0, 0, 0, 1, 2, 8, 24])), int(r.choice([0, 0, 1, 2, 3, 4, 8]))
    flat = torch.empty(n * (d + pad) + at, dtype=t.dtype, device="cuda")
    return flat[at:].view(n, d + pad)[:, :d].copy_(t)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(60))
def test_random_layer_norms(v, seed):
    r = np.random.default_rng(seed)
    g = gen(seed)
    d = int(round(np.exp(r.uniform(0, np.log(20000)))))
    n = int(min(round(np.exp(r.uniform(0, np.log(20000)))), max(1, 4_000_000 // d)))
    dtype, wtype = TYPES[r.integers(2)], TYPES[r.integers(2)]
    x = _spot(r, matrix(g, n, d, dtype, "dense", 2.0, float(r.choice([0.0, 1.0, -30.0]))))
    grad = _spot(r, matrix(g, n, d, dtype))
    w, b = (t if t is None or r.integers(2) else torch.cat([t[:1], t])[1:]
            for t in weights(g, d, wtype, r.choice(["both", "both", "weight", "bias", "none"])))
    w64 = w.double() if w is not None else torch.ones(d, device="cuda", dtype=torch.float64)
    b64 = b.double() if b is not None else torch.zeros(d, device="cuda", dtype=torch.float64)
    wy, wm, wr, h, bm, br, dh, by = R.norm(x.double(), w64, b64, float(np.float32(1e-5)))
    y, mean, rstd = v.layer_norm(x, w, b, out=_spot(r, x))
    close(mean, wm, bm + R.U * wm.abs(), torch.float32)
    close(rstd, wr, wr * br, torch.float32)
    close(y, wy, by, dtype)
    y, rstd8, k = v.layer_norm_checkpoint8(x, w, b, out=_spot(r, x))
    close(y, wy, by, dtype)
    step = k.scales.double().repeat_interleave(128, 1)[:, :d]
    kept = k.codes[:, :d].double() * step
    assert ((kept - h).abs() <= 0.5 * step * (1 + 300 * R.U) + dh).all()
    assert not k.codes[:, d:].any()
    back = v.checkpoint8_restore(k, w, b, out=_spot(r, x))
    close(back, kept * w64 + b64, 3 * R.U * ((kept * w64).abs() + b64.abs()), dtype)
    wtype = w.dtype if w is not None else torch.float32
    hx = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for kept_form in (False, True):
        want = R.norm_grad(grad.double(), kept if kept_form else hx,
                           (rstd8 if kept_form else rstd).double(), w64)
        if kept_form:
            got = v.layer_norm_backward_checkpoint8(grad, k, rstd8, w, dx=_spot(r, x))
        else:
            got = v.layer_norm_backward(grad, x, mean, rstd, w, dx=_spot(r, x))
        for a, c, e, t in zip(got, want[:3], want[3:], (dtype, wtype, wtype)):
            close(a, c, e, t)
    codes, scales = R.pack8(R.f64(x))
    k = v.checkpoint8(x)
    assert np.array_equal(k.codes[:, :d].cpu().numpy(), codes) and not k.codes[:, d:].any()
    assert np.array_equal(k.scales.cpu().numpy(), scales)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(60))
def test_random_embeddings(v, seed):
    r = np.random.default_rng(1000 + seed)
    g = gen(1000 + seed)
    d = int(round(np.exp(r.uniform(0, np.log(6000)))))
    n = int(min(round(np.exp(r.uniform(0, np.log(60000)))), max(1, 4_000_000 // d)))
    V = int(min(round(np.exp(r.uniform(0, np.log(300000)))), max(1, 6_000_000 // d)))
    dtype, ttype = TYPES[r.integers(2)], TYPES[r.integers(2)]
    tokens = tokens_of(g, n, V, str(r.choice(["any", "skewed", "skewed", "one", "none"])),
                       torch.int32 if r.integers(2) else torch.int64)
    scale = float(r.choice([1.0, 0.37, 45.25]))
    t, s = tokens.long(), float(np.float32(scale))
    inside = (t >= 0) & (t < V)
    table = _spot(r, matrix(g, V, d, dtype))
    out = v.embedding(tokens, table, scale=scale, out=_spot(r, torch.empty(n, d, dtype=dtype, device="cuda")))
    want = table.double()[t.clamp(0, V - 1)] * s * inside[:, None]
    assert torch.equal(out, want.float().to(dtype))
    grad = _spot(r, matrix(g, n, d, dtype))
    grad[~inside] = float("nan")  # rows of padding hold anything
    base = _spot(r, matrix(g, V, d, ttype, "dense", 3.0)) if r.integers(3) else None
    rows, g64 = t[inside], grad[inside].double()
    total = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, rows, g64) * s
    size = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, rows, g64.abs()) * abs(s)
    count = torch.bincount(rows, minlength=V)[:, None].double()
    want = total if base is None else base.double() + total
    bound = (count + 4) * R.U * size + 2 * R.U * want.abs()
    if base is not None and r.integers(2):
        got = v.embedding_backward(grad, tokens, V, scale=scale, base=base, out=base)
    else:
        got = v.embedding_backward(grad, tokens, V, scale=scale, base=base,
                                   out=_spot(r, torch.empty(V, d, dtype=ttype, device="cuda")))
    close(got, want, bound, ttype)


@pytest.mark.gpu
@pytest.mark.parametrize("ttype", TYPES)
@pytest.mark.parametrize("n,V,d,layout", [
    (2300, 400, 4097, "odd"), (2300, 700, 8200, "dense"), (2100, 300, 9001, "dense"),
    (4200, 5000, 2050, "slice"), (2060, 1500, 17000, "dense"), (1500, 900, 6001, "odd"),
])
def test_absent_rows_of_wide_tables(v, ttype, n, V, d, layout):
    """Rows that several warps fill, before, beside and after the sums."""
    g = gen(n + V + d)
    grad = matrix(g, n, d, torch.bfloat16)
    base = matrix(g, V, d, ttype, layout, 3.0)
    tokens = tokens_of(g, n, V, "skewed")
    absent = torch.ones(V, dtype=torch.bool, device="cuda")
    absent[tokens[(tokens >= 0) & (tokens < V)]] = False
    assert absent.any()
    for b in (None, base):
        out = like(torch.full((V, d), float("nan"), dtype=ttype, device="cuda"), layout)
        out.fill_(float("nan"))
        assert v.embedding_backward(grad, tokens, V, base=b, out=out) is out
        assert torch.equal(out[absent], base[absent] if b is not None else torch.zeros_like(base[absent]))
        assert out.isfinite().all()
