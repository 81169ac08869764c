"""The layer operators' results where a NaN counts as wrong, and written over
outputs that hold nothing but NaN beforehand, so that an element that a kernel
leaves out, or a value that leaks in from padding, shows."""
import numpy as np
import pytest
import torch

import layers_ref as R
import test_layers as L

TYPES = L.TYPES


@pytest.fixture(scope="module")
def v():
    from collective_reduction_virtual_gb300 import build
    build.build()
    import collective_reduction_virtual_gb300 as vc
    return vc


def close(got, want, bound, dtype):
    """got is within the bound of want everywhere, and a number."""
    tol = bound * 1.01 + R.out_unit(dtype) * (want.abs() + bound)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


def test_close_takes_no_nan():
    want, bound = torch.ones(3, dtype=torch.float64), torch.full((3,), 1e-6, dtype=torch.float64)
    close(torch.ones(3), want, bound, torch.float32)
    for wrong in (float("nan"), float("inf"), 1.1):
        with pytest.raises(AssertionError):
            close(torch.tensor([1.0, wrong, 1.0]), want, bound, torch.float32)


# The random and the many-row tests once more, by this comparison.

@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(60))
def test_random_layer_norms(v, seed, monkeypatch):
    monkeypatch.setattr(L, "close", close)
    L.test_random_layer_norms(v, seed)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(60))
def test_random_embeddings(v, seed, monkeypatch):
    monkeypatch.setattr(L, "close", close)
    L.test_random_embeddings(v, seed)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d", [(20011, 16), (20000, 40), (30001, 64), (3000, 200), (5000, 128), (5000, 256),
                                 (5000, 512), (3000, 1024), (2500, 1536), (1500, 4096), (700, 8192), (700, 12288),
                                 (700, 16384), (100, 32768)])
@pytest.mark.parametrize("at", [0, 2, 1])
def test_every_width_and_alignment_over_many_rows(v, dtype, n, d, at, monkeypatch):
    monkeypatch.setattr(L, "close", close)
    L.test_layer_norm_every_width_and_alignment_over_many_rows(v, dtype, n, d, at)


# ------------------------------------------------------- outputs full of NaN

def blank(n, d, dtype, layout):
    """An output of n x d NaN, with NaN around it."""
    pad, at = {"dense": (0, 0), "slice": (24, 8), "odd": (3, 1)}[layout]
    flat = torch.full((n * (d + pad) + at,), float("nan"), dtype=dtype, device="cuda")
    return flat, flat[at:].view(n, d + pad)[:, :d]


def untouched_around(flat, out):
    """What lies around the output is as it was."""
    n = int(torch.isnan(flat).sum()) if flat.numel() else 0
    return n == flat.numel() - out.numel()


def poison(*shapes):
    """Leaves NaN in the memory that the next allocations of these sizes get."""
    held = [torch.full(s, float("nan"), device="cuda") for s in shapes]
    del held


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d,layout", [
    (1, 1, "odd"), (33, 7, "slice"), (1001, 40, "odd"), (257, 100, "slice"), (999, 129, "dense"), (77, 250, "odd"),
    (513, 258, "slice"), (1300, 1001, "dense"), (40, 2050, "odd"), (640, 4098, "dense"), (9, 9002, "slice"),
    (700, 12290, "dense"), (3, 20001, "odd"), (2, 40000, "dense"),
])
def test_layer_norms_over_nan(v, dtype, n, d, layout):
    g = L.gen(n * 11 + d)
    x, grad = (L.matrix(g, n, d, dtype, layout, 2.0, 0.5) for _ in range(2))
    w, b = L.weights(g, d, TYPES[(n + d) % 2])
    w64, b64 = w.double(), b.double()
    wy, wm, wr, h, bm, br, dh, by = R.norm(x.double(), w64, b64, float(np.float32(1e-5)))
    poison((n,), (n,))
    flat, out = blank(n, d, dtype, layout)
    y, mean, rstd = v.layer_norm(x, w, b, out=out)
    close(mean, wm, bm + R.U * wm.abs(), torch.float32)
    close(rstd, wr, wr * br, torch.float32)
    close(y, wy, by, dtype)
    assert untouched_around(flat, out)
    flat, out = blank(n, d, dtype, layout)
    poison((n,), (n, -(-d // 128)))
    y8, rstd8, k = v.layer_norm_checkpoint8(x, w, b, out=out)
    close(y8, wy, by, dtype)
    close(rstd8, wr, wr * br, torch.float32)
    assert untouched_around(flat, out) and not k.codes[:, d:].any() and torch.isfinite(k.scales).all()
    kept = k.codes[:, :d].double() * k.scales.double().repeat_interleave(128, 1)[:, :d]
    flat, out = blank(n, d, dtype, layout)
    close(v.checkpoint8_restore(k, w, b, out=out), kept * w64 + b64,
          3 * R.U * ((kept * w64).abs() + b64.abs()), dtype)
    assert untouched_around(flat, out)
    hx = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for form in (False, True):
        want = R.norm_grad(grad.double(), kept if form else hx, (rstd8 if form else rstd).double(), w64)
        flat, out = blank(n, d, dtype, layout)
        wflat = torch.full((2 * d + 1,), float("nan"), dtype=w.dtype, device="cuda")
        outs = dict(dx=out, dweight=wflat[1:d + 1], dbias=wflat[d + 1:])
        need = v.layer_norm_workspace_bytes(n, d)
        ws = torch.full((max(1, -(-need // 4)),), float("nan"), device="cuda")
        if form:
            got = v.layer_norm_backward_checkpoint8(grad, k, rstd8, w, workspace=ws, **outs)
        else:
            got = v.layer_norm_backward(grad, x, mean, rstd, w, workspace=ws, **outs)
        for a, c, e, t in zip(got, want[:3], want[3:], (dtype, w.dtype, w.dtype)):
            close(a, c, e, t)
        assert untouched_around(flat, out) and torch.isnan(wflat[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ttype", [(a, b) for a in TYPES for b in TYPES])
@pytest.mark.parametrize("n,V,d,kind,layout", [
    (1, 3, 5, "any", "odd"), (700, 90, 77, "skewed", "slice"), (1500, 4000, 130, "skewed", "odd"),
    (2050, 700, 514, "skewed", "dense"), (3001, 65, 1001, "any", "slice"), (5000, 9000, 258, "one", "odd"),
    (9001, 3000, 100, "none", "dense"), (40000, 20001, 66, "skewed", "slice"),
])
def test_embeddings_over_nan(v, dtype, ttype, n, V, d, kind, layout):
    g = L.gen(n + V + d)
    tokens = L.tokens_of(g, n, V, kind)
    inside = (tokens >= 0) & (tokens < V)
    table = L.matrix(g, V, d, dtype, layout)
    flat, out = blank(n, d, dtype, layout)
    v.embedding(tokens, table, scale=1.7, out=out)
    want = table.double()[tokens.clamp(0, V - 1)] * float(np.float32(1.7)) * inside[:, None]
    assert torch.equal(out, want.float().to(dtype)) and untouched_around(flat, out)
    grad = L.matrix(g, n, d, dtype, layout)
    grad[~inside] = float("nan")  # rows of padding hold anything
    base = L.matrix(g, V, d, ttype, layout, 3.0)
    rows, g64 = tokens[inside], grad[inside].double()
    total = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, rows, g64)
    size = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, rows, g64.abs())
    count = torch.bincount(rows, minlength=V)[:, None].double()
    need = v.embedding_workspace_bytes(n, V, d)
    ws = torch.full((max(1, -(-need // 4)),), float("nan"), device="cuda")
    for from_base in (False, True):
        want = base.double() + total if from_base else total
        flat, out = blank(V, d, ttype, layout)
        v.embedding_backward(grad, tokens, V, base=base if from_base else None, out=out, workspace=ws)
        close(out, want, (count + 4) * R.U * size + 2 * R.U * want.abs(), ttype)
        assert untouched_around(flat, out)
