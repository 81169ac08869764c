"""Layer operators at the edges of their arguments: scales, values and sizes
far from the usual ones."""
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


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,layout", [(8, "dense"), (33, "odd"), (250, "slice"), (1024, "dense"), (2049, "odd")])
@pytest.mark.parametrize("scale", [-1.5, float("inf"), float("-inf"), float("nan"), 0.0, -0.0])
def test_padding_is_zero_whatever_the_scale(v, dtype, d, layout, scale):
    g = L.gen(d)
    table = L.matrix(g, 40, d, dtype, layout)
    tokens = torch.tensor([3, -1, 39, 40, 0, 2 ** 40, 7], device="cuda")
    out = v.embedding(tokens, table, scale=scale, out=L.like(torch.empty(7, d, dtype=dtype, device="cuda"), layout))
    inside = [0, 2, 4, 6]
    want = (table[tokens[inside]].float() * scale).to(dtype)
    assert torch.equal(torch.nan_to_num(out[inside], 7.0), torch.nan_to_num(want, 7.0))
    bits = out[[1, 3, 5]].contiguous().view(torch.int32 if dtype == torch.float32 else torch.int16)
    assert not bits.any()  # +0


# One value whose last bits a sum of many equal terms drops at every addition: the errors of a
# chain all have the same sign, and grow with its length.  Sums in parts of 64 terms, m terms a
# thread, are off by (64 + m / 64) u, and a few more where threads and warps are joined.
BIASED = float(np.float32(1.0 + 0.99 * 2.0 ** -14))


def test_one_chain_of_biased_terms_would_not_do():
    terms = np.full(2500, BIASED, np.float32)
    chain = np.cumsum(terms, dtype=np.float32)[-1]
    parts = np.add.reduce([np.cumsum(terms[a:a + 64], dtype=np.float32)[-1] for a in range(0, 2500, 64)])
    exact, bound = 2500 * BIASED, (64 + 2500 / 64 + 16) * R.U * 2500 * BIASED
    assert abs(float(chain) - exact) > 2 * bound and abs(float(parts) - exact) <= bound


@pytest.mark.gpu
@pytest.mark.parametrize("n", [20000, 4001])
def test_weight_gradients_of_wide_rows_over_many_rows(v, n):
    d = 16400  # above what a team of warps holds
    grad = torch.full((n, d), BIASED, device="cuda")
    x = torch.ones(n, d, device="cuda")
    x[:, 1::2] = -1.0
    mean, rstd = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    _, dw, db = v.layer_norm_backward(grad, x, mean, rstd, dx=grad)
    bound = (64 + n / 8 / 64 + 16) * R.U * n * BIASED
    assert ((db.double() - n * BIASED).abs() <= bound).all()
    assert ((dw.double() - n * BIASED * x[0].double()).abs() <= bound).all()


@pytest.mark.gpu
def test_statistics_of_rows_of_millions(v):
    n, d = 2, 2 ** 22
    x = torch.full((n, d), BIASED, device="cuda")
    bound = (64 + d / 256 / 64 + 24) * R.U * BIASED
    _, mean, rstd = v.layer_norm(x)
    assert ((mean.double() - BIASED).abs() <= bound).all()
    # the gradient of equal values, with h = 0: what is left is the error of their mean
    dx, _, _ = v.layer_norm_backward(x, torch.zeros_like(x), mean * 0, mean * 0 + 1)
    assert (dx.double().abs() <= bound + 2 * R.U * BIASED).all()
    # and of their squares: x of +-c has the variance c^2
    x[:, 1::2] *= -1.0
    _, _, rstd = v.layer_norm(x, eps=0.0)
    assert ((rstd.double() * BIASED - 1.0).abs() <= 0.5 * (64 + d / 256 / 64 + 24) * R.U + 2.0 ** -22 + 4 * R.U).all()


def test_a_workspace_without_memory_of_its_own_is_refused(v):
    # one byte seen many times, or bytes with gaps between them: its elements times their size say
    # nothing about the memory behind it
    from collective_reduction_virtual_gb300 import layers
    host = -1  # get_device() of a host tensor
    one = torch.empty(1, dtype=torch.uint8)
    for given in (one.expand(4096), torch.empty(64, 64, dtype=torch.uint8)[:, ::2], torch.empty(8, 8).t()):
        with pytest.raises(v.VcollError):
            layers._workspace(given, 1024, host, None)
    given = torch.empty(2048, dtype=torch.uint8)
    assert layers._workspace(given, 1024, host, None)[:2] == (given.data_ptr(), 2048)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,value,eps", [(100, 2.0 ** 120, 1e-5), (249, 2.0 ** 119, 1e-5), (24, -2.0 ** 121, 1e-5),
                                         (300, 2.0 ** 112, 1e-12), (1001, 2.0 ** 112, 1e-12),
                                         (1002, -2.0 ** 112, 1e-12), (2056, 2.0 ** 112, 1e-12),
                                         (9001, 2.0 ** 110, 1e-12), (20001, 2.0 ** 110, 1e-12)])
def test_gradient_of_rows_of_one_large_value(v, dtype, d, value, eps):
    # h is 0 throughout, though mean * rstd is above the largest fp32: what a lane holds past the
    # row's end, (0 - mean) * rstd, may not reach the sums
    g = L.gen(d)
    n = 5
    x = torch.full((n, d), value, device="cuda", dtype=dtype)
    x[3] = torch.randn(d, generator=g, device="cuda").to(dtype)
    grad = L.matrix(g, n, d, dtype)
    y, mean, rstd = v.layer_norm(x, eps=eps)
    rows = [0, 1, 2, 4]
    assert (mean[rows] == value).all() and not y[rows].any() and torch.isfinite(rstd).all()
    dx, dw, db = v.layer_norm_backward(grad, x, mean, rstd)
    h = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    h[3] = (x[3].double() - mean[3].double()) * rstd[3].double()
    want = R.norm_grad(grad.double(), h, rstd.double(), torch.ones(d, dtype=torch.float64, device="cuda"))
    for got, w, b, t in zip((dx, dw, db), want[:3], want[3:], (dtype, torch.float32, torch.float32)):
        assert ((got.double() - w).abs() <= 1.01 * b + R.out_unit(t) * (w.abs() + b)).all()


@pytest.mark.gpu
def test_outputs_are_seen_by_a_dispatch_mode(v):
    from torch.utils._python_dispatch import TorchDispatchMode

    class Allocations(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.shapes = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            if "empty" in func.name():
                self.shapes.append(tuple(out.shape))
            return out

    x = torch.randn(6, 96, device="cuda")
    want = v.layer_norm(x)
    with Allocations() as seen:
        got = v.layer_norm(x)
    assert sorted(seen.shapes) == [(6,), (6,), (6, 96)]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_an_allocator_that_does_something_else_is_not_used(v):
    from collective_reduction_virtual_gb300 import layers

    def refuses(*args):
        raise TypeError("three arguments")

    # on the host, or nothing, or not as asked for
    for new in (refuses, lambda s, t, d: None, lambda s, t, d: torch.empty(s, dtype=d),
                lambda s, t, d: torch.empty(0)):
        assert not layers._sound(new)


@pytest.mark.gpu
def test_the_allocator_is_tried(v):
    from collective_reduction_virtual_gb300 import layers

    def new(shape, strides, dtype, device="cuda"):
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)

    assert layers._sound(new)
    for other in (lambda s, t, d: new(s, (1, 2), d), lambda s, t, d: new(s, t, torch.float32),
                  lambda s, t, d: new((3, 2), (2, 1), d), lambda s, t, d: new(s, t, d, "cpu")):
        assert not layers._sound(other)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,V,d", [(700, 90, 256), (5000, 300, 512), (40000, 9000, 64), (2100, 17, 1000)])
def test_where_buffers_lie_does_not_change_lookups_and_codes(v, dtype, n, V, d):
    g = L.gen(n + d)
    tokens = L.tokens_of(g, n, V, "skewed")
    grad, base, table = L.matrix(g, n, d, dtype), L.matrix(g, V, d, torch.float32), L.matrix(g, V, d, dtype)
    k = v.checkpoint8(grad)
    want = [v.embedding(tokens, table, 1.3), v.embedding_backward(grad, tokens, V, 0.7, base=base), k.codes, k.scales]
    for layout in ("slice", "odd"):
        def moved(t):
            return L.like(t, layout).copy_(t)
        gm, bm = moved(grad), moved(base)
        k = v.checkpoint8(gm)
        got = [v.embedding(tokens, moved(table), 1.3, out=L.like(want[0], layout)),
               v.embedding_backward(gm, tokens, V, 0.7, base=bm, out=bm), k.codes, k.scales]
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [100, 1024, 1001, 9000, 40000])
def test_layer_norms_repeat_their_bits_on_the_same_buffers(v, dtype, d):
    g = L.gen(d)
    x, grad = L.matrix(g, 300, d, dtype, "slice"), L.matrix(g, 300, d, dtype, "odd")
    w, b = L.weights(g, d, dtype)

    def run():
        y, mean, rstd = v.layer_norm(x, w, b)
        y8, rstd8, k = v.layer_norm_checkpoint8(x, w, b)
        return [y, mean, rstd, y8, rstd8, k.codes, k.scales, *v.layer_norm_backward(grad, x, mean, rstd, w),
                *v.layer_norm_backward_checkpoint8(grad, k, rstd8, w), v.checkpoint8_restore(k, w, b)]

    want = run()
    for _ in range(3):
        for a, c in zip(run(), want):
            assert torch.equal(a, c)
