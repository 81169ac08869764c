"""The products' rarer ways through the tiles, each reached by sizes of its own:
sums that are both cut into splits and added up in chunks, sums longer than a
chunk of bf16 results, backward products in a launch each, one weight's gradient
alone; operands at the ends of their range.  Against the 64-bit definitions and
bounds of products_ref.py."""
import pytest
import torch

import products_ref as R
from test_layers import gen, matrix
from test_products import TYPES, near


@pytest.fixture(scope="module")
def v():
    from collective_reduction_virtual_gb300 import build
    build.build()
    import collective_reduction_virtual_gb300 as vc
    return vc


def splits_room(v, n, D, F, dtype):
    """Bytes of the workspace that the splits' sums of a gated block take."""
    if dtype == torch.bfloat16:
        return v.gated_ff_workspace_bytes(n, D, F, dtype, 1)
    wide = (D + 63) // 64 * 64 * 2 * 3  # a row laid out as three parts
    laid = sum((rows * wide + 255) // 256 * 256 for rows in (n, F, F))
    return v.gated_ff_workspace_bytes(n, D, F, dtype, 0) - laid


# Single CTAs and pairs whose tiles have 256 columns: two warps share a tile's rows,
# and a unit's sum is taken out of the tensor cores in several chunks.
SPLIT = [(torch.float32, 100, 1024, 4096), (torch.float32, 128, 4096, 4096), (torch.float32, 64, 2048, 4096),
         (torch.float32, 512, 4096, 2671), (torch.bfloat16, 700, 100000, 1000)]


def test_these_blocks_are_cut_into_splits(v):
    for dtype, n, D, F in SPLIT:
        rows = min(n, 128 if n <= 128 else 256)
        assert splits_room(v, n, D, F, dtype) >= 2 * rows * 256 * 4, (n, D, F)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,n,D,F", SPLIT)
def test_splits_of_a_gated_block_in_chunks(v, dtype, n, D, F):
    g = gen(n + D)
    x, wg, wu = matrix(g, n, D, dtype), matrix(g, F, D, dtype, scale=0.03), matrix(g, F, D, dtype, scale=0.03)
    if D > 4096:  # of terms of one sign, the bound of a long sum is a small share of it
        x.abs_(), wg.abs_(), wu.abs_()
    out = v.gated_ff(x, wg, wu, activation="silu", keep=True)
    want = R.gated(x, wg, wu, "silu")
    for got, w, b in zip(out, want[:3], want[3:]):
        near(got, w, b, dtype)
    for _ in range(8):
        for got, again in zip(out, v.gated_ff(x, wg, wu, activation="silu", keep=True)):
            assert torch.equal(got, again)
    assert v.device_errors() == 0


# ------------------------------------------------- operands at their range's ends

INF = float("inf")
FAR = [200.0, 1e4, 1e13, 1e20, 3e38]


def same(got, want, rel):
    """got is want to a relative bound, with its infinities and NaN."""
    want = want.double()
    far = want.abs() > torch.finfo(got.dtype).max  # rounds to infinity
    want = torch.where(far, torch.copysign(torch.full_like(want, INF), want), want)
    got = got.double()
    ok = (got == want) | ((got - want).abs() <= rel * want.abs()) | (got.isnan() & want.isnan())
    assert ok.all(), (got[~ok], want[~ok])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("copies", [1, 30])  # a few fp32 rows, and tiles
def test_activations_far_out(v, dtype, act, copies):
    # gate is x's first value (or ten times it, which overflows at the last), up is 2;
    # so far out each activation is its argument or zero, and its slope one or zero
    ends = torch.tensor(FAR + [-e for e in FAR], device="cuda").to(dtype).repeat(copies)
    n = len(ends)
    x = torch.stack([ends, torch.ones_like(ends)], 1)
    wg = torch.tensor([[1.0, 0.0], [10.0, 0.0]] * 40, device="cuda").to(dtype)
    wu = torch.tensor([[0.0, 2.0]] * 80, device="cuda").to(dtype)
    h, gate, up = v.gated_ff(x, wg, wu, act, keep=True)
    # an fp32 value of three parts is put together by fp32 additions that may cut a bit off each
    rel = 2.0 ** -21 if dtype == torch.float32 else 2.0 ** -8
    exact = (ends.double()[:, None] * torch.tensor([1.0, 10.0], device="cuda").double()).repeat(1, 40)
    same(gate, exact, rel)
    same(up, torch.full_like(exact, 2.0), rel)
    same(h, 2.0 * exact.clamp(min=0.0), rel)

    # the slopes of these and of infinite ones: x is one row's one, so that a weight's gradient is a row's
    gate = torch.cat([ends, torch.tensor([INF, -INF, float("nan")], device="cuda").to(dtype)])
    n = len(gate)
    pick = torch.eye(n, device="cuda").to(dtype)
    w = torch.zeros(1, n, device="cuda").to(dtype)
    one = torch.ones(n, 1, device="cuda").to(dtype)
    slope = torch.where(gate.isnan(), gate.double(), (gate > 0).double())
    dg = v.gated_ff_backward(one[:-1], pick[:-1], w, w, gate[:-1, None], one[:-1], act, x_grad=False)[1]
    same(dg[0, :-1], slope[:-1], rel)
    dg, du = v.gated_ff_backward(one[:-3], pick[:-3], w, w, gate[:-3, None], one[:-3], act, x_grad=False)[1:]
    same(du[0, :-3], gate[:-3].double().clamp(min=0.0), rel)
    # one row of them all
    dg, du = v.gated_ff_backward(one.t(), one[:1], one, one, gate[None], one.t(), act, x_grad=False)[1:]
    same(dg[:, 0], slope, rel)
    same(du[:, 0], torch.where(gate.isnan(), gate.double(), gate.double().clamp(min=0.0)), rel)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,V,D", [(7, 1000, 2), (40, 1000, 2), (300, 5000, 8), (3, 40000, 640), (20, 130, 4000)])
def test_loss_of_sure_rows_is_exact(v, dtype, n, V, D):
    # one logit stands 500 above the others: lse is that logit, and the loss of its token zero
    g = gen(n + V)
    x = torch.zeros(n, D, device="cuda", dtype=dtype)
    x[:, 0] = (torch.rand(n, generator=g, device="cuda") * 2000 - 1000).to(dtype)
    x[:, 1] = 1.0
    table = torch.zeros(V, D, device="cuda", dtype=dtype)
    table[:, 0] = 1.0
    sure = V // 3
    table[:, 1] = -500.0
    table[sure, 1] = 0.0
    t = torch.full((n,), sure, device="cuda")
    t[1::2] = V - 1
    loss, lse = v.cross_entropy(x, table, t)
    assert torch.equal(lse, x[:, 0].float())
    assert not loss[::2].any()
    # the other logits: a sum of two terms below 1500, cut off at most twice
    assert ((loss[1::2] - 500.0).abs() <= 4 * 2.0 ** -24 * 1500).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,V,D", [(5, 700, 16), (40, 700, 16), (300, 3000, 64), (6, 40000, 640), (20, 130, 4000)])
def test_infinite_logits(v, dtype, n, V, D):
    # rows 0, 3, ...: one token's logit overflows; rows 1, 4, ...: many do, to both sides; the others are finite
    g = gen(n * V)
    x = (torch.rand(n, D, generator=g, device="cuda") + 0.5).to(dtype)
    table = (torch.randn(V, D, generator=g, device="cuda") * 0.1).to(dtype)
    table[:, :2] = 0.0
    table[V - 2, 0] = 10.0
    table[::7, 1], table[1::7, 1] = 10.0, -10.0
    x[:, :2] = 0.0
    x[::3, 0] = 3e38
    x[1::3, 1] = 3e38
    t = torch.full((n,), 3, device="cuda")  # of a finite logit in every row
    t[-1] = -1
    loss, lse = v.cross_entropy(x, table, t)
    over = torch.arange(n, device="cuda") % 3 < 2
    assert (lse[over] == INF).all()
    want, wlse, bound, blse = R.loss(x[~over], table, t[~over])
    near(loss[~over], want, bound)
    near(lse[~over], wlse, blse)
    assert loss[-1] == 0
    over[-1] = False
    assert (loss[over] == INF).all()
    # the token whose own logit is infinite has no loss: inf - inf
    t[0] = V - 2
    assert v.cross_entropy(x, table, t)[0][0].isnan()


@pytest.mark.gpu
def test_infinite_bf16_operands(v):
    g = gen(31)
    for n, V in ((5, 700), (200, 3000)):
        x = torch.randn(n, 64, generator=g, device="cuda").bfloat16()
        table = torch.randn(V, 64, generator=g, device="cuda").bfloat16()
        table[:, 0] = table[:, 0].abs() + 1.0
        x[0, 0], x[1, 0], x[2, 0] = INF, -INF, float("nan")
        t = torch.full((n,), 1, device="cuda")
        lse = v.cross_entropy(x, table, t)[1]
        assert lse[0] == INF and lse[1] == -INF and lse[2].isnan() and lse[3:].isfinite().all()


# --------------------------------------------------------- long and separate sums

@pytest.mark.gpu
def test_gated_sums_longer_than_a_chunk(v):
    # bf16 sums of more than 32768 places leave the tensor cores in two pieces, and no tile is split
    dtype, n, D, F = torch.bfloat16, 513, 33000, 4864
    assert splits_room(v, n, D, F, dtype) == 0
    g = gen(21)
    x, wg, wu = (matrix(g, r, D, dtype, scale=s).abs_() for r, s in ((n, 1.0), (F, 1e-3), (F, 1e-3)))
    wg[1::2] *= -1  # gates of both signs, each a sum of one sign
    want = R.gated(x, wg, wu, "gelu_tanh")
    for got, w, b in zip(v.gated_ff(x, wg, wu, "gelu_tanh", keep=True), want[:3], want[3:]):
        near(got, w, b, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_gated_gradients_in_a_launch_each(v, dtype):
    # both sums of 8192 places and more, and a wave of tiles in each product
    n, D, F = 8200, 616, 4200
    g = gen(22)
    x, wg, wu = matrix(g, n, D, dtype), matrix(g, F, D, dtype, scale=0.05), matrix(g, F, D, dtype, scale=0.05)
    dh, gate, up = (matrix(g, n, F, dtype) for _ in range(3))
    want = R.gated_grad(dh, x, wg, wu, gate, up, "silu", dtype)
    got = v.gated_ff_backward(dh, x, wg, wu, gate, up, "silu")
    for t, w, b in zip(got, want[:3], want[3:]):
        near(t, w, b, dtype)
    for t, again in zip(got, v.gated_ff_backward(dh, x, wg, wu, gate, up, "silu")):
        assert torch.equal(t, again)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("with_base", [False, True])
def test_loss_gradients_in_a_launch_each(v, dtype, with_base):
    n, V, D = 8200, 8300, 616
    g = gen(23)
    x, table = matrix(g, n, D, dtype), matrix(g, V, D, dtype, scale=0.08)
    t = torch.randint(-200, V, (n,), generator=g, device="cuda")
    base = matrix(g, V, D, dtype) if with_base else None
    gloss = torch.randn(n, generator=g, device="cuda")
    lse = v.cross_entropy(x, table, t)[1]
    dx, dt = v.cross_entropy_backward(gloss, x, table, t, lse, base=base)
    want = R.loss_grad(gloss, x, table, t, lse, base, dtype)
    near(dx, want[0], want[2], dtype)
    near(dt, want[1], want[3], dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,D,F,layout", [(1, 64, 100, "dense"), (9, 129, 67, "odd"), (16, 320, 1030, "slice"),
                                          (17, 33, 5, "odd"), (300, 200, 500, "dense"), (700, 1001, 259, "odd")])
@pytest.mark.parametrize("which", ["gate", "up"])
@pytest.mark.parametrize("x_grad", [False, True])
def test_one_weights_gradient_alone(v, dtype, n, D, F, layout, which, x_grad):
    g = gen(n + D + F)
    x, wg, wu = (matrix(g, r, D, dtype, layout) for r in (n, F, F))
    dh, gate, up = (matrix(g, n, F, dtype, layout) for _ in range(3))
    out = matrix(g, F, D, dtype, layout).fill_(float("nan"))
    got = v.gated_ff_backward(dh, x, wg, wu, gate, up, "gelu", x_grad=x_grad, weight_grads=False, **{"dw_" + which: out})
    want = R.gated_grad(dh, x, wg, wu, gate, up, "gelu", dtype)
    at = 1 if which == "gate" else 2
    assert got[at] is out and got[3 - at] is None and (got[0] is not None) == x_grad
    near(out, want[at], want[3 + at], dtype)
    if x_grad:
        near(got[0], want[0], want[3], dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,n,V,D", [(torch.float32, 40000, 5001, 24), (torch.bfloat16, 70001, 5001, 16)])
def test_table_gradient_of_tokens_that_no_row_aims_at(v, dtype, n, V, D):
    # A vocabulary in pieces.  With rows, weights and e of one sign a sum's bound is a small share of it.
    # The sum over all rows is off by 2 n u of its terms, beside what products_ref has for each part of them.
    g = gen(24)
    x, table = matrix(g, n, D, dtype).abs_(), matrix(g, V, D, dtype, scale=0.5)
    t = torch.randint(-50, V // 2, (n,), generator=g, device="cuda")
    gloss = torch.rand(n, generator=g, device="cuda") + 0.5
    lse = v.cross_entropy(x, table, t)[1]
    dt = v.cross_entropy_backward(gloss, x, table, t, lse, x_grad=False)[1]
    total = bound = 0.0
    for a in range(0, n, 8192):
        part = slice(a, a + 8192)
        w = R.loss_grad(gloss[part], x[part], table, t[part], lse[part], None, dtype)
        total, bound = total + w[1], bound + w[3]
    free = slice(V // 2, V)
    bound = bound[free] + 2 * n * R.U * total[free]
    assert (bound <= 0.02 * total[free]).all()
    near(dt[free], total[free], bound, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_products_repeat_their_bits(v, dtype):
    g = gen(25)
    for n, D, F in ((5, 700, 900), (40, 1024, 3000), (300, 2048, 1000), (1000, 320, 1280)):
        x, w, u = (matrix(g, r, D, dtype) for r in (n, F, F))
        t = torch.randint(-3, F, (n,), generator=g, device="cuda")
        one = torch.ones(1, device="cuda")

        def calls():
            loss, lse = v.cross_entropy(x, w, t)
            h, gate, up = v.gated_ff(x, w, u, keep=True)
            return (loss, lse, *v.cross_entropy_backward(one, x, w, t, lse, base=u), h, gate, up,
                    *v.gated_ff_backward(h, x, w, u, gate, up))

        first = calls()
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(first, calls()))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,D,F", [(1, 8, 3), (7, 130, 1000), (16, 513, 77), (100, 1024, 4096), (513, 320, 1280), (33, 1001, 2671)])
def test_workspaces_are_not_left(v, dtype, n, D, F):
    # each call has exactly the bytes that it asks for, between others that it leaves alone
    g = gen(n + D + F + 2)
    x, w, u = (matrix(g, r, D, dtype) for r in (n, F, F))
    dh = matrix(g, n, F, dtype)
    t = torch.randint(-1, F, (n,), generator=g, device="cuda")
    one = torch.ones(1, device="cuda")
    def inside(need, call):
        room = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        out = call(room[4096:4096 + need])
        assert (room[:4096] == 0xA5).all() and (room[4096 + need:] == 0xA5).all()
        return out

    loss, lse = inside(v.cross_entropy_workspace_bytes(n, F, D, dtype), lambda ws: v.cross_entropy(x, w, t, workspace=ws))
    grads = inside(v.cross_entropy_backward_workspace_bytes(n, F, D, dtype),
                   lambda ws: v.cross_entropy_backward(one, x, w, t, lse, base=u, workspace=ws))
    h, gate, up = inside(v.gated_ff_workspace_bytes(n, D, F, dtype), lambda ws: v.gated_ff(x, w, u, keep=True, workspace=ws))
    more = inside(v.gated_ff_backward_workspace_bytes(n, D, F, dtype),
                  lambda ws: v.gated_ff_backward(dh, x, w, u, gate, up, workspace=ws))
    for got, again in zip((loss, lse, *grads, h, gate, up, *more),
                          (*v.cross_entropy(x, w, t), *v.cross_entropy_backward(one, x, w, t, lse, base=u),
                           *v.gated_ff(x, w, u, keep=True), *v.gated_ff_backward(dh, x, w, u, gate, up))):
        assert torch.equal(got, again)


# ----------------------------------------------------- many rows, block by block

def test_the_loss_gradients_workspace_is_bounded(v):
    # 1 GB of e at most (256 MB where that has 2048 columns) beside what has the rows' own size: x laid out
    # and dx's sums so far
    for n, V, D, dtype, e in ((65536, 128000, 64, torch.bfloat16, 1 << 28), (21000, 128000, 64, torch.float32, 1 << 28),
                              (1 << 19, 128000, 64, torch.float32, 1 << 30), (1 << 20, 128000, 64, torch.float32, 1 << 30),
                              (1 << 20, 50000, 1, torch.bfloat16, 1 << 30)):
        parts = 3 if dtype == torch.float32 else 1
        wide = (D + 63) // 64 * 64
        rows = n * (wide * 2 * parts + (D + 1) // 2 * 2 * 4)
        table = 2 * V * wide * 2 * parts  # a piece laid out and its gradient's sums, and splits of these
        assert v.cross_entropy_backward_workspace_bytes(n, V, D, dtype) <= e + rows + table + (64 << 20), (n, V, D)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,n,V,D,index", [
    (torch.bfloat16, 270000, 2100, 40, torch.int32), (torch.bfloat16, 530001, 2049, 7, torch.int64),
    (torch.float32, 88000, 4100, 33, torch.int64), (torch.float32, 174081, 2500, 16, torch.int32),
    (torch.bfloat16, 524289, 2500, 8, torch.int64)])
@pytest.mark.parametrize("form", ["dense", "odd", "one"])
def test_a_loss_gradient_in_blocks_of_rows(v, dtype, n, V, D, index, form):
    g = gen(n + V)
    layout = "odd" if form == "odd" else "dense"
    x, table = matrix(g, n, D, dtype, layout).abs_(), matrix(g, V, D, dtype, layout, scale=0.5)
    t = torch.randint(-500, V // 2, (n,), generator=g, device="cuda").to(index)
    t[-1], t[n // 2] = V // 2, -1
    gloss = torch.rand(1 if form == "one" else n, generator=g, device="cuda") + 0.5
    base = matrix(g, V, D, dtype, layout)
    lse = v.cross_entropy(x, table, t)[1]
    plain = v.cross_entropy_backward(gloss, x, table, t, lse)
    kept = base.clone()
    dx, dt = v.cross_entropy_backward(gloss, x.clone(), table, t, lse, base=base, dtable=base)
    assert dt is base and torch.equal(dx, plain[0])
    total = bound = 0.0
    wants = []
    for a in range(0, n, 8192):
        part = slice(a, a + 8192)
        w = R.loss_grad(gloss[part] if form != "one" else gloss, x[part], table, t[part], lse[part], None, dtype)
        wants.append((part, w[0], w[2]))
        near(dx[part], w[0], w[2], dtype)
        total, bound = total + w[1], bound + w[3]
    # The sum over all rows is off by 2 n u of its terms' magnitudes, beside what each part's is.  These are
    # g p x, which the total has, and g x of the rows that aim at the token, which it has the other way round.
    inside = (t >= 0).nonzero().flatten()
    aimed = torch.zeros_like(total).index_add_(0, t[inside].long(), x[inside].double() * gloss.expand(n)[inside, None])
    bound = bound + 2 * n * R.U * (total + 2 * aimed)
    near(plain[1], total, bound, dtype)
    added = bound + 8 * R.U * (total.abs() + 2 * aimed + kept.double().abs())
    near(dt, total + kept.double(), added, dtype)
    # each gradient alone
    near(v.cross_entropy_backward(gloss, x, table, t, lse, base=kept, x_grad=False)[1], total + kept.double(), added, dtype)
    dx = v.cross_entropy_backward(gloss, x, table, t, lse, dx=x, table_grad=False)[0]
    assert dx is x
    for part, w, b in wants:
        near(dx[part], w, b, dtype)


# ------------------------------------------------------------------- precision

@pytest.mark.gpu
@pytest.mark.parametrize("n,D,F", [(300, 512, 400), (700, 448, 1000), (300, 1500, 400), (40, 1500, 2000)])
def test_fp32_sums_are_as_close_as_fp32_adders(v, n, D, F):
    # against adders that round to nearest after each of the terms in turn
    g = gen(26)
    x, wg, wu = matrix(g, n, D, torch.float32), matrix(g, F, D, torch.float32), matrix(g, F, D, torch.float32)
    _, gate, up = v.gated_ff(x, wg, wu, keep=True)
    for got, w in ((gate, wg), (up, wu)):
        exact = x.double() @ w.double().t()
        adders = torch.zeros_like(got)
        for k in range(D):
            adders += x[:, k, None] * w[None, :, k]
        assert (got.double() - exact).norm() <= (adders.double() - exact).norm()
