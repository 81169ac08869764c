"""Plain 64-bit definitions of the products with their epilogues (the loss
against a vocabulary, the gated feed-forward block), and bounds on how far a
computation in fp32 sums may be from them.

u = 2^-24.  A sum of K products, each exact, accumulated in fp32 in any order
by adders that round or cut off (off by 2 u of the running sum each), is off by
at most 2 K u times the sum of the products' magnitudes S; some 16 additions
join its pieces.  fp32 operands stand as three parts of 8 bits: with |part 1| <=
2^-8 and |part 2| <= 2^-16 of the value, the products left out are below 4.1 u
of S.  A rounding to bf16 is off by at most 2^-8 of the value.
"""
import math

import torch

U = 2.0 ** -24
BF16 = 2.0 ** -8


def unit(dtype):
    return BF16 if dtype == torch.bfloat16 else U


def product(a, b, K=None):
    """a @ b, and the bound of its fp32 sum"""
    K = a.shape[1] if K is None else K
    return a @ b, (2 * (K + 16) + 4.1) * U * (a.abs() @ b.abs())


def loss(x, table, targets):
    """(loss, lse, and their bounds)"""
    x, table, t = x.double(), table.double(), targets.long().flatten()
    V = table.shape[0]
    z, dz = product(x, table.t())
    n = len(z)
    inside = (t >= 0) & (t < V)
    if not V:
        zero = torch.zeros(n, dtype=torch.float64, device=z.device)
        return zero, zero - math.inf, zero, zero
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    # e^y from the rounded product of y and a constant, 2 ulp of its own
    dexp = 4 * U * (2 + 2 * (z - z.amax(1, keepdim=True)).abs())
    # the largest term's reference is itself off by nothing: it is subtracted exactly once
    dsum = (p * (dz + dexp)).sum(1) + (256 + V / 256 + 64) * U
    dlse = dsum + 4 * U * (lse.abs() + z.amax(1).abs() + math.log(V) + 1)
    at = t.clamp(0, V - 1)[:, None]
    zt, dzt = z.gather(1, at)[:, 0], dz.gather(1, at)[:, 0]
    value = torch.where(inside, lse - zt, 0.0)
    return value, lse, torch.where(inside, dlse + dzt + 2 * U * (lse.abs() + zt.abs()), 0.0), dlse


def loss_grad(gloss, x, table, targets, lse, base, dtype):
    """(dx, dtable, and their bounds before the output's rounding)"""
    x, table, t = x.double(), table.double(), targets.long().flatten()
    V, n = table.shape[0], len(x)
    inside = (t >= 0) & (t < V)
    x = torch.where(inside[:, None], x, 0.0)
    g = torch.where(inside, gloss.double().expand(n), 0.0)
    z, dz = product(x, table.t())
    y = torch.where(inside[:, None], z - lse.double()[:, None], 0.0)
    p = torch.exp(y)
    e, size = p.clone(), p.clone()
    rows = torch.nonzero(inside).flatten()
    e[rows, t[rows]] -= 1.0
    size[rows, t[rows]] += 1.0
    dexp = 4 * U * (2 + 2 * y.abs()) + 2 * U * (z.abs() + lse.double()[:, None].abs().nan_to_num(0.0, 0.0, 0.0))
    de = p * torch.expm1(dz + dexp) + 6 * U * size  # the difference, its weight, the scale taken out and put back
    de = de + (unit(dtype) if dtype == torch.bfloat16 else U) * (e.abs() + de)
    # parts of an fp32 e hold its 24 bits
    e, de = torch.where(inside[:, None], e * g[:, None], 0.0), torch.where(inside[:, None], de * g[:, None].abs(), 0.0)
    dx, bx = product(e, table)
    bx = bx + de @ table.abs() + 4 * U * (e.abs() @ table.abs())
    dt, bt = product(e.t(), x)
    bt = bt + de.t() @ x.abs() + 4 * U * dt.abs()
    if base is not None:
        dt = dt + base.double()
        bt = bt + 2 * U * dt.abs()
    return dx, dt, bx, bt


def act(g, kind):
    """(activation, derivative)"""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if kind == "gelu":
        phi = 0.5 * torch.special.erfc(g * -math.sqrt(0.5))  # 1 + erf loses its bits below 0
        return g * phi, phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * c * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * (1 - s) * 2 * c * (1 + 0.134145 * g * g)


def act_rel(g):
    """Relative bound of a factor act(g) / g or its complement's: an exponential
    or a complementary error function of a rounded argument up to g^2 / 2 or
    0.8 (g + 0.045 g^3) times 2, a few ulp of its own, a sum and a division."""
    return 2.0 ** -20 * (1 + g.abs() + g.abs() ** 3 / 8)


def gated(x, wg, wu, kind):
    """(h, gate, up, and their bounds)"""
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, dg = product(x, wg.t())
    u, du = product(x, wu.t())
    a, _ = act(g, kind)
    h = a * u
    # |act'| <= 1.13 everywhere
    dh = 1.13 * dg * (u.abs() + du) + a.abs() * du + (act_rel(g) + 4 * U) * h.abs()
    return h, g, u, dh * (1 + 2.0 ** -10), dg, du


def gated_grad(dh, x, wg, wu, gate, up, kind, dtype):
    """(dx, dwg, dwu, and their bounds)"""
    dh, x, wg, wu, g, u = (t.double() for t in (dh, x, wg, wu, gate, up))
    a, slope = act(g, kind)
    dg, du = dh * u * slope, dh * a
    # act' = s + g ds: each term bounded by itself
    s = torch.where(g == 0, torch.full_like(g, 0.5), a / torch.where(g == 0, 1.0, g))
    size = s.abs() + (slope - s).abs()
    r = BF16 if dtype == torch.bfloat16 else 0.0
    bg = (dh * u).abs() * size * (act_rel(g) + 8 * U)
    bg = bg + r * (dg.abs() + bg)
    bu = du.abs() * (act_rel(g) + 4 * U)
    bu = bu + r * (du.abs() + bu)
    # one sum over both halves
    dx, bx = product(torch.cat([dg, du], 1), torch.cat([wg, wu]))
    bx = bx + bg @ wg.abs() + bu @ wu.abs()
    dwg, bwg = product(dg.t(), x)
    dwu, bwu = product(du.t(), x)
    return dx, dwg, dwu, bx, bwg + bg.t() @ x.abs(), bwu + bu.t() @ x.abs()
