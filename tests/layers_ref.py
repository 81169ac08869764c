"""Plain 64-bit definitions of the layer operators, and bounds on how far a
32-bit computation may be from them.

u = 2^-24 is half a unit in the last place of fp32, relative.  A sum of m
values in any order is off by at most (m - 1) u times the sum of their
magnitudes to first order; a row of D columns is summed by 32 lanes or more,
so the longest chain of additions there is D / 32 and the few steps that join
the lanes.  A bf16 output adds half its own unit, 2^-9 relative (2^-8 is
allowed, which also covers the second rounding from fp32).
"""
import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -100
BLOCK = 128


def f64(t):
    return t.detach().cpu().double().numpy()


def out_unit(dtype):
    return 2.0 ** -8 if "bfloat16" in str(dtype) else 2.0 ** -23


def chain(D):
    return -(-D // 32) + 16


def lookup_grad(grad, tokens, V, scale, base):
    """(value, bound without the output's rounding)"""
    D = grad.shape[1]
    total, size, count = np.zeros((V, D)), np.zeros((V, D)), np.zeros(V)
    for g, t in zip(grad, tokens):
        if 0 <= t < V:
            total[t] += g
            size[t] += np.abs(g)
            count[t] += 1
    total *= scale
    size *= abs(scale)
    value = total if base is None else base + total
    return value, (count[:, None] + 4) * U * size + 2 * U * np.abs(value)


def norm(x, w, b, eps):
    """(y, mean, rstd, h, and the bounds of mean, rstd relative, h, y); arrays
    or tensors of 64 bits"""
    D = x.shape[1]
    mean = x.mean(1)
    dev = x - mean[:, None]
    var = (dev * dev).mean(1)
    rstd = (var + eps) ** -0.5
    h = dev * rstd[:, None]
    c = chain(D) * U
    dmean = (c + U) * abs(x).mean(1)
    # deviations are taken from the computed mean: dmean enters the variance squared
    dvar = (c + 4 * U) * (var + dmean ** 2) + dmean ** 2
    drel = 0.5 * dvar / (var + eps) + 2.0 ** -22 + 2 * U
    dh = rstd[:, None] * (dmean[:, None] + U * abs(dev)) + abs(h) * (drel[:, None] + 3 * U)
    y = h * w + b
    dy = dh * abs(w) + 3 * U * (abs(h * w) + abs(b))
    return y, mean, rstd, h, dmean, drel, dh, dy


def norm_grad(grad, h, rstd, w):
    """(dx, dw, db, and their bounds) for h off by at most 3 u of itself"""
    N, D = grad.shape
    g = grad * w
    m1, m2 = g.mean(1, keepdims=True), (g * h).mean(1, keepdims=True)
    dx = (g - m1 - h * m2) * rstd[:, None]
    c = (chain(D) + 8) * U
    size = abs(g) + abs(m1) + abs(h * m2)
    bx = rstd[:, None] * (c * (abs(g).mean(1, keepdims=True) +
                               abs(h) * abs(g * h).mean(1, keepdims=True)) + 10 * U * size)
    dw, db = (grad * h).sum(0), grad.sum(0)
    bw = (N + 8) * U * abs(grad * h).sum(0)
    bb = (N + 4) * U * abs(grad).sum(0)
    return dx, dw, db, bx, bw, bb


def pack8(x):
    """(codes, scales) of an fp32 array, by the definition's own fp32 steps"""
    N, D = x.shape
    x = x.astype(np.float32)
    B = -(-D // BLOCK)
    codes, scales = np.zeros((N, D), np.int8), np.zeros((N, B), np.float32)
    f = np.float32
    with np.errstate(all="ignore"):
        for b in range(B):
            part = x[:, b * BLOCK:(b + 1) * BLOCK]
            top = np.abs(part).max(1)
            bad = ~np.isfinite(top)
            zero = top < f(TINY)
            unit = f(127) / np.where(bad | zero, f(1), top)
            q = np.rint(part * unit[:, None])
            q[bad | zero] = 0
            codes[:, b * BLOCK:(b + 1) * BLOCK] = q.astype(np.int8)
            scales[:, b] = np.where(bad, f("nan"), np.where(zero, f(0), top / f(127)))
    return codes, scales


def unpack8(codes, scales):
    D = codes.shape[1]
    return codes.astype(np.float64) * np.repeat(scales.astype(np.float64), BLOCK, 1)[:, :D]
