"""The gated feed-forward block and the log probabilities from hidden rows in
64 bits, straight from their formulas, with the error bounds of kernels that
multiply on the matrix cores and hold sums and statistics in f32.

As in token_reference: float64 / int64 arrays in, (outputs, bounds) out.

A product's sum over k of a b: the matrix cores add 32 products at a time to an
f32 sum, so a term meets at most 32 additions inside of an instruction and
k / 32 outside, each off by at most 2 U of what it adds (U for rounding, 2 U
where it truncates); parts of k add a few more. f32 operands are three bf16
numbers: x1 <= 2^-8 x, x2 <= 2^-16 x, and 2^-24 x is left; of the nine products
the three of x1 y2, x2 y1, x2 y2 are not there (2 * 2^-24 + 2^-32 of x y), the
rests cost 2 * 2^-24: 4 U with the small terms, and the six others lengthen the
chain.
"""
import numpy as np

from tests.token_reference import HALF, TINY, U, f32_range, rounded

erf = np.vectorize(__import__("math").erf, otypes=[float])


def product_bound(k, size, dtype):
    """Bound of the sum of k products whose sizes add up to `size`."""
    if dtype == "f32":
        return (4.0 + 2.05 * (6.0 * k / 32 + 48)) * U * size + 2.0 ** -126
    return 2.0 * (k / 32.0 + 48) * U * size


def held(y, dtype):
    """What holding y between two products costs (f32: within product_bound)."""
    return 0.0 * y if dtype == "f32" else HALF[dtype] * np.abs(y) + TINY[dtype]


def act(g, name):
    """act(g), act'(g) and the bounds of their evaluation."""
    if name == "relu":
        return np.maximum(g, 0.0), (g > 0).astype(float), 0.0 * g, 0.0 * g
    far = np.abs(g)
    if name == "silu":
        s = np.where(g >= 0, 1.0, np.exp(-far)) / (1.0 + np.exp(-far))
        e = (3.0 * far + 8.0) * U * np.minimum(s, 1.0) + 2.0 ** -126
        return g * s, s + g * s * (1 - s), far * e, (1 + far) * e * 2 + 4 * U
    # gelu: the integral to 0.75e-7 by its formula, and a few roundings
    p = 0.5 * (1.0 + erf(g * np.sqrt(0.5)))
    w = np.exp(-0.5 * g * g) / np.sqrt(2 * np.pi)
    e = 0.76e-7 + 10 * U + 2 * U * g * g * np.exp(-0.5 * g * g)
    return g * p, p + g * w, far * e, e + far * w * (g * g + 8) * U + 4 * U


STEEP = 1.13  # the largest slope of the three


def ffn(x, w_in, w_out, name, dtype):
    f = w_out.shape[1]
    pre = x @ w_in.T
    e_pre = product_bound(x.shape[1], np.abs(x) @ np.abs(w_in).T, dtype)
    g, u, eg, eu = pre[:, :f], pre[:, f:], e_pre[:, :f], e_pre[:, f:]
    a, _, ea, _ = act(g, name)
    h = a * u
    # the error of g moves act by at most its slope
    e_a = ea + STEEP * eg
    e_h = e_a * (np.abs(u) + eu) + np.abs(a) * eu + 2 * U * np.abs(h)
    e_h = e_h + held(np.abs(h) + e_h, dtype)
    y = h @ w_out.T
    e_y = (e_h @ np.abs(w_out).T
           + product_bound(f, (np.abs(h) + e_h) @ np.abs(w_out).T, dtype))
    return (y, pre), (rounded(y, e_y, dtype), rounded(pre, e_pre, dtype))


def ffn_grad(d_out, x, pre, w_in, w_out, name, dtype):
    """With the rounded pre that the call is given."""
    n, f = x.shape[0], w_out.shape[1]
    g, u = pre[:, :f], pre[:, f:]
    a, da, ea, eda = act(g, name)
    dh = d_out @ w_out
    e_dh = product_bound(w_out.shape[0], np.abs(d_out) @ np.abs(w_out), dtype)
    h = a * u
    e_h = ea * np.abs(u) + 2 * U * np.abs(h)
    e_h = e_h + held(np.abs(h) + e_h, dtype)
    dg, du = dh * u * da, dh * a
    big = np.abs(dh) + e_dh
    e_dg = e_dh * np.abs(u * da) + big * np.abs(u) * eda + 4 * U * np.abs(dg)
    e_du = e_dh * np.abs(a) + big * ea + 4 * U * np.abs(du)
    d_pre, e = np.hstack([dg, du]), np.hstack([e_dg, e_du])
    e = e + held(np.abs(d_pre) + e, dtype)
    s = np.abs(d_pre) + e
    d_x = d_pre @ w_in
    e_x = e @ np.abs(w_in) + product_bound(2 * f, s @ np.abs(w_in), dtype)
    d_in = d_pre.T @ x
    e_in = e.T @ np.abs(x) + product_bound(n, s.T @ np.abs(x), dtype)
    d_w = d_out.T @ h
    e_w = np.abs(d_out).T @ e_h + product_bound(n, np.abs(d_out).T @ (np.abs(h) + e_h), dtype)
    return ((d_x, d_in, d_w),
            (rounded(d_x, e_x, dtype), rounded(d_in, e_in, dtype), rounded(d_w, e_w, dtype)))


def _logits(x, table, bias, dtype):
    z = x @ table.T
    e = product_bound(x.shape[1], np.abs(x) @ np.abs(table).T, dtype)
    if bias is not None:
        shut = bias == -np.inf
        b = np.where(shut, 0.0, bias)
        z = z + b
        e = e + U * (np.abs(z) + e)
        z[:, shut] = -np.inf
        e[:, shut] = 0.0
    return z, e


def loss(x, table, bias, targets, dtype):
    """Outputs (logp, entropy, stats) and bounds."""
    z, e = _logits(x, table, bias, dtype)
    n, v = z.shape
    m = z.max(axis=1)
    empty = m == -np.inf
    base = np.where(empty, 0.0, m)[:, None]
    with np.errstate(invalid="ignore"):
        t = z - base
        q = np.exp(t)
        s = np.where(empty, 1.0, q.sum(axis=1))
        ls = np.log(s)
        p = q / s[:, None]
        tp = np.where(p > 0, np.abs(t) * p, 0.0).sum(axis=1)
        ttp = np.where(p > 0, t * t * p, 0.0).sum(axis=1)
        lp = np.where(p > 0, t - ls[:, None], 0.0)
    H = np.where(empty, 0.0, ls + tp)
    e_m = e.max(axis=1, initial=0.0)  # the largest computed z is not above the largest + e
    mean_e = (p * e).sum(axis=1)
    L = 64 + v / 1024.0
    # (as logprobs' bounds: a term's exponential and its rescaling, the chain)
    e_s = U * (2 * (3 * tp + 2) + 4 * L)
    e_ls = e_s + 2 * U * np.abs(ls) + U + mean_e + e_m
    e_u = U * (6 * ttp + (7 + 4 * L) * tp)
    turn = np.where(p > 0, p * np.abs(lp + H[:, None]), 0.0)
    far = np.where(np.isfinite(z), e, 0.0)
    e_H = (e_s + e_u + tp * e_s + 4 * U * (np.abs(ls) + tp)
           + 1.1 * (turn * far).sum(axis=1) + (p * (1 + np.abs(lp)) * far * far).sum(axis=1))
    ok = (targets >= 0) & (targets < v)
    at = np.where(ok, targets, 0)
    with np.errstate(invalid="ignore"):
        zt = t[np.arange(n), at]
        logp = np.where(ok, np.where(empty, -np.inf, zt - ls), 0.0)
        size = np.where(np.isfinite(zt), np.abs(zt), 0.0)
    e_logp = e[np.arange(n), at] + e_ls + e_m + 2 * U * (size + np.abs(ls) + np.abs(base[:, 0]))
    stats = np.stack([m, np.where(empty, 0.0, ls)], axis=1)
    e_stats = np.stack([e_m, e_ls], axis=1)
    return ((f32_range(logp), H, stats),
            (1.05 * e_logp, 1.05 * e_H, 1.05 * e_stats))


def loss_grad(x, table, bias, targets, stats, entropy, d_logp, d_entropy, dtype):
    """With the f32 stats and entropies that the call is given. Outputs (d_x,
    d_table, d_bias)."""
    z, e = _logits(x, table, bias, dtype)
    n, v = z.shape
    m, ls = stats[:, :1], stats[:, 1:]
    empty = m == -np.inf
    shut = (z == -np.inf) | empty
    zz = np.where(shut, 0.0, z)
    lp = zz - np.where(empty, 0.0, m) - ls
    p = np.where(shut, 0.0, np.exp(lp))
    ok = (targets >= 0) & (targets < v)
    g = np.where(ok, d_logp, 0.0)[:, None]
    h, H = d_entropy[:, None], entropy[:, None]
    hit = np.zeros((n, v))
    hit[np.nonzero(ok)[0], targets[ok]] = 1.0
    hit[shut] = 0.0
    fac = g + h * (lp + H)
    dz = np.where(shut, 0.0, g * hit - p * fac)
    e_lp = e + U * (np.abs(zz - m) * 2 + np.abs(ls) + np.abs(zz) + np.abs(lp)) if not empty.any() else \
        e + U * (4 * np.abs(zz) + 4 * np.abs(np.where(empty, 0.0, m)) + 4 * np.abs(ls))
    # p is between exp(lp - e_lp) and the mirror image's height above it; where that is 0 in 64
    # bits (lp < -745) it is 0 in f32 too, with no error for the factor to enlarge
    top = np.where(shut, 0.0, np.exp(lp + e_lp))
    e_p = np.where(top > 0, (top - p) + top * (3 * np.abs(lp) + 4) * U + 2.0 ** -126, 0.0)
    e_fac = np.abs(h) * e_lp + 4 * U * (np.abs(g) + np.abs(h) * (np.abs(lp) + np.abs(H)))
    e_dz = np.where(shut, 0.0, e_p * (np.abs(fac) + e_fac) + p * e_fac
                    + 3 * U * (np.abs(g * hit) + np.abs(p * fac)))
    d_bias = dz.sum(axis=0)
    e_b = e_dz.sum(axis=0) + (n + 4.0) * U * (np.abs(dz) + e_dz).sum(axis=0)
    if dtype == "f16":  # held times a power of two: its bound is within 2^15 and 2^13
        most = (np.abs(d_logp) + 17 * np.abs(d_entropy)).max(initial=0.0)
        e_dz = e_dz + HALF[dtype] * (np.abs(dz) + e_dz) + 2.0 ** -25 * most * 2.0 ** -13
    else:
        e_dz = e_dz + held(np.abs(dz) + e_dz, dtype)
    s = np.abs(dz) + e_dz
    d_x, d_t = dz @ table, dz.T @ x
    # (the pieces' sums of d_x: one more addition each)
    e_x = e_dz @ np.abs(table) + product_bound(v, s @ np.abs(table), dtype)
    e_t = e_dz.T @ np.abs(x) + product_bound(n, s.T @ np.abs(x), dtype)
    return ((d_x, d_t, d_bias),
            (rounded(d_x, 1.02 * e_x, dtype), rounded(d_t, 1.02 * e_t, dtype),
             rounded(d_bias, 1.02 * e_b, "f32")))
