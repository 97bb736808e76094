"""The token operators in 64 bits, straight from their formulas, with the
error bound of a kernel that holds sums and statistics in f32.

Every function takes float64 / int64 numpy arrays that hold the operands'
exact values and returns (outputs, bounds). U is f32's largest relative
rounding error; ``half(t)`` the half step of an output type. Bounds count,
for every f32 operation on the way to an output, U times the size of its
result; a sum of c terms held in parts costs at most (its longest chain) U
times the sum of the terms' sizes. A row's chain is taken for its length / 64
+ 16: a wave's lane adds 1/64 of the row, rounded up to its vectors, and some
levels join the lanes. That is not the longest chain of every spread of a row.
The norms' is up to 37 for halves of 1025 to 2048 elements (32 per lane, 6
levels), 5 more than said at 1025; log probabilities of short rows, 8 to 32
lanes of up to 32 elements, have up to 37 where chain() says 18, and their
bounds count four chains.
"""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half a subnormal step


def rounded(y, bound, dtype):
    """The bound with the output's own rounding."""
    return bound + HALF[dtype] * (np.abs(y) + bound) + TINY[dtype]


def chain(length):
    return length / 64.0 + 16.0


def embed(table, tokens, scale, dtype):
    ok = (tokens >= 0) & (tokens < table.shape[0])
    y = np.where(ok[:, None], table[np.where(ok, tokens, 0)] * scale, 0.0)
    return y, rounded(y, U * np.abs(y) if dtype != "f32" else 0.0 * y, dtype)


def embed_grad(tokens, d_out, v, scale, add_to, dtype):
    ok = (tokens >= 0) & (tokens < v)
    g = np.zeros((v, d_out.shape[1]))
    size = np.zeros_like(g)
    count = np.zeros(v)
    np.add.at(g, tokens[ok], d_out[ok] * scale)
    np.add.at(size, tokens[ok], np.abs(d_out[ok] * scale))
    np.add.at(count, tokens[ok], 1.0)
    b = U * (count[:, None] + 2.0) * size
    if add_to is not None:
        g = g + add_to
        b = b + U * (np.abs(add_to) + size)
    return g, rounded(g, b, dtype)


def layer_norm(x, w, b, eps, dtype):
    n, d = x.shape
    mean = x.mean(axis=1, keepdims=True)
    c = x - mean
    var = (c * c).mean(axis=1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    h = c * rstd
    y = h * w + b
    L = chain(d)
    # the first mean is off by up to L U mean|x|; the residuals' mean takes
    # that out again, to within its own sum's error
    e1 = (L + 2) * U * np.abs(x).mean(axis=1, keepdims=True)
    e_mean = U * np.abs(mean) + (L + 4) * U * (np.abs(c).mean(axis=1, keepdims=True) + e1)
    spread = np.abs(c) + e1
    e_var = (L + 6) * U * (spread * spread).mean(axis=1, keepdims=True) + e_mean * e_mean
    e_rel = 0.5 * e_var / (var + eps) + 4 * U
    e_h = rstd * (e_mean + U * np.abs(c)) + np.abs(h) * (e_rel + 2 * U)
    e_y = e_h * np.abs(w) + 3 * U * (np.abs(h * w) + np.abs(b))
    return ((y, mean[:, 0], rstd[:, 0]),
            (rounded(y, 1.05 * e_y, dtype), 1.05 * e_mean[:, 0] + U * np.abs(mean[:, 0]),
             1.05 * (e_rel * rstd)[:, 0] + U * rstd[:, 0]))


def layer_norm_grad(dy, x, mean, rstd, w, dtype, w_dtype):
    """With the f32 mean and rstd that the call is given."""
    n, d = x.shape
    mu, rs = mean[:, None], rstd[:, None]
    h = (x - mu) * rs
    g = dy * w
    a = g.mean(axis=1, keepdims=True) if n else np.zeros((0, 1))
    b = (g * h).mean(axis=1, keepdims=True) if n else np.zeros((0, 1))
    d_x = rs * (g - a - h * b)
    L = chain(d)
    e_h = 2 * U * np.abs(h)
    e_a = (L + 4) * U * np.abs(g).mean(axis=1, keepdims=True) if n else a
    e_b = (L + 7) * U * np.abs(g * h).mean(axis=1, keepdims=True) if n else b
    e = rs * (e_a + np.abs(h) * e_b + e_h * np.abs(b)
              + 5 * U * (np.abs(g) + np.abs(a) + np.abs(h * b)))
    d_w, d_b = (dy * h).sum(axis=0), dy.sum(axis=0)
    e_w = (n + 6) * U * np.abs(dy * h).sum(axis=0)
    e_db = (n + 2) * U * np.abs(dy).sum(axis=0)
    return ((d_x, d_w, d_b),
            (rounded(d_x, 1.05 * e, dtype), rounded(d_w, 1.05 * e_w, w_dtype),
             rounded(d_b, 1.05 * e_db, w_dtype)))


def f32_range(y):
    """What an f32 output holds of a value past the type's range: infinity."""
    big = float(np.finfo(np.float32).max) * (1 + U)
    return np.where(y > big, np.inf, np.where(y < -big, -np.inf, y))


def _row_parts(x):
    m = x.max(axis=1)
    empty = m == -np.inf
    none = ~(m < np.inf)  # NaN or +inf
    plain = ~(empty | none)
    safe = np.where(plain[:, None], x, 0.0)
    ms = np.where(plain, m, 0.0)
    t = safe - ms[:, None]
    e = np.exp(t)
    s = e.sum(axis=1)
    return m, empty, none, ms, t, e, s


def logprobs(x, targets, top_k):
    """Outputs (logp, entropy, stats, top_idx, top_logp) and bounds (of logp,
    entropy, stats, top_logp)."""
    n, v = x.shape
    m, empty, none, ms, t, e, s = _row_parts(x)
    ls = np.log(s)
    p = e / s[:, None]
    with np.errstate(invalid="ignore"):
        tp = np.where(p > 0, np.abs(t) * p, 0.0)
        ttp = np.where(p > 0, t * t * p, 0.0)
    H = ls + tp.sum(axis=1)  # t <= 0
    L = chain(v)
    # a term's own exponential costs (3 |t| + 2) U; what it is rescaled by on
    # the way costs as much again (the exponents add up to at most |t|)
    e_s = U * (2 * (3 * tp.sum(axis=1) + 2) + 4 * L)
    e_ls = e_s + 2 * U * np.abs(ls) + U
    mean_t = tp.sum(axis=1)
    e_u = U * (6 * ttp.sum(axis=1) + (7 + 4 * L) * mean_t)
    e_H = e_ls + e_u + mean_t * e_s + 4 * U * (np.abs(ls) + mean_t)

    def fill(y, when_empty):
        return np.where(none, np.nan, np.where(empty, when_empty, y))

    ok = (targets >= 0) & (targets < v)
    xt = t[np.arange(n), np.where(ok, targets, 0)]
    logp = np.where(ok, fill(xt - ls, -np.inf), 0.0)
    with np.errstate(invalid="ignore"):
        far = np.where(np.isfinite(xt), np.abs(xt), 0.0)
    e_logp = e_ls + 2 * U * (far + np.abs(ls))
    stats = np.stack([fill(ms, -np.inf), fill(ls, 0.0)], axis=1)
    e_stats = np.stack([0.0 * ls, e_ls], axis=1)
    idx = np.full((n, top_k), -1, np.int64)
    val = np.full((n, top_k), -np.inf)
    e_val = np.zeros((n, top_k))
    for i in range(n):
        if none[i]:
            val[i] = np.nan
            continue
        order = np.argsort(-x[i], kind="stable")[:top_k]
        order = order[x[i, order] > -np.inf]
        idx[i, :order.size] = order
        val[i, :order.size] = t[i, order] - ls[i]
        e_val[i, :order.size] = e_ls[i] + 2 * U * (np.abs(t[i, order]) + np.abs(ls[i]))
    return ((f32_range(logp), fill(H, 0.0), stats, idx, f32_range(val)),
            (1.05 * e_logp, 1.05 * e_H, 1.05 * e_stats, 1.05 * e_val))


def logprobs_grad(x, targets, stats, entropy, d_logp, d_entropy, dtype):
    """With the f32 stats and entropies that the call is given."""
    n, v = x.shape
    m, ls = stats[:, :1], stats[:, 1:]
    none = np.isnan(m)
    empty = m == -np.inf
    shut = ~(x > -np.inf) & ~none | empty
    t = np.where(shut, 0.0, x - np.where(empty, 0.0, m))
    lp = t - ls
    p = np.where(shut, 0.0, np.exp(lp))
    ok = (targets >= 0) & (targets < v)
    g = np.where(ok, d_logp, 0.0)[:, None]
    h, H = d_entropy[:, None], entropy[:, None]
    hit = np.zeros((n, v))
    hit[np.nonzero(ok)[0], targets[ok]] = 1.0
    hit[shut] = 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        f = np.where(p > 0, g + h * (lp + H), 0.0)
        y = g * hit - p * f
        far = np.where(p > 0, np.abs(t) + np.abs(lp), 0.0)
        e_f = np.where(p > 0, np.abs(h) * (2 * U * far + 2 * U * (np.abs(lp) + np.abs(H)))
                       + 2 * U * np.abs(f) + U * np.abs(g), 0.0)
        e = p * np.abs(f) * U * (2 * far + 3 * np.abs(np.where(p > 0, lp, 0.0)) + 6) + p * e_f
        e = e + U * np.abs(g * hit) + 2.0 ** -126 * np.abs(f)
    y = np.where(none, np.nan, y)
    return y, rounded(np.where(none, 0.0, y), 1.05 * np.where(none, 0.0, e), dtype)
