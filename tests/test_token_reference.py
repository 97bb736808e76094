"""The 64-bit forms that the token operators are tested against, themselves
against central differences and small cases worked by hand (CPU)."""
import numpy as np
import pytest

from tests import token_reference as R

STEP = 1e-5


def differences(f, x):
    """Central differences of the scalar f at x."""
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += STEP
        lo[i] -= STEP
        out[i] = (f(hi) - f(lo)) / (2 * STEP)
    return out


def close(a, b):
    # (third derivatives of these functions are of order 1, so a difference is
    # off by about STEP^2 and the rounding of f over STEP, 1e-16 / 1e-5)
    np.testing.assert_allclose(a, b, rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("n,v,d", [(7, 5, 3), (1, 1, 1), (9, 4, 2)])
def test_embed_grad_is_the_lookup_s_gradient(n, v, d):
    rng = np.random.default_rng(n)
    table, tok = rng.normal(size=(v, d)), rng.integers(-1, v, n)
    dy = rng.normal(size=(n, d))
    got = R.embed_grad(tok, dy, v, 1.5, None, "f32")[0]
    close(got, differences(lambda w: (R.embed(w, tok, 1.5, "f32")[0] * dy).sum(), table))


@pytest.mark.parametrize("n,d", [(1, 2), (3, 5), (2, 16)])
def test_layer_norm_grad_is_the_forward_s_gradient(n, d):
    rng = np.random.default_rng(d)
    x, dy = rng.normal(size=(n, d)) * 2 + 0.5, rng.normal(size=(n, d))
    w, b, eps = 1 + 0.2 * rng.normal(size=d), rng.normal(size=d), 1e-2
    (_, mean, rstd), _ = R.layer_norm(x, w, b, eps, "f32")
    (dx, dw, db), _ = R.layer_norm_grad(dy, x, mean, rstd, w, "f32", "f32")

    def loss(x, w, b):
        return (R.layer_norm(x, w, b, eps, "f32")[0][0] * dy).sum()

    close(dx, differences(lambda q: loss(q, w, b), x))
    close(dw, differences(lambda q: loss(x, q, b), w))
    close(db, differences(lambda q: loss(x, w, q), b))


@pytest.mark.parametrize("n,v", [(3, 4), (1, 1), (2, 9)])
def test_logprobs_grad_is_the_forward_s_gradient(n, v):
    rng = np.random.default_rng(v)
    x = rng.normal(size=(n, v))
    tgt = rng.integers(-1, v, n)
    gl, ge = rng.normal(size=n), rng.normal(size=n)
    (_, H, stats, _, _), _ = R.logprobs(x, tgt, 0)

    def loss(q):
        (lp, h, _, _, _), _ = R.logprobs(q, tgt, 0)
        return (gl * lp + ge * h).sum()

    close(R.logprobs_grad(x, tgt, stats, H, gl, ge, "f32")[0], differences(loss, x))


def test_logprobs_of_masked_and_lost_rows():
    inf = np.inf
    x = np.array([[0.0, -inf, 0.0], [-inf] * 3, [0.0, inf, 1.0], [np.nan, 0.0, 0.0]])
    (lp, H, stats, idx, val), _ = R.logprobs(x, np.array([1, 0, -1, 0]), 3)
    assert lp[0] == -inf and lp[1] == -inf and lp[2] == 0.0 and np.isnan(lp[3])
    assert abs(H[0] - np.log(2)) < 1e-12 and H[1] == 0.0 and np.isnan(H[2:]).all()
    assert stats[1, 0] == -inf and stats[1, 1] == 0.0
    assert idx.tolist() == [[0, 2, -1], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1]]
    assert val[0, 2] == -inf and (val[1] == -inf).all() and np.isnan(val[2:]).all()
    g, _ = R.logprobs_grad(x[:2], np.array([0, 0]), stats[:2], H[:2], np.ones(2), np.ones(2), "f32")
    assert g[0, 1] == 0.0 and (g[1] == 0.0).all()
    close(g[0, [0, 2]], [0.5, -0.5])
