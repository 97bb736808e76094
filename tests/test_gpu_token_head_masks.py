"""Log probabilities from hidden rows where runs of classes have a bias at
f32's low end beside classes that have not: such a class has no probability,
in its own slice of the classes or beside others, and the entropy and every
gradient are those of the classes that are left. Against the 64-bit forms of
tests/block_reference.py with the run masked."""
import math

import numpy as np
import pytest
import torch

import sparse_archetypal_analysis_amd as saa
from tests import block_reference as R
from tests.test_gpu_token import TYPES, exact, flags, within
from tests.test_gpu_token_block import head, vector

pytestmark = pytest.mark.gpu
INF = math.inf
LOWEST = float(np.finfo(np.float32).min)


def low_classes(run, v):
    """A padded table's end (whole slices of 64 and 128); one lane's first
    classes; everything but a few."""
    low = np.zeros(v, dtype=bool)
    if run == "end":
        low[v - 200:] = True
    elif run == "start":
        low[:16] = True
    else:
        low[:] = True
        low[[5, 130, v - 1]] = False
    return low


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("run", ["end", "start", "most"])
@pytest.mark.parametrize("level", [LOWEST, -1e38, -1e37])
@pytest.mark.parametrize("n", [3, 200])
def test_runs_of_classes_at_f32s_low_end(n, level, run, dtype):
    rng = np.random.default_rng(6)
    v = 700
    x, table, b = head(rng, n, 40, v, dtype, "plain")
    low = low_classes(run, v)
    left = np.nonzero(~low)[0]
    b[torch.from_numpy(low).cuda()] = level
    tgt = rng.choice(left, n).astype(np.int32)
    tgt[0] = -1
    tgt = torch.from_numpy(tgt).cuda()
    logp, H, stats, st = saa.seacells_linear_logprobs(x, table, tgt, b)
    assert flags(st) == []
    masked = np.where(low, -INF, exact(b))  # e^(level - maximum) is 0 in 64 bits too
    want, bounds = R.loss(exact(x), exact(table), masked, exact(tgt), dtype)
    for what, g, w, e in zip(("logp", "entropy", "stats"), (logp, H, stats), want, bounds):
        within(g, w, e, what)
    gl, ge = vector(rng, n, 1.0 / n), vector(rng, n, 0.1 / n)
    for entropies in (ge, torch.zeros(n, device="cuda")):
        got = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, entropies, b)
        want, bounds = R.loss_grad(exact(x), exact(table), masked, exact(tgt), exact(stats), exact(H),
                                   exact(gl), exact(entropies), dtype)
        for what, g, w, e in zip(("d_x", "d_table", "d_bias"), got, want, bounds):
            within(g, w, e, what)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [3, 200])
@pytest.mark.parametrize("level", [LOWEST, -1e30, 3e38])
def test_gradients_where_every_class_has_the_types_end(n, level, dtype):
    """A level whose step in f32 is above every product: z is the level for all
    classes, p is 1 / v, and d_z is the incoming gradient's part alone (log p + H
    is 0 but for roundings)."""
    rng = np.random.default_rng(6)
    v = 300
    x, table, b = head(rng, n, 40, v, dtype, "plain")
    b.fill_(level)
    tgt = torch.from_numpy(rng.integers(0, v, n).astype(np.int32)).cuda()
    _, H, stats, _ = saa.seacells_linear_logprobs(x, table, tgt, b)
    one = torch.ones(n, device="cuda")
    got = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, one, one, b)
    dz = np.full((n, v), -1.0 / v)
    dz[np.arange(n), exact(tgt)] += 1.0
    # log p and H: the logarithm's rounding, the entropy's sums, H's; p: log p's error and the
    # exponential's (3 |log p| + 4), as the 64-bit form counts them
    far = math.log(v)
    e_fac = 64 * R.U * (1.0 + far)
    e_dz = (1.0 / v) * ((3 * far + 16) * R.U + e_fac) * (1 + e_fac) + 3 * R.U * np.abs(dz)
    e_b = e_dz.sum(axis=0) + (n + 4.0) * R.U * (np.abs(dz) + e_dz).sum(axis=0)
    e_dz = e_dz + (R.HALF[dtype] * (np.abs(dz) + e_dz) + 2.0 ** -38 * 18 if dtype == "f16"
                   else R.held(np.abs(dz) + e_dz, dtype))
    s, tx, tt = np.abs(dz) + e_dz, exact(x), exact(table)
    e_x = e_dz @ np.abs(tt) + R.product_bound(v, s @ np.abs(tt), dtype)
    e_t = e_dz.T @ np.abs(tx) + R.product_bound(n, s.T @ np.abs(tx), dtype)
    for what, g, w, e, t in zip(("d_x", "d_table", "d_bias"), got, (dz @ tt, dz.T @ tx, dz.sum(axis=0)),
                                (e_x, e_t, e_b), (dtype, dtype, "f32")):
        within(g, w, R.rounded(w, e, t), what)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [5, 300])
def test_masked_classes_under_large_finite_gradients(n, dtype):
    """A finite gradient whose product with a masked class' log p is past f32
    gives it nothing."""
    rng = np.random.default_rng(10)
    v = 512
    x, table, b = head(rng, n, 64, v, dtype, "plain")
    b[256:] = -INF
    tgt = torch.from_numpy(rng.integers(-1, v, n).astype(np.int32)).cuda()
    tgt[1], tgt[2] = 7, 300
    _, H, stats, _ = saa.seacells_linear_logprobs(x, table, None, b)
    gl, ge = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    ge[::2], ge[1::4] = 1e37, -1e37
    got = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, ge, b)
    want, bounds = R.loss_grad(exact(x), exact(table), exact(b), exact(tgt), exact(stats), exact(H),
                               exact(gl), exact(ge), dtype)
    assert not got[1][256:].any() and not got[2][256:].any()
    within(got[2], want[2], bounds[2], "d_bias")
    if dtype == "f16":  # (most of the others are past its range)
        assert not got[0].isnan().any() and not got[1].isnan().any()
        return
    within(got[0], want[0], bounds[0], "d_x")
    within(got[1], want[1], bounds[1], "d_table")
