"""f16 gradients of the head where the incoming gradients are far from 1, or
where some rows' are and have no part: d_z is held times a power of two that
the rows which take part choose."""
import math

import numpy as np
import pytest
import torch

import sparse_archetypal_analysis_amd as saa
from tests import block_reference as R
from tests.test_gpu_token import TYPES, exact, flags, rows, within
from tests.test_gpu_token_block import classes, head, vector

pytestmark = pytest.mark.gpu
INF = math.inf


def same(a, b):
    for p, q in zip(a, b):
        assert (p is None and q is None) or torch.equal(p, q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("huge", [3e38, 1e30, 2e4])
@pytest.mark.parametrize("n", [5, 500, 5000])
def test_ignored_rows_have_no_part(n, huge, dtype):
    """d_logp of a row whose target is ignored, of any size: the bits that 0
    there gives."""
    rng = np.random.default_rng(9)
    x, table, b = head(rng, n, 64, 800, dtype, "masked")
    tgt = classes(rng, n, 800)
    tgt[1], tgt[n - 1] = -1, 800
    out = (tgt < 0) | (tgt >= 800)
    _, H, stats, _ = saa.seacells_linear_logprobs(x, table, None, b)
    gl, ge = vector(rng, n, 1.0 / n), vector(rng, n, 0.1 / n)
    gl[out] = 0.0
    want = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, ge, b)
    bounds = R.loss_grad(exact(x), exact(table), exact(b), exact(tgt), exact(stats), exact(H), exact(gl),
                         exact(ge), dtype)
    within(want[0], bounds[0][0], bounds[1][0], "d_x")
    gl[out] = huge
    gl[1] = -huge
    got = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, ge, b)
    assert flags(got[3]) == ["BAD_INDEX"]
    same(want[:3], got[:3])
    # no targets at all: d_logp has no part
    same(saa.seacells_linear_logprobs_grad(x, table, None, stats, H, None, ge, b)[:3],
         saa.seacells_linear_logprobs_grad(x, table, None, stats, H, gl, ge, b)[:3])


@pytest.mark.parametrize("dtype", ("f16", "bf16"))
@pytest.mark.parametrize("lost", [-INF, float("nan")])
def test_rows_with_nothing_left_have_no_part(lost, dtype):
    """Rows whose z are all -inf, or NaN, under large incoming gradients: the
    other rows' d_x has the bits that 0 there gives."""
    rng = np.random.default_rng(9)
    x, table, _ = head(rng, 60, 64, 800, dtype, None)
    table.abs_()
    tgt = classes(rng, 60, 800)
    tgt[7], tgt[8] = 3, 4
    x[7:9] = lost
    _, H, stats, _ = saa.seacells_linear_logprobs(x, table, None)
    assert bool((stats[7:9, 0] == -INF).all() if lost == -INF else stats[7:9, 0].isnan().all())
    gl, ge = vector(rng, 60, 1e-3), vector(rng, 60, 1e-4)
    gl[7:9] = ge[7:9] = 0.0
    want = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, ge, d_table=False)[0]
    gl[7] = ge[8] = 1e30
    got = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, ge, d_table=False)[0]
    keep = torch.ones(60, dtype=torch.bool, device="cuda")
    keep[7:9] = False
    assert torch.equal(want[keep], got[keep])
    assert not got[7:9].any() if lost == -INF else bool(got[7:9].isnan().all())


@pytest.mark.parametrize("which", ["logp", "entropy"])
@pytest.mark.parametrize("n", [5, 300])
def test_incoming_gradients_at_f32s_end(n, which):
    """Gradients as large as f32 goes (for entropy: as 17 times them does not
    go) stay numbers: where x or the table is 0 their products are 0, elsewhere
    they are past f16, to the side that the formula says."""
    rng = np.random.default_rng(9)
    x, table, b = head(rng, n, 64, 800, "f16", "plain")
    x *= 0.25  # (log p stays above -15: with entropies' gradients it is a number)
    x[:, 3] = 0.0
    table[:, 5] = 0.0
    tgt = classes(rng, n, 800)
    tgt[0] = 7
    _, H, stats, _ = saa.seacells_linear_logprobs(x, table, None, b)
    sign = torch.where(vector(rng, n) > 0, 1.0, -1.0)
    zero = torch.zeros(n, device="cuda")
    gl, ge = (3e38 * sign, zero) if which == "logp" else (zero, 2.1e37 * sign)
    dx, dt, _, _ = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, ge, b)
    assert not dx[:, 5].any() and not dt[:, 3].any()
    want, bounds = R.loss_grad(exact(x), exact(table), exact(b), exact(tgt), exact(stats), exact(H),
                               exact(gl), exact(ge), "f16")
    sure = np.abs(want[0]) > bounds[0] + 1e6
    assert sure.mean() > 0.5
    assert np.array_equal(exact(dx)[sure], np.sign(want[0][sure]) * INF)
