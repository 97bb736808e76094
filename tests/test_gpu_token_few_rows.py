"""The block and the log probabilities of few rows in every form that they are
launched in: one, two and four tiles of 16 rows, weights of one tile a block
with 8 and 16 waves and of two tiles a block, each with rests; several tiles of
classes a wave, their sums carried on."""
import numpy as np
import pytest
import torch

import sparse_archetypal_analysis_amd as saa
from tests import block_reference as R
from tests.test_gpu_token import TYPES, blank, exact, flags, untouched, within
from tests.test_gpu_token_block import ACTS, block, classes, head, vector
from tests.test_gpu_token_head_masks import LOWEST

pytestmark = pytest.mark.gpu

# (n, d, f, m): rows in two tiles and in four (f32); f of 4096 and up and of 8192 and up, m of
# 8192 and up (two tiles of weights a block), with all numbers of tiles of rows
SIZES = [(17, 40, 24, 9), (32, 72, 520, 33), (33, 40, 24, 9), (64, 136, 300, 50), (1, 64, 4099, 40),
         (16, 33, 4200, 17), (20, 24, 4100, 24), (20, 24, 8200, 24), (32, 40, 8193, 9), (1, 16, 40, 8209),
         (20, 16, 40, 8209), (31, 72, 88, 8193), (50, 24, 8200, 24), (40, 16, 40, 8209)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d,f,m", SIZES)
def test_block_of_few_rows(n, d, f, m, dtype):
    rng = np.random.default_rng(n + d + f + m)
    x, w_in, w_out = block(rng, n, d, f, m, dtype, 3, 1)
    name = ACTS[(n + d) % 3]
    base, out = blank(n, m, dtype, gap=3, start=1)
    pbase, pre = blank(n, 2 * f, dtype, gap=3, start=1)
    saa.seacells_gated_ffn(x, w_in, w_out, name, out=out, pre=pre)
    (y, p), (by, bp) = R.ffn(exact(x), exact(w_in), exact(w_out), name, dtype)
    within(pre, p, bp, "pre")
    within(out, y, by, "out")
    untouched(base, out)
    untouched(pbase, pre)
    alone, _ = saa.seacells_gated_ffn(x, w_in, w_out, name, pre=False)
    assert torch.equal(alone, out)


# (n, d, v): more than 65536 classes are several tiles of a wave
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bias", [None, "plain", "masked", "low"])
@pytest.mark.parametrize("n,d,v", [(1, 8, 140001), (3, 24, 70001), (17, 3, 66001), (30, 2, 66001),
                                   (40, 1, 131073), (64, 24, 5000)])
def test_log_probabilities_of_few_rows(n, d, v, bias, dtype):
    rng = np.random.default_rng(n + d + v)
    x, table, b = head(rng, n, d, v, dtype, "plain" if bias == "low" else bias, 3, 1)
    tgt = classes(rng, n, v)
    masked = None if b is None else exact(b)
    if bias == "low":  # (the first class tiles of some waves, the last of others)
        low = np.zeros(v, dtype=bool)
        low[1000:3000] = low[v - 3000:] = True
        b[torch.from_numpy(low).cuda()] = LOWEST
        masked = np.where(low, -np.inf, masked)
        tgt = torch.where((tgt >= 1000) & (tgt < 3000) | (tgt >= v - 3000), -1, tgt)
    logp, H, stats, st = saa.seacells_linear_logprobs(x, table, tgt, b)
    assert flags(st) == []
    want, bounds = R.loss(exact(x), exact(table), masked, exact(tgt), dtype)
    for what, g, w, e in zip(("logp", "entropy", "stats"), (logp, H, stats), want, bounds):
        within(g, w, e, what)


@pytest.mark.parametrize("dtype", TYPES)
def test_targets_of_few_rows_in_every_tile(dtype):
    """Each row's target in another tile of another wave."""
    rng = np.random.default_rng(1)
    v = 70001
    x, table, b = head(rng, 16, 24, v, dtype, "plain")
    tgt = torch.from_numpy(np.linspace(0, v - 1, 16).astype(np.int32)).cuda()
    logp, H, stats, st = saa.seacells_linear_logprobs(x, table, tgt, b)
    want, bounds = R.loss(exact(x), exact(table), exact(b), exact(tgt), dtype)
    within(logp, want[0], bounds[0], "logp")
    one = vector(rng, 16)
    got = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, one, None, b)
    want, bounds = R.loss_grad(exact(x), exact(table), exact(b), exact(tgt), exact(stats), exact(H),
                               exact(one), 0.0 * exact(one), dtype)
    for what, g, w, e in zip(("d_x", "d_table", "d_bias"), got, want, bounds):
        within(g, w, e, what)
