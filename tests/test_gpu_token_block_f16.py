"""The gated block's gradient in f16 for incoming gradients far below 1, as a
mean over rows has them: d_pre is held times a power of two by the largest of
them, and without where that would take it past f16. Against the 64-bit form
with the incoming gradients moved to 1: nothing that is held comes near f16's
smallest numbers there."""
import math

import numpy as np
import pytest
import torch

import sparse_archetypal_analysis_amd as saa
from tests import block_reference as R
from tests.test_gpu_token import DT, TYPES, exact, rows, within
from tests.test_gpu_token_block import ACTS, block

pytestmark = pytest.mark.gpu
INF = math.inf
NAMES = ("d_x", "d_w_in", "d_w_out")


def reference(d_out, x, pre, w_in, w_out, name):
    """As block_reference.ffn_grad for incoming gradients times the power of two
    that takes their largest to between 1 and 2, and back."""
    d = exact(d_out)
    up = 2.0 ** -math.floor(math.log2(np.abs(d[np.isfinite(d)]).max()))
    want, bounds = R.ffn_grad(d * up, exact(x), exact(pre), exact(w_in), exact(w_out), name, "f16")
    # (the outputs' own rounding has f16's smallest step where it is)
    return [w / up for w in want], [b / up + 1.01 * R.TINY["f16"] for b in bounds]


def operands(n, d, f, m, size):
    """x and w_in of tens: products of small d_pre are well inside of f16."""
    rng = np.random.default_rng(n + d + f)
    x, w_in, w_out = block(rng, n, d, f, m, "f16")
    x *= 50.0
    w_in *= 50.0
    return rows(rng, n, m, "f16", size), x, rows(rng, n, 2 * f, "f16"), w_in, w_out


# one row; a few; parts of k for dh; more than one block's d_out; ragged widths
SIZES = [(1, 64, 96, 72), (4, 33, 41, 17), (5, 64, 130, 4100), (66, 40, 72, 1500), (300, 130, 75, 64)]


@pytest.mark.parametrize("size", [1e-3, 1e-5, 1e-6, 2e-7])
@pytest.mark.parametrize("n,d,f,m", SIZES)
def test_small_incoming_gradients(n, d, f, m, size):
    d_out, x, pre, w_in, w_out = operands(n, d, f, m, size)
    name = ACTS[(n + d) % 3]
    got = saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out, name)
    want, bounds = reference(d_out, x, pre, w_in, w_out, name)
    for what, g, w, e in zip(NAMES, got, want, bounds):
        within(g, w, e, what)


@pytest.mark.parametrize("n,d,f,m", SIZES)
def test_a_power_of_two_less_gives_the_same_bits(n, d, f, m):
    """Gradients of d_out and of d_out / 4, both exact in f16 (from 2^-14 on)."""
    d_out, x, pre, w_in, w_out = operands(n, d, f, m, 1.0)
    d_out[d_out.abs() < 2.0 ** -4] = 0.0
    d_out.div_(256.0)
    a = saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out)
    b = saa.seacells_gated_ffn_grad(d_out / 4, x, pre, w_in, w_out)
    for p, q in zip(a, b):
        # (quarters below 2^-14 are rounded to f16's smallest step, some of them up to 2^-14)
        in_full = q.abs() > 2.0 ** -14
        assert bool(in_full.any()) and torch.equal(p[in_full], 4 * q[in_full])


@pytest.mark.parametrize("n,d,f,m", SIZES)
def test_scaled_numbers_past_f16_are_done_without(n, d, f, m):
    """d_out of 2^-10 against w_out of tens and up rows of thousands: times 2^10
    d_pre would be past f16, as it is it is not."""
    rng = np.random.default_rng(n + d + f)
    x, w_in, w_out = block(rng, n, d, f, m, "f16")
    x *= 2.0 ** -8
    w_in *= 2.0 ** -8
    w_out *= 128.0
    pre = rows(rng, n, 2 * f, "f16")
    pre[:, f:] *= 3000.0
    d_out = rows(rng, n, m, "f16", 2.0 ** -12)
    d_out[0, 0] = 2.0 ** -10
    want, bounds = R.ffn_grad(exact(d_out), exact(x), exact(pre), exact(w_in), exact(w_out), "silu", "f16")
    g, u = exact(pre)[:, :f], exact(pre)[:, f:]
    d_pre = np.abs((exact(d_out) @ exact(w_out)) * u * R.act(g, "silu")[1])
    assert d_pre.max() < 6e4 and d_pre.max() * 2.0 ** 9 > 7e4
    got = saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out, "silu")
    for what, a, w, e in zip(NAMES, got, want, bounds):
        assert bool(a.isfinite().all())
        within(a, w, e, what)


@pytest.mark.parametrize("n,d,f,m", SIZES)
def test_each_gradient_alone(n, d, f, m):
    given = operands(n, d, f, m, 1e-5)
    want = saa.seacells_gated_ffn_grad(*given)
    for i in range(3):
        alone = saa.seacells_gated_ffn_grad(*given, **{k: False for j, k in enumerate(NAMES) if j != i})
        for j in range(3):
            assert alone[j] is None if j != i else torch.equal(alone[j], want[j])


@pytest.mark.parametrize("bad", [INF, -INF, float("nan"), 0.0])
def test_rows_that_are_not_finite_choose_no_scale(bad):
    """A row of infinities or NaN, or of 0, changes no other row's bits."""
    d_out, x, pre, w_in, w_out = operands(70, 40, 72, 90, 1e-5)
    want = saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out)[0]
    top = d_out.abs().amax(dim=1).argmin()  # (the largest stays where it is)
    d_out[top] = bad
    got = saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out)
    keep = torch.ones(70, dtype=torch.bool, device="cuda")
    keep[top] = False
    assert torch.equal(want[keep], got[0][keep])
    if bad == 0.0:
        assert not got[0][top].any()
        d_out.zero_()
        assert not any(g.any() for g in saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out))


def test_a_graph_scales_each_replay():
    """Replays with other gradients: small ones, ones that are done without a
    scale, ones of 1 and more."""
    d_out, x, pre, w_in, w_out = operands(300, 64, 200, 96, 1.0)
    x.div_(2.0 ** 10)
    w_in.div_(2.0 ** 10)
    w_out.mul_(128.0)
    saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out)
    plain, large = pre.clone(), pre.clone()
    large[:, 200:] *= 2000.0
    base = d_out.clone()
    for size, p in ((1e-5, plain), (2.0 ** -12, large), (1e-5, plain), (1.0, plain), (2.0 ** -12, large)):
        d_out.copy_(base * size)
        pre.copy_(p)
        want = saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b) and bool(a.isfinite().all())


@pytest.mark.parametrize("dtype", TYPES)
def test_workspaces_of_many_rows(dtype):
    """Exactly the query's bytes, between marks that stay."""
    rng = np.random.default_rng(5)
    n, d, f, m = 900, 40, 72, 1500
    x, w_in, w_out = block(rng, n, d, f, m, dtype)
    d_out, pre = rows(rng, n, m, dtype, 1e-5), rows(rng, n, 2 * f, dtype)
    want = saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out)
    for on_16 in (True, False):
        size = saa.seacells_gated_ffn_grad_workspace(DT[dtype], n, d, f, m, on_16_bytes=on_16)
        if on_16 and m % 8:  # (d_out's rows are copied)
            continue
        base = torch.full((size + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        got = saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out, workspace=base[256:256 + size])
        assert all(torch.equal(p, q) for p, q in zip(want, got))
        assert bool((base[:256] == 0x5A).all()) and bool((base[256 + size:] == 0x5A).all())
