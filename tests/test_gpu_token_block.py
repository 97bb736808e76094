"""The gated feed-forward block and the log probabilities from hidden rows
(include/seacells_token.h) against their 64-bit forms
(tests/block_reference.py), element by element within the bounds derived
there: sizes from one element on, odd widths, row strides and starts at any
element, masks, empty rows, parts of k and pieces of the classes, both sizes
of tiles, side streams, graph replays and a run of the operators together."""
import math

import numpy as np
import pytest
import torch

import sparse_archetypal_analysis_amd as saa
from tests import block_reference as R
from tests.test_gpu_token import DT, TYPES, blank, exact, flags, rows, untouched, within

pytestmark = pytest.mark.gpu
INF = math.inf
ACTS = ["silu", "gelu", "relu"]


def classes(rng, n, v):
    t = rng.integers(0, v, n)
    t[rng.random(n) < 0.1] = -1 - int(rng.integers(0, 5))
    return torch.from_numpy(t.astype(np.int32)).cuda()


def vector(rng, n, scale=1.0):
    return torch.from_numpy(scale * rng.normal(size=n)).cuda().float()


# --- gated block ----------------------------------------------------------------

# (n, d, f, m): one element; whole tiles; odd everything; more rows than a tile;
# few rows against wide weights (parts of k); many rows against narrow ones (parts of the
# weights' gradients); enough of all for tiles of 256
FFN_SIZES = [(1, 1, 1, 1), (1, 64, 128, 64), (3, 8, 16, 8), (2, 33, 7, 5), (65, 100, 70, 90),
             (129, 256, 300, 257), (300, 130, 520, 64), (257, 1003, 131, 77), (1030, 64, 96, 40),
             (7, 1100, 2050, 520), (16, 2048, 96, 1032), (5000, 24, 40, 17), (2300, 72, 2600, 1030)]


def block(rng, n, d, f, m, dtype, gap=0, start=0):
    x = rows(rng, n, d, dtype, gap=gap, start=start)
    w_in = rows(rng, 2 * f, d, dtype, 1.5 / math.sqrt(d), gap=gap, start=start)
    w_out = rows(rng, m, f, dtype, 1.0 / math.sqrt(f), gap=gap, start=start)
    return x, w_in, w_out


def layout(width):
    return (0, 0) if width % 8 == 0 else (3, 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d,f,m", FFN_SIZES)
def test_gated_ffn(n, d, f, m, dtype):
    rng = np.random.default_rng(n + d + f)
    gap, start = layout(d | f | m)
    x, w_in, w_out = block(rng, n, d, f, m, dtype, gap, start)
    name = ACTS[(n + d) % 3]
    base, out = blank(n, m, dtype, gap=gap, start=start)
    pbase, pre = blank(n, 2 * f, dtype, gap=gap, start=start)
    got, kept = saa.seacells_gated_ffn(x, w_in, w_out, name, out=out, pre=pre)
    assert got is out and kept is pre
    (y, p), (by, bp) = R.ffn(exact(x), exact(w_in), exact(w_out), name, dtype)
    within(pre, p, bp, "pre")
    within(out, y, by, "out")
    untouched(base, out)
    untouched(pbase, pre)
    alone, none = saa.seacells_gated_ffn(x, w_in, w_out, name, pre=False)
    assert none is None and torch.equal(alone, out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d,f,m", FFN_SIZES)
def test_gated_ffn_grad(n, d, f, m, dtype):
    rng = np.random.default_rng(n + d + f)
    gap, start = layout(d | f | m)
    x, w_in, w_out = block(rng, n, d, f, m, dtype, gap, start)
    name = ACTS[(n + d + 1) % 3]
    pre = rows(rng, n, 2 * f, dtype, gap=gap, start=start)
    d_out = rows(rng, n, m, dtype, gap=gap, start=start)
    outs = [blank(*s, dtype, gap=gap, start=start) for s in ((n, d), (2 * f, d), (m, f))]
    got = saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out, name, d_x=outs[0][1],
                                      d_w_in=outs[1][1], d_w_out=outs[2][1])
    want, bounds = R.ffn_grad(exact(d_out), exact(x), exact(pre), exact(w_in), exact(w_out), name,
                              dtype)
    for what, g, (base, out), w, b in zip(("d_x", "d_w_in", "d_w_out"), got, outs, want, bounds):
        assert g is out
        within(out, w, b, what)
        untouched(base, out)
    for left_out in range(3):
        kw = {k: False for i, k in enumerate(("d_x", "d_w_in", "d_w_out")) if i == left_out}
        some = saa.seacells_gated_ffn_grad(d_out, x, pre, w_in, w_out, name, **kw)
        for i in range(3):
            assert some[i] is None if i == left_out else torch.equal(some[i], got[i])


@pytest.mark.parametrize("name", ACTS)
def test_activations_from_end_to_end(name):
    """g over the type's range through a block that passes it: d = f = m, one
    weight each (f32: the type's largest steps of act and act')."""
    g = torch.cat([torch.linspace(-30, 30, 4001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 80.0, -80.0,
                                                                -120.0, 120.0, 1e4, -1e4])])
    x = torch.stack([g, torch.ones_like(g)], dim=1).cuda()
    w_in = torch.eye(2, device="cuda")
    w_out = torch.ones(1, 1, device="cuda")
    y, pre = saa.seacells_gated_ffn(x, w_in, w_out, name)
    (want, p), (bound, bp) = R.ffn(exact(x), exact(w_in), exact(w_out), name, "f32")
    within(pre, p, bp, "pre")
    within(y, want, bound, "act")
    one = torch.ones(g.numel(), 1, device="cuda")
    got = saa.seacells_gated_ffn_grad(one, x, pre, w_in, w_out, name)
    want, bounds = R.ffn_grad(exact(one), exact(x), exact(pre), exact(w_in), exact(w_out), name, "f32")
    for what, a, w, b in zip(("d_x", "d_w_in", "d_w_out"), got, want, bounds):
        within(a, w, b, what)


@pytest.mark.parametrize("name", ACTS)
def test_gated_ffn_grad_against_differences(name):
    """Central differences of the 64-bit block, on the inputs' own grid."""
    rng = np.random.default_rng(8)
    n, d, f, m = 4, 6, 9, 5
    x, w_in, w_out = (exact(t) for t in block(rng, n, d, f, m, "f32"))
    d_out = rng.normal(size=(n, m)).astype(np.float32)
    pre = (x @ w_in.T).astype(np.float32)
    pre[np.abs(pre) < 1e-2] = 0.5  # away from relu's corner
    dev = [torch.from_numpy(np.float32(t)).cuda() for t in (d_out, x, pre, w_in, w_out)]
    got = [exact(t) for t in saa.seacells_gated_ffn_grad(*dev, name)]
    p, e = pre.astype(np.float64), 1e-5

    def value(dx, dwi, dwo):
        # pre moves with x and w_in from where it is given
        q = p + (x + dx) @ (w_in + dwi).T - x @ w_in.T
        return ((R.act(q[:, :f], name)[0] * q[:, f:]) @ (w_out + dwo).T * d_out).sum()

    zero = [0.0 * x, 0.0 * w_in, 0.0 * w_out]
    for i, g in enumerate(got):
        for at in [tuple(rng.integers(0, s) for s in g.shape) for _ in range(12)]:
            step = [z.copy() for z in zero]
            step[i][at] = e
            up = value(*step)
            step[i][at] = -e
            want = (up - value(*step)) / (2 * e)
            # the differences' own error: e^2 times a third derivative of a few
            assert abs(g[at] - want) <= 1e-5 * (1.0 + abs(want)), (i, at)


def test_gated_ffn_of_no_rows():
    for dt in DT.values():
        x = torch.empty(0, 24, dtype=dt, device="cuda")
        w_in, w_out = (torch.ones(s, dtype=dt, device="cuda") for s in ((20, 24), (7, 10)))
        y, pre = saa.seacells_gated_ffn(x, w_in, w_out)
        assert y.shape == (0, 7) and pre.shape == (0, 20)
        dx, di, do = saa.seacells_gated_ffn_grad(y, x, pre, w_in, w_out)
        assert dx.shape == (0, 24) and not di.any() and not do.any()
        assert di.shape == (20, 24) and do.shape == (7, 10)


def test_gated_ffn_keeps_leading_dimensions_and_lost_rows_apart():
    """A row of NaN or infinities changes no other row; NaN reaches every
    gradient of the weights that it has a part in."""
    rng = np.random.default_rng(3)
    for dtype in TYPES:
        x, w_in, w_out = block(rng, 12, 40, 24, 16, dtype)
        y, _ = saa.seacells_gated_ffn(x.view(3, 4, 40), w_in, w_out)
        assert y.shape == (3, 4, 16)
        x2 = x.clone()
        x2[5] = float("nan")
        x2[7, 3] = INF
        y2, _ = saa.seacells_gated_ffn(x2, w_in, w_out)
        keep = torch.ones(12, dtype=torch.bool, device="cuda")
        keep[[5, 7]] = False
        assert torch.equal(y2[keep], y.view(12, 16)[keep])
        assert bool(y2[5].isnan().all()) and not bool(y2[7].isfinite().any())


def test_gated_ffn_rows_beyond_4_gib():
    far = 2 ** 31 + 16
    base = torch.empty(far + 4096, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(3)
    x, w_in, w_out = block(rng, 2, 512, 64, 24, "bf16")
    apart = base.as_strided((2, 512), (far, 1))
    apart.copy_(x)
    want = saa.seacells_gated_ffn(x, w_in, w_out)
    got = saa.seacells_gated_ffn(apart, w_in, w_out)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    d_out = rows(rng, 2, 24, "bf16")
    a = saa.seacells_gated_ffn_grad(d_out, x, want[1], w_in, w_out)
    b = saa.seacells_gated_ffn_grad(d_out, apart, want[1], w_in, w_out, d_x=apart.clone())
    for p, q in zip(a, b):
        assert torch.equal(p, q)


# --- log probabilities from hidden rows -------------------------------------------

# (n, d, v)
LOSS_SIZES = [(1, 1, 1), (1, 16, 2), (3, 33, 7), (2, 64, 500), (130, 100, 129), (64, 24, 1300),
              (1, 520, 5000), (17, 300, 4099), (300, 72, 257), (2100, 40, 1000), (700, 1003, 65),
              (5000, 8, 33), (1100, 264, 2500)]


def head(rng, n, d, v, dtype, bias, gap=0, start=0):
    x = rows(rng, n, d, dtype, gap=gap, start=start)
    table = rows(rng, v, d, dtype, 2.5 / math.sqrt(d), gap=gap, start=start)
    b = None
    if bias:
        b = vector(rng, v)
        if bias == "masked":
            b[torch.from_numpy(rng.random(v) < 0.4).cuda()] = -INF
            b[-1] = 0.25
            if v > 2:
                b[1] = -3e38  # a mask of nearly the type's lowest value
    return x, table, b


def check_loss(x, table, b, tgt, dtype):
    logp, H, stats, st = saa.seacells_linear_logprobs(x, table, tgt, b)
    assert flags(st) == []
    want, bounds = R.loss(exact(x), exact(table), None if b is None else exact(b), exact(tgt), dtype)
    for what, g, w, e in zip(("logp", "entropy", "stats"), (logp, H, stats), want, bounds):
        within(g, w, e, what)
    return logp, H, stats


@pytest.mark.parametrize("bias", [None, "plain", "masked"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d,v", LOSS_SIZES)
def test_linear_logprobs(n, d, v, dtype, bias):
    rng = np.random.default_rng(n + d + v)
    gap, start = layout(d)
    x, table, b = head(rng, n, d, v, dtype, bias, gap, start)
    check_loss(x, table, b, classes(rng, n, v), dtype)
    logp, H, stats, _ = saa.seacells_linear_logprobs(x, table, None, b)
    assert logp is None and H.shape == (n,) and stats.shape == (n, 2)


@pytest.mark.parametrize("bias", [None, "masked"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d,v", LOSS_SIZES)
def test_linear_logprobs_grad(n, d, v, dtype, bias):
    rng = np.random.default_rng(n + d + v)
    gap, start = layout(d)
    x, table, b = head(rng, n, d, v, dtype, bias, gap, start)
    tgt = classes(rng, n, v)
    _, H, stats, _ = saa.seacells_linear_logprobs(x, table, None, b)
    gl, ge = vector(rng, n, 1.0 / n), vector(rng, n, 0.1 / n)
    outs = [blank(*s, dtype, gap=gap, start=start) for s in ((n, d), (v, d))]
    d_bias = torch.full((v,), 7.0, device="cuda") if b is not None else None
    got = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, ge, b, d_x=outs[0][1],
                                            d_table=outs[1][1], d_bias=d_bias)
    assert flags(got[3]) == []
    bx = None if b is None else exact(b)
    ref = (exact(x), exact(table), bx, exact(tgt), exact(stats), exact(H))
    want, bounds = R.loss_grad(*ref, exact(gl), exact(ge), dtype)
    for what, (base, out), w, e in zip(("d_x", "d_table"), outs, want, bounds):
        within(out, w, e, what)
        untouched(base, out)
    if b is not None:
        within(d_bias, want[2], bounds[2], "d_bias")
    # each gradient alone, each incoming gradient alone
    only = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, ge, b, d_table=False,
                                             d_bias=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], outs[0][1])
    only = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, ge, b, d_x=False)
    assert only[0] is None and torch.equal(only[1], outs[1][1])
    zero = np.zeros(n)
    want, bounds = R.loss_grad(*ref, exact(gl), zero, dtype)
    within(saa.seacells_linear_logprobs_grad(x, table, tgt, stats, None, gl, None, b)[0], want[0],
           bounds[0], "d_x of logp")
    want, bounds = R.loss_grad(*ref, zero, exact(ge), dtype)
    within(saa.seacells_linear_logprobs_grad(x, table, None, stats, H, gl, ge, b)[1], want[1],
           bounds[1], "d_table of entropy")


@pytest.mark.parametrize("dtype", TYPES)
def test_loss_gradient_in_pieces_of_the_classes(dtype):
    """Enough rows that d_z takes several pieces (256 MB each), checked on a
    few of the rows and classes."""
    n, d, v = 300000, 16, 1000
    rng = np.random.default_rng(6)
    x, table, b = head(rng, n, d, v, dtype, "plain")
    tgt = classes(rng, n, v)
    _, H, stats, _ = saa.seacells_linear_logprobs(x, table, None, b)
    gl, ge = vector(rng, n), vector(rng, n, 0.1)
    # rows without a gradient of their own drop out of the sums over rows
    keep = torch.zeros(n, dtype=torch.bool, device="cuda")
    keep[torch.from_numpy(rng.choice(n, 700, replace=False)).cuda()] = True
    gl[~keep] = 0.0
    ge[~keep] = 0.0
    dx, dt, db, _ = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, ge, b)
    assert not dx[~keep].any()
    want, bounds = R.loss_grad(exact(x[keep]), exact(table), exact(b), exact(tgt[keep]),
                               exact(stats[keep]), exact(H[keep]), exact(gl[keep]), exact(ge[keep]),
                               dtype)
    within(dx[keep], want[0], bounds[0], "d_x")
    within(dt, want[1], bounds[1], "d_table")
    within(db, want[2], bounds[2], "d_bias")


@pytest.mark.parametrize("dtype", TYPES)
def test_every_class_masked(dtype):
    rng = np.random.default_rng(6)
    x, table, b = head(rng, 5, 40, 300, dtype, "plain")
    tgt = torch.tensor([3, -1, 299, 0, 7], dtype=torch.int32, device="cuda")
    b.fill_(-INF)
    table[7] = float("nan")  # (a masked class' row holds anything)
    logp, H, stats, st = saa.seacells_linear_logprobs(x, table, tgt, b)
    assert flags(st) == [] and logp.tolist() == [-INF, 0.0, -INF, -INF, -INF]
    assert not H.any() and stats.tolist() == [[-INF, 0.0]] * 5
    table[7] = 1.0
    one = torch.ones(5, device="cuda")
    dx, dt, db, _ = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, one, one, b)
    assert not dx.any() and not dt.any() and not db.any()


@pytest.mark.parametrize("n", [3, 200])
@pytest.mark.parametrize("level", [-3.4028234e38, -1e30, 3e38])
def test_biases_of_the_types_ends(n, level):
    """Every class shifted as far as f32 goes: the classes are equally likely,
    whatever their z was, as where logits are masked by the lowest value."""
    rng = np.random.default_rng(6)
    x, table, b = head(rng, n, 40, 300, "bf16", "plain")
    b.fill_(level)
    tgt = classes(rng, n, 300)
    logp, H, stats = check_loss(x, table, b, tgt, "bf16")
    assert bool((H - math.log(300)).abs().max() < 1e-5)
    one = torch.ones(n, device="cuda")
    got = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, one, one, b)
    want, bounds = R.loss_grad(exact(x), exact(table), exact(b), exact(tgt), exact(stats), exact(H),
                               np.ones(n), np.ones(n), "bf16")
    for what, g in zip(("d_x", "d_table", "d_bias"), got):
        assert bool(g.isfinite().all()), what
    # p is 1 / 300 to its rounding: z and m are the same number
    p = np.full((n, 300), 1.0 / 300)
    dz = -p
    t = exact(tgt)
    dz[t < 0] = 0.0
    dz[np.nonzero(t >= 0)[0], t[t >= 0]] += 1.0
    assert np.abs(exact(got[2]) - dz.sum(axis=0)).max() < 1e-4 * n


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_classes_have_no_part(dtype):
    """What a masked class' row holds reaches no output but its own d_table;
    a masked target has log probability -inf and no gradient."""
    rng = np.random.default_rng(7)
    x, table, b = head(rng, 40, 48, 700, dtype, "plain")
    b[100:500] = -INF
    tgt = classes(rng, 40, 700)
    tgt[0] = 250
    a = saa.seacells_linear_logprobs(x, table, tgt, b)
    t2 = table.clone()
    t2[100:500] = float("nan")
    c = saa.seacells_linear_logprobs(x, t2, tgt, b)
    for p, q in zip(a, c):
        assert torch.equal(p, q)
    assert a[0][0] == -INF
    one = torch.ones(40, device="cuda")
    dx, dt, db, _ = saa.seacells_linear_logprobs_grad(x, table, tgt, a[2], a[1], one, one, b)
    assert not dt[100:500].any() and not db[100:500].any() and bool(dx.isfinite().all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [INF, -INF, float("nan")])
def test_masked_places_under_gradients_that_are_not_finite(dtype, bad):
    """Masked classes get nothing from a row whose incoming gradients are not
    finite, and a row with nothing left gets and gives nothing."""
    rng = np.random.default_rng(11)
    x, table, b = head(rng, 300, 48, 700, dtype, "plain")
    b[100:500] = -INF
    tgt = classes(rng, 300, 700)
    tgt[7], tgt[8], tgt[9] = 20, 250, -1
    _, H, stats, _ = saa.seacells_linear_logprobs(x, table, tgt, b)
    for which in ("logp", "entropy"):
        g, h = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
        (g if which == "logp" else h)[7:10] = bad
        dx, dt, db, _ = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, g, h, b)
        assert not dt[100:500].any() and not db[100:500].any()
        assert bool(dx[10:].isfinite().all()) and bool(dx[:7].isfinite().all())
    b[:] = -INF
    _, H, stats, _ = saa.seacells_linear_logprobs(x, table, tgt, b)
    g, h = torch.full((300,), bad, device="cuda"), torch.full((300,), bad, device="cuda")
    dx, dt, db, _ = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, g, h, b)
    assert not dx.any() and not dt.any() and not db.any()


@pytest.mark.parametrize("dtype", ("f16", "bf16"))
def test_rows_with_nothing_left_without_a_bias(dtype):
    """Every z is -inf from the operands: no gradient either."""
    x = torch.ones(5, 8, device="cuda").to(DT[dtype])
    table = torch.full((12, 8), -INF, device="cuda").to(DT[dtype])
    tgt = torch.tensor([0, 11, 3, -1, 4], dtype=torch.int32, device="cuda")
    logp, H, stats, _ = saa.seacells_linear_logprobs(x, table, tgt)
    assert bool((stats[:, 0] == -INF).all()) and not stats[:, 1].any() and not H.any()
    assert torch.equal(logp.cpu(), torch.tensor([-INF, -INF, -INF, 0.0, -INF]))
    g = torch.full((5,), 2.0, device="cuda")
    _, dt, db, _ = saa.seacells_linear_logprobs_grad(
        x, table, tgt, stats, H, g, g, d_x=False, d_bias=torch.empty(12, device="cuda"))
    assert not dt.any() and not db.any()


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_without_a_distribution(dtype):
    rng = np.random.default_rng(7)
    x, table, b = head(rng, 30, 48, 900, dtype, "plain")
    tgt = classes(rng, 30, 900)
    tgt[4], tgt[5] = -1, 3
    want = saa.seacells_linear_logprobs(x, table, tgt, b)
    x2 = x.clone()
    x2[4, 1] = float("nan")
    x2[5] = INF
    got = saa.seacells_linear_logprobs(x2, table, tgt, b)
    keep = torch.ones(30, dtype=torch.bool, device="cuda")
    keep[[4, 5]] = False
    for p, q in zip(want[:3], got[:3]):
        assert torch.equal(p[keep], q[keep])
    assert got[0][4] == 0 and bool(got[0][5].isnan())
    assert bool(got[1][4:6].isnan().all()) and bool(got[2][4:6].isnan().all())
    one = torch.ones(30, device="cuda")
    full = saa.seacells_linear_logprobs_grad(x, table, tgt, want[2], want[1], one, one, b)
    lost = saa.seacells_linear_logprobs_grad(x2, table, tgt, got[2], got[1], one, one, b)
    assert torch.equal(full[0][keep], lost[0][keep]) and bool(lost[0][4:6].isnan().all())
    assert bool(lost[1].isnan().all()) and bool(lost[2].isnan().all())


def test_classes_beyond_the_table():
    rng = np.random.default_rng(7)
    x, table, b = head(rng, 20, 16, 30, "f32", None)
    tgt, st = classes(rng, 20, 30), torch.full((1,), -1, dtype=torch.int32, device="cuda")
    assert flags(saa.seacells_linear_logprobs(x, table, tgt, status=st)[3]) == []
    tgt[19] = 30
    logp, H, stats, _ = saa.seacells_linear_logprobs(x, table, tgt, status=st)
    assert flags(st) == ["BAD_INDEX"] and logp[19] == 0
    one = torch.ones(20, device="cuda")
    st.fill_(-1)
    a = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, d_logp=one, status=st)
    assert flags(st) == ["BAD_INDEX"] and not a[0][19].any()
    tgt[19] = -1
    b = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, d_logp=one, status=st)
    assert flags(st) == [] and torch.equal(a[1], b[1])
    st.fill_(-1)
    saa.seacells_linear_logprobs_grad(x, table, None, stats, d_logp=one, status=st)
    assert flags(st) == []


def test_loss_of_no_rows():
    x, table = torch.empty(0, 9, device="cuda"), torch.ones(4, 9, device="cuda")
    none, b = torch.empty(0, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    logp, H, stats, _ = saa.seacells_linear_logprobs(x, table, none, b, status=st)
    assert logp.shape == (0,) and H.shape == (0,) and stats.shape == (0, 2) and flags(st) == []
    st.fill_(-1)
    dx, dt, db, _ = saa.seacells_linear_logprobs_grad(x, table, none, stats, H, H, H, b, status=st)
    assert dx.shape == (0, 9) and not dt.any() and not db.any() and flags(st) == []


@pytest.mark.parametrize("scale", [1e-6, 1.0, 1e4])
def test_f16_gradients_of_any_size(scale):
    """d_z of a mean over many rows is far below f16's range, the sums are not."""
    rng = np.random.default_rng(9)
    n, d, v = 500, 64, 800
    x, table, _ = head(rng, n, d, v, "f16", None)
    table *= 0.25
    x *= 0.25
    tgt = classes(rng, n, v)
    _, H, stats, _ = saa.seacells_linear_logprobs(x, table, None)
    gl, ge = vector(rng, n, scale), vector(rng, n, 0.1 * scale)
    got = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, ge)
    want, bounds = R.loss_grad(exact(x), exact(table), None, exact(tgt), exact(stats), exact(H),
                               exact(gl), exact(ge), "f16")
    within(got[0], want[0], bounds[0], "d_x")
    within(got[1], want[1], bounds[1], "d_table")


def test_loss_rows_beyond_4_gib():
    far = 2 ** 31 + 16
    base = torch.empty(far + 4096, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(3)
    x, table, _ = head(rng, 2, 512, 900, "bf16", None)
    apart = base.as_strided((2, 512), (far, 1))
    apart.copy_(x)
    tgt = torch.tensor([5, 899], dtype=torch.int32, device="cuda")
    a, b = (saa.seacells_linear_logprobs(t, table, tgt) for t in (x, apart))
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    one = torch.ones(2, device="cuda")
    a, b = (saa.seacells_linear_logprobs_grad(t, table, tgt, a[2], a[1], one, one) for t in (x, apart))
    for p, q in zip(a, b):
        assert (p is None and q is None) or torch.equal(p, q)


# --- sizes of large tiles, strides, workspaces ---------------------------------------

def some(rng, n, count=48):
    """Indexes at both ends and between."""
    at = np.unique(np.concatenate([[0, 1, n - 1], rng.integers(0, n, count)]))
    return at, torch.from_numpy(at).cuda()


@pytest.mark.parametrize("dtype", TYPES)
def test_large_blocks_of_results(dtype):
    """Enough rows and columns that tiles of 256 are taken, with ragged ends, on
    a few of the rows and columns."""
    rng = np.random.default_rng(4)
    n, d, f, m = 4103, 1040, 8200, 4104
    x, w_in, w_out = block(rng, n, d, f, m, dtype)
    y, pre = saa.seacells_gated_ffn(x, w_in, w_out, "silu")
    at, dev = some(rng, n)
    want, bounds = R.ffn(exact(x[dev]), exact(w_in), exact(w_out), "silu", dtype)
    within(y[dev], want[0], bounds[0], "out")
    within(pre[dev], want[1], bounds[1], "pre")
    dy = rows(rng, n, m, dtype)
    dx, di, do = saa.seacells_gated_ffn_grad(dy, x, pre, w_in, w_out, "silu")
    want, bounds = R.ffn_grad(exact(dy[dev]), exact(x[dev]), exact(pre[dev]), exact(w_in), exact(w_out),
                              "silu", dtype)
    within(dx[dev], want[0], bounds[0], "d_x")
    cols, dcols = some(rng, f)
    both = torch.cat([dcols, dcols + f])
    want, bounds = R.ffn_grad(exact(dy), exact(x), exact(pre[:, both]), exact(w_in[both]),
                              exact(w_out[:, dcols]), "silu", dtype)
    within(di[both], want[1], bounds[1], "d_w_in")
    within(do[:, dcols], want[2], bounds[2], "d_w_out")


@pytest.mark.parametrize("bias", [None, "plain"])
@pytest.mark.parametrize("dtype", TYPES)
def test_large_blocks_of_logits(dtype, bias):
    rng = np.random.default_rng(4)
    n, d, v = 4103, 1040, 8199
    x, table, b = head(rng, n, d, v, dtype, bias)
    at, dev = some(rng, n)
    cls, dcls = some(rng, v)
    local = rng.integers(0, cls.size, n)
    tgt = torch.from_numpy(cls[local].astype(np.int32)).cuda()
    logp, H, stats, _ = saa.seacells_linear_logprobs(x, table, tgt, b)
    want, bounds = R.loss(exact(x[dev]), exact(table), None if b is None else exact(b), exact(tgt[dev]), dtype)
    for what, g, w, e in zip(("logp", "entropy", "stats"), (logp, H, stats), want, bounds):
        within(g[dev], w, e, what)
    gl, ge = vector(rng, n, 1.0 / n), vector(rng, n, 0.1 / n)
    dx, dt, db, _ = saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, gl, ge, b)
    pick = lambda t: exact(t[dev])  # noqa: E731
    bx = None if b is None else exact(b)
    want, bounds = R.loss_grad(pick(x), exact(table), bx, pick(tgt), pick(stats), pick(H), pick(gl), pick(ge),
                               dtype)
    if dtype == "f16":  # (the scale goes by all rows' gradients)
        most = float((gl.abs() + 17 * ge.abs()).max())
        bounds = (bounds[0] + 2.0 ** -38 * most * np.abs(exact(table)).sum(axis=0), *bounds[1:])
    within(dx[dev], want[0], bounds[0], "d_x")
    want, bounds = R.loss_grad(exact(x), exact(table[dcls]), None if b is None else bx[cls], local,
                               exact(stats), exact(H), exact(gl), exact(ge), dtype)
    within(dt[dcls], want[1], bounds[1], "d_table")
    if b is not None:
        within(db[dcls], want[2], bounds[2], "d_bias")


def test_rows_in_several_launches():
    """More rows than the sums of one launch's slices are kept for, checked on
    rows on both sides of the cut (at a multiple of 256 below 22000) and at the
    ends."""
    rng = np.random.default_rng(4)
    n, d, v = 23000, 8, 131072
    x, table, b = head(rng, n, d, v, "bf16", "plain")
    tgt = classes(rng, n, v)
    tgt[n - 2] = v
    got = saa.seacells_linear_logprobs(x, table, tgt, b)
    assert flags(got[3]) == ["BAD_INDEX"] and got[0][n - 2] == 0
    at = np.unique(np.concatenate([[0, 1, n - 2, n - 1], np.arange(20480, 22017, 256),
                                   np.arange(20480, 22017, 256) - 1]))
    dev = torch.from_numpy(at).cuda()
    want, bounds = R.loss(exact(x[dev]), exact(table), exact(b), exact(tgt[dev]), "bf16")
    for what, g, w, e in zip(("logp", "entropy", "stats"), got, want, bounds):
        within(g[dev], w, e, what)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gap,start", [(0, 1), (5, 0), (8, 8), (3, 7), (2 ** 22, 0)])
def test_even_widths_at_any_stride_and_start(dtype, gap, start):
    """Widths of whole chunks in rows that start anywhere: the same bits as in
    plain matrices."""
    rng = np.random.default_rng(11)
    n, d, f, m, v = 70, 64, 128, 72, 200

    def moved(t):
        base = torch.full((start + t.shape[0] * (t.shape[1] + gap) + 8,), float("nan"), dtype=t.dtype,
                          device="cuda")
        out = base[start:start + t.shape[0] * (t.shape[1] + gap)].view(t.shape[0], -1)[:, :t.shape[1]]
        return out.copy_(t)

    x, w_in, w_out = block(rng, n, d, f, m, dtype)
    if gap > 100:  # (one operand with rows 2^22 apart is enough memory)
        a = saa.seacells_gated_ffn(x, w_in, w_out)
        b = saa.seacells_gated_ffn(moved(x[:65].contiguous()), w_in, w_out)
        assert torch.equal(a[0][:65], b[0]) and torch.equal(a[1][:65], b[1])
        return
    a = saa.seacells_gated_ffn(x, w_in, w_out)
    b = saa.seacells_gated_ffn(moved(x), moved(w_in), moved(w_out))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dy = rows(rng, n, m, dtype)
    for p, q in zip(saa.seacells_gated_ffn_grad(dy, x, a[1], w_in, w_out),
                    saa.seacells_gated_ffn_grad(moved(dy), moved(x), moved(a[1]), moved(w_in),
                                                moved(w_out))):
        assert torch.equal(p, q)
    table, tgt = rows(rng, v, d, dtype), classes(rng, n, v)
    a = saa.seacells_linear_logprobs(x, table, tgt)
    b = saa.seacells_linear_logprobs(moved(x), moved(table), tgt)
    one = torch.ones(n, device="cuda")
    g = saa.seacells_linear_logprobs_grad(x, table, tgt, a[2], a[1], one, one)
    h = saa.seacells_linear_logprobs_grad(moved(x), moved(table), tgt, b[2], b[1], one, one)
    for p, q in zip(a[:3] + g[:2], b[:3] + h[:2]):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d", [(5, 24), (5, 23), (150, 24), (150, 23)])
def test_workspaces_are_as_large_as_the_queries_say(n, d, dtype):
    """Calls with exactly the bytes of the queries, between marks that stay; one
    byte less is refused."""
    rng = np.random.default_rng(n + d)
    f, m, v, dt = 40, d, 70, DT[dtype]
    x, w_in, w_out = block(rng, n, d, f, m, dtype)
    table, tgt, dy = rows(rng, v, d, dtype), classes(rng, n, v), rows(rng, n, m, dtype)
    b, one = vector(rng, v), torch.ones(n, device="cuda")
    y, pre = saa.seacells_gated_ffn(x, w_in, w_out)
    _, H, stats, _ = saa.seacells_linear_logprobs(x, table, tgt, b)
    for query, sizes, go in (
            (saa.seacells_gated_ffn_workspace, (n, d, f, m),
             lambda ws: saa.seacells_gated_ffn(x, w_in, w_out, workspace=ws)),
            (saa.seacells_gated_ffn_grad_workspace, (n, d, f, m),
             lambda ws: saa.seacells_gated_ffn_grad(dy, x, pre, w_in, w_out, workspace=ws)),
            (saa.seacells_linear_logprobs_workspace, (n, d, v),
             lambda ws: saa.seacells_linear_logprobs(x, table, tgt, b, workspace=ws)),
            (saa.seacells_linear_logprobs_grad_workspace, (n, d, v),
             lambda ws: saa.seacells_linear_logprobs_grad(x, table, tgt, stats, H, one, one, b,
                                                          workspace=ws))):
        want = [t for t in go(None) if t is not None]
        for on_16 in ((True, False) if d % 8 == 0 else (False,)):
            size = query(dt, *sizes, on_16_bytes=on_16)
            base = torch.full((size + 512,), 0x5A, dtype=torch.uint8, device="cuda")
            got = [t for t in go(base[256:256 + size]) if t is not None]
            assert all(torch.equal(p, q) for p, q in zip(want, got))
            assert bool((base[:256] == 0x5A).all()) and bool((base[256 + size:] == 0x5A).all())
        # (these operands start on 16 bytes; those whose rows do not are copied either way)
        least = query(dt, *sizes, on_16_bytes=True)
        with pytest.raises(saa.SeacellsError):
            go(torch.empty(least - 1, dtype=torch.uint8, device="cuda"))


# --- together, streams, graphs, refusals -------------------------------------------

def model_step(s):
    """A training step of a model of one block: embed, norm, block, residual by
    the caller, head and loss, and all the way back. The outputs."""
    kw = dict(stream=s.get("stream"))
    x, _ = saa.seacells_embed(s["table"], s["tok"], 2.0, **kw)
    h, mean, rstd = saa.seacells_layer_norm(x, s["w"], s["b"], **kw)
    y, pre = saa.seacells_gated_ffn(h, s["w_in"], s["w_out"], "silu", **kw)
    logp, H, stats, _ = saa.seacells_linear_logprobs(y, s["head"], s["tgt"], s["bias"], **kw)
    dy, dhead, dbias, _ = saa.seacells_linear_logprobs_grad(y, s["head"], s["tgt"], stats, H, s["one"],
                                                            s["one"], s["bias"], **kw)
    dh, di, do = saa.seacells_gated_ffn_grad(dy, h, pre, s["w_in"], s["w_out"], "silu", **kw)
    dx, dw, db = saa.seacells_layer_norm_grad(dh, x, mean, rstd, s["w"], **kw)
    dt, _ = saa.seacells_embed_grad(s["tok"], dx, 50, 2.0, **kw)
    return [x, h, mean, rstd, y, pre, logp, H, stats, dy, dhead, dbias, dh, di, do, dx, dw, db, dt]


def model_state(n, dtype, seed=1, d=96, f=200, v=300):
    rng = np.random.default_rng(seed)
    tok = torch.from_numpy(rng.integers(0, 50, n).astype(np.int32)).cuda()
    return dict(table=rows(rng, 50, d, dtype), tok=tok, w=1 + rows(rng, 1, d, dtype)[0] / 4,
                b=rows(rng, 1, d, dtype)[0] / 4, w_in=rows(rng, 2 * f, d, dtype, d ** -0.5),
                w_out=rows(rng, d, f, dtype, f ** -0.5), head=rows(rng, v, d, dtype, 2 * d ** -0.5),
                bias=vector(rng, v), tgt=classes(rng, n, v), one=torch.full((n,), 1.0 / n, device="cuda"))


@pytest.mark.parametrize("n", [1, 40, 700])
def test_a_model_step_gives_autograds_gradients(n):
    """The operators in a row against 64-bit autograd of the formulas (f32)."""
    s = model_state(n, "f32")
    got = dict(zip("x h mean rstd y pre logp H stats dy dhead dbias dh di do dx dw db dt".split(),
                   model_step(s)))
    p = {k: s[k].cpu().double().requires_grad_() for k in ("table", "w", "b", "w_in", "w_out", "head",
                                                           "bias")}
    x = p["table"][s["tok"].cpu().long()] * 2.0
    c = x - x.mean(dim=1, keepdim=True)
    h = c / (c.square().mean(dim=1, keepdim=True) + float(np.float32(1e-5))).sqrt() * p["w"] + p["b"]
    g, u = (h @ p["w_in"].t()).chunk(2, dim=1)
    y = (g * torch.sigmoid(g) * u) @ p["w_out"].t()
    lp = (y @ p["head"].t() + p["bias"]).log_softmax(dim=1)
    t = s["tgt"].cpu().long()
    logp = torch.where(t >= 0, lp.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    H = -(lp.exp() * lp).sum(dim=1)
    ((logp + H) / n).sum().backward()
    # a chain of eight operators, each a few dozen roundings of values near the largest
    for name, want in (("logp", logp), ("H", H), ("dt", p["table"].grad), ("dw", p["w"].grad),
                       ("db", p["b"].grad), ("di", p["w_in"].grad), ("do", p["w_out"].grad),
                       ("dhead", p["head"].grad), ("dbias", p["bias"].grad)):
        w = want.detach()
        assert float((got[name].cpu().double() - w).abs().max()) <= 2e-5 * float(w.abs().max()), name


def test_block_and_loss_on_another_stream():
    for dtype in TYPES:
        s = model_state(500, dtype)
        want = model_step(s)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = model_step(dict(s, stream=side))
        with torch.cuda.stream(side):
            got2 = model_step(s)
        side.synchronize()
        for a, b, c in zip(want, got, got2):
            assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [3, 900])
def test_block_and_loss_in_a_graph(n, dtype):
    s = model_state(n, dtype)
    model_step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = model_step(s)
    for seed in (2, 3, 4):
        for k, t in model_state(n, dtype, seed=seed).items():
            s[k].copy_(t)
        want = model_step(s)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_two_calls_at_once():
    """Two streams, each with its own workspace, over the same weights."""
    s = model_state(900, "bf16")
    s2 = dict(model_state(900, "bf16", seed=5), **{k: s[k] for k in ("w_in", "w_out", "head", "bias")})
    want, want2 = model_step(s), model_step(s2)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(4):
        with torch.cuda.stream(a):
            outs.append((model_step(s), want))
        with torch.cuda.stream(b):
            outs.append((model_step(s2), want2))
    torch.cuda.synchronize()
    for got, ref in outs:
        for p, q in zip(got, ref):
            assert torch.equal(p, q)


def test_two_graphs_of_one_workspace():
    """Graphs that share a workspace and run one after the other."""
    rng = np.random.default_rng(2)
    x, w_in, w_out = block(rng, 300, 96, 200, 64, "bf16")
    x2 = rows(rng, 40, 96, "bf16")
    ws = torch.empty(saa.seacells_gated_ffn_workspace(torch.bfloat16, 300, 96, 200, 64), dtype=torch.uint8,
                     device="cuda")
    want = [saa.seacells_gated_ffn(t, w_in, w_out)[0] for t in (x, x2)]
    graphs, outs = [], []
    for t in (x, x2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(saa.seacells_gated_ffn(t, w_in, w_out, workspace=ws)[0])
        graphs.append(g)
    for _ in range(3):
        for g, o, w in zip(graphs, outs, want):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, w)


def test_the_same_call_gives_the_same_bits():
    s = model_state(900, "bf16")
    first = model_step(s)
    for _ in range(3):
        for a, b in zip(first, model_step(s)):
            assert torch.equal(a, b)


def test_binding_refuses_wrong_block_operands():
    x, wi, wo = (torch.zeros(s, device="cuda") for s in ((4, 8), (12, 8), (5, 6)))
    pre, dy = torch.zeros(4, 12, device="cuda"), torch.zeros(4, 5, device="cuda")
    tab, t = torch.zeros(9, 8, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    st, f = torch.zeros(4, 2, device="cuda"), torch.zeros(4, device="cuda")
    for go in (
            lambda: saa.seacells_gated_ffn(x, wi, wo, "tanh"),
            lambda: saa.seacells_gated_ffn(x, wi[:10], wo),
            lambda: saa.seacells_gated_ffn(x, wi.half(), wo),
            lambda: saa.seacells_gated_ffn(x, wi, wo.half()),
            lambda: saa.seacells_gated_ffn(x.double(), wi, wo),
            lambda: saa.seacells_gated_ffn(x, wi[:, :7], wo),
            lambda: saa.seacells_gated_ffn(x, wi.t().contiguous().t(), wo),
            lambda: saa.seacells_gated_ffn(x, wi.cpu(), wo),
            lambda: saa.seacells_gated_ffn(x, wi, wo, out=torch.empty(4, 6, device="cuda")),
            lambda: saa.seacells_gated_ffn(x, wi, wo, pre=torch.empty(4, 11, device="cuda")),
            lambda: saa.seacells_gated_ffn(x, wi, wo, workspace=torch.empty(8, device="cuda")),
            lambda: saa.seacells_gated_ffn_grad(dy[:, :4], x, pre, wi, wo),
            lambda: saa.seacells_gated_ffn_grad(dy[:3], x, pre, wi, wo),
            lambda: saa.seacells_gated_ffn_grad(dy, x, pre[:, :11], wi, wo),
            lambda: saa.seacells_gated_ffn_grad(dy, x, pre.half(), wi, wo),
            lambda: saa.seacells_gated_ffn_grad(dy, x, pre, wi, wo, d_w_in=torch.empty(6, 8, device="cuda")),
            lambda: saa.seacells_gated_ffn_grad(dy, x, pre, wi, wo, workspace=torch.empty(8, device="cuda")),
            lambda: saa.seacells_linear_logprobs(x, tab[:, :7], t),
            lambda: saa.seacells_linear_logprobs(x, tab.half(), t),
            lambda: saa.seacells_linear_logprobs(x, tab, t.long()),
            lambda: saa.seacells_linear_logprobs(x, tab, t[:3]),
            lambda: saa.seacells_linear_logprobs(x, tab, t, f),
            lambda: saa.seacells_linear_logprobs(x, tab, t, torch.zeros(9, device="cuda").half()),
            lambda: saa.seacells_linear_logprobs(x, tab, t, stats=f),
            lambda: saa.seacells_linear_logprobs(x, tab, t, workspace=torch.empty(8, device="cuda")),
            lambda: saa.seacells_linear_logprobs_grad(x, tab, t, f),
            lambda: saa.seacells_linear_logprobs_grad(x, tab, t, st, d_entropy=f),
            lambda: saa.seacells_linear_logprobs_grad(x, tab, t, st, d_x=torch.empty(4, 9, device="cuda")),
            lambda: saa.seacells_linear_logprobs_grad(x, tab, t, st, d_bias=f)):
        with pytest.raises(saa.SeacellsError):
            go()
