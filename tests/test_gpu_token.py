"""The token operators (include/seacells_token.h) against their 64-bit forms
(tests/token_reference.py), element by element within the bounds derived
there: sizes from one element to several thousand, odd widths, row strides
and starts at any element, masks, ties, empty and lost rows, in-place use,
offsets past 2^32 bytes, side streams and graph replays."""
import math

import numpy as np
import pytest
import torch

import sparse_archetypal_analysis_amd as saa
from tests import token_reference as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TYPES = list(DT)
INF = math.inf


def exact(t):
    """A device tensor's exact values as float64 / int64."""
    t = t.detach().cpu()
    return t.double().numpy() if t.is_floating_point() else t.long().numpy()


def within(got, want, bound, what):
    got = exact(got).reshape(np.shape(want))
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    far = ~fin & ~np.isnan(want)
    assert np.array_equal(got[far], want[far]), what
    off = np.abs(got[fin] - want[fin]) - bound[fin]
    assert off.size == 0 or off.max() <= 0, "%s: %.3g over its bound of %.3g" % (
        what, off.max(), bound[fin][off.argmax()])


def rows(rng, n, d, dtype, scale=1.0, gap=0, start=0):
    """[n, d] normal values in a buffer whose rows start at any element."""
    base = torch.full((start + n * (d + gap) + 16,), float("nan"), dtype=DT[dtype], device="cuda")
    out = base[start:start + n * (d + gap)].view(n, d + gap)[:, :d]
    out.copy_(torch.from_numpy(scale * rng.normal(size=(n, d))))
    return out


def blank(n, d, dtype, gap=0, start=0):
    """An output whose surroundings must keep their value."""
    base = torch.full((start + n * (d + gap) + 16,), 7.0, dtype=DT[dtype], device="cuda")
    return base, base[start:start + n * (d + gap)].view(n, d + gap)[:, :d]


def untouched(base, out):
    n, d = out.shape
    mark = torch.ones_like(base, dtype=torch.bool)
    mark[out.storage_offset():].as_strided(out.shape, out.stride()).fill_(False)
    assert bool((base[mark] == 7.0).all())


def ids(rng, n, v, pad=0.1, heavy=0.3):
    t = rng.integers(0, v, n)
    t[rng.random(n) < heavy] = v // 2
    t[rng.random(n) < pad] = -1 - int(rng.integers(0, 5))
    return torch.from_numpy(t.astype(np.int32)).cuda()


def flags(status):
    return saa.status_flags(status)


# --- embedding ----------------------------------------------------------------

EMBED_SIZES = [(1, 1, 1), (3, 2, 5), (32, 100, 256), (257, 7, 25), (64, 33, 1003), (19, 1300, 64),
               (5, 3, 4099), (2000, 50, 8), (40000, 9, 3), (2, 5, 20000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", EMBED_SIZES)
def test_embed(n, v, d, dtype):
    rng = np.random.default_rng(n + v + d)
    gap, start = (0, 0) if d % 2 == 0 else (3, 1)
    table, tok = rows(rng, v, d, dtype, gap=gap, start=start), ids(rng, n, v)
    base, out = blank(n, d, dtype, gap=gap, start=start)
    scale = float(np.float32(math.sqrt(d)))
    got, st = saa.seacells_embed(table, tok, scale, out=out)
    assert got is out and flags(st) == []
    want, bound = R.embed(exact(table), exact(tok), scale, dtype)
    within(out, want, bound, "out")
    untouched(base, out)


def test_embed_flags_ids_beyond_the_table():
    rng = np.random.default_rng(0)
    table = rows(rng, 10, 8, "f32")
    for n in (5, 40000):
        tok = ids(rng, n, 10)
        st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        saa.seacells_embed(table, tok, status=st)
        assert flags(st) == []
        tok[n - 2] = 10
        out, _ = saa.seacells_embed(table, tok, status=st)
        assert flags(st) == ["BAD_INDEX"]
        want, bound = R.embed(exact(table), exact(tok), 1.0, "f32")
        within(out, want, bound, "out")


def test_embed_takes_tokens_of_any_shape_and_none():
    rng = np.random.default_rng(0)
    table = rows(rng, 10, 8, "bf16")
    out, _ = saa.seacells_embed(table, ids(rng, 12, 10).view(3, 4))
    assert out.shape == (3, 4, 8)
    out, st = saa.seacells_embed(table, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 8) and flags(st) == []


GRAD_SIZES = [(1, 1, 1), (4, 3, 5), (50, 1300, 64), (300, 7, 25), (1000, 257, 100),
              (5000, 600, 33), (3000, 2, 130), (700, 5, 1003), (9, 4, 5000), (20, 3000, 2),
              (70000, 40, 3), (130, 300000, 1), (2500, 1, 260)]


@pytest.mark.parametrize("dtype,out_dtype,add", [
    ("f32", "f32", None), ("bf16", "f32", "other"), ("bf16", "bf16", "same"),
    ("f16", "f16", "other"), ("f16", "f32", None), ("f32", "f32", "same")])
@pytest.mark.parametrize("n,v,d", GRAD_SIZES)
def test_embed_grad(n, v, d, dtype, out_dtype, add):
    rng = np.random.default_rng(n + v + d)
    gap, start = (0, 0) if d % 2 == 0 else (3, 1)
    tok = ids(rng, n, v)
    d_out = rows(rng, n, d, dtype, gap=gap, start=start)
    base, out = blank(v, d, out_dtype, gap=gap, start=start)
    so_far = None
    if add is not None:
        so_far = rows(rng, v, d, out_dtype, gap=gap, start=start)
        if add == "same":
            out.copy_(so_far)
            so_far = out
    before = exact(so_far) if add else None
    scale = float(np.float32(1.7))
    got, st = saa.seacells_embed_grad(tok, d_out, v, scale, add_to=so_far, d_table=out)
    assert got is out and flags(st) == []
    want, bound = R.embed_grad(exact(tok), exact(d_out), v, scale, before, out_dtype)
    within(out, want, bound, "d_table")
    untouched(base, out)


@pytest.mark.parametrize("n,v,d", [(2047, 900, 5), (2048, 300, 9), (2049, 300, 9), (33000, 513, 2),
                                   (100000, 5000, 7), (600000, 3000, 1), (600000, 5, 1),
                                   (40000, 1200000, 1), (30000, 1, 515), (20000, 9, 1031)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_embed_grad_of_many_tokens_and_ids(n, v, d, dtype):
    """Sizes around the steps of the sort: tokens read by the buckets or by
    chunks, chunks beyond a block's threads, several ranges of ids per bucket,
    ids that cross many windows."""
    rng = np.random.default_rng(n + v + d)
    tok, d_out = ids(rng, n, v), rows(rng, n, d, dtype, gap=1, start=1)
    base, out = blank(v, d, "f32", gap=1, start=1)
    _, st = saa.seacells_embed_grad(tok, d_out, v, d_table=out)
    assert flags(st) == []
    want, bound = R.embed_grad(exact(tok), exact(d_out), v, 1.0, None, "f32")
    within(out, want, bound, "d_table")
    untouched(base, out)
    tok[n // 2] = v
    assert flags(saa.seacells_embed_grad(tok, d_out, v, d_table=out)[1]) == ["BAD_INDEX"]


@pytest.mark.parametrize("n", [4096, 4097, 8192, 16383, 16384])
@pytest.mark.parametrize("v", [523776, 523777, 524288, 524289, 1047552, 1048576])
def test_embed_grad_where_the_buckets_meet_their_counters(n, v):
    """Tables around the largest number of buckets, with tokens in the last
    ones, for token counts with and without chunks and a frequent id's bucket;
    a workspace that an earlier call left full."""
    p = saa.seacells_debug_embed_plan(n, v, 2)
    assert p["chunks"] == 0 or p["buckets"] < p["counters"]
    rng = np.random.default_rng(n + v)
    tok = ids(rng, n, v)
    tok[: n // 4] = torch.from_numpy(rng.integers(v - 2000, v, n // 4).astype(np.int32)).cuda()
    tok[n // 2], tok[0] = v - 1, 0
    d_out = rows(rng, n, 2, "bf16", gap=1, start=1)
    base, out = blank(v, 2, "f32", gap=1, start=1)
    ws = torch.full((saa.seacells_embed_grad_workspace(n, v, 2),), 255, dtype=torch.uint8,
                    device="cuda")
    _, st = saa.seacells_embed_grad(tok, d_out, v, d_table=out, workspace=ws)
    assert flags(st) == []
    want, bound = R.embed_grad(exact(tok), exact(d_out), v, 1.0, None, "f32")
    within(out, want, bound, "d_table")
    untouched(base, out)
    tok[n - 1] = v
    assert flags(saa.seacells_embed_grad(tok, d_out, v, d_table=out, workspace=ws)[1]) == [
        "BAD_INDEX"]


@pytest.mark.parametrize("n", [1, 2, 63, 255, 256, 257])
@pytest.mark.parametrize("v,d", [(1, 3), (15, 1031), (16, 8), (17, 2049), (900, 64), (5001, 20),
                                 (262144, 1), (4200000, 1)])
@pytest.mark.parametrize("spread", ["even", "one", "two", "beside"])
def test_embed_grad_of_few_tokens(n, v, d, spread):
    """The sizes that take one launch and the first that do not; tokens spread,
    on one id, on two, on neighbouring ids; with and without add_to, in place."""
    rng = np.random.default_rng(n + v + d)
    t = {"even": rng.integers(-1, v, n), "one": np.full(n, v - 1),
         "two": np.where(rng.random(n) < 0.5, 0, v // 2),
         "beside": np.arange(n) % min(v, 96)}[spread]
    tok = torch.from_numpy(t.astype(np.int32)).cuda()
    d_out = rows(rng, n, d, "bf16", gap=1, start=1)
    base, out = blank(v, d, "f32", gap=2, start=3)
    before = rows(rng, v, d, "f32", gap=2)
    for add in (None, before):
        _, st = saa.seacells_embed_grad(tok, d_out, v, 0.5, add_to=add, d_table=out)
        assert flags(st) == []
        want, bound = R.embed_grad(exact(tok), exact(d_out), v, 0.5,
                                   None if add is None else exact(add), "f32")
        within(out, want, bound, "d_table")
        untouched(base, out)
    again = out.clone()
    saa.seacells_embed_grad(tok, d_out, v, 0.5, add_to=before, d_table=before)
    assert torch.equal(before, again)
    tok[n // 2] = v
    assert flags(saa.seacells_embed_grad(tok, d_out, v, d_table=out)[1]) == ["BAD_INDEX"]


@pytest.mark.parametrize("n,v", [(16383, 3000), (16384, 3000), (20001, 512), (50000, 262144),
                                 (50000, 261889), (300001, 40000), (600001, 700)])
@pytest.mark.parametrize("often", ["first", "second", "last", "middle", "two", "none", "all"])
def test_embed_grad_of_frequent_ids(n, v, often):
    """Ids that many tokens share, at the ends of the table and of the buckets
    that the sort forms, beside other ids and without any."""
    rng = np.random.default_rng(n + v)
    t = rng.integers(-1, v, n)
    id = {"first": 0, "second": 1, "last": v - 1}.get(often, v // 2)
    if often == "all":
        t[:] = id
    elif often != "none":
        t[rng.random(n) < 0.4] = id
        t[rng.random(n) < 0.05] = max(id - 1, 0)
        t[rng.random(n) < 0.05] = min(id + 1, v - 1)
    if often == "two":
        t[rng.random(n) < 0.4] = id // 2
    tok = torch.from_numpy(t.astype(np.int32)).cuda()
    d_out = rows(rng, n, 2, "f32")
    got, st = saa.seacells_embed_grad(tok, d_out, v)
    assert flags(st) == []
    want, bound = R.embed_grad(exact(tok), exact(d_out), v, 1.0, None, "f32")
    within(got, want, bound, "d_table")
    assert torch.equal(saa.seacells_embed_grad(tok, d_out, v)[0], got)
    tok[-1] = v
    assert flags(saa.seacells_embed_grad(tok, d_out, v)[1]) == ["BAD_INDEX"]


@pytest.mark.parametrize("n", [4095, 4096, 4097, 131071, 131500])
@pytest.mark.parametrize("v,d", [(1, 9), (31, 3), (3000, 17), (70001, 2)])
def test_embed_grad_around_the_steps_of_its_sort(n, v, d):
    """The last direct size and the first by chunks; runs of one batch per wave
    and longer ones; a bucket that holds nearly all the tokens."""
    rng = np.random.default_rng(3 * n + v)
    tok, d_out = ids(rng, n, v), rows(rng, n, d, "f32")
    tok[rng.permutation(n)[:n - n // 8]] = v // 2
    got, st = saa.seacells_embed_grad(tok, d_out, v)
    assert flags(st) == []
    want, bound = R.embed_grad(exact(tok), exact(d_out), v, 1.0, None, "f32")
    within(got, want, bound, "d_table")
    assert torch.equal(saa.seacells_embed_grad(tok, d_out, v)[0], got)


@pytest.mark.parametrize("n,v,d", [(5000, 600, 33), (9000, 3, 130), (70000, 40, 3)])
def test_embed_grad_is_the_same_every_time(n, v, d):
    rng = np.random.default_rng(1)
    tok, d_out = ids(rng, n, v), rows(rng, n, d, "f32")
    first, _ = saa.seacells_embed_grad(tok, d_out, v)
    for _ in range(3):
        again, _ = saa.seacells_embed_grad(tok, d_out, v)
        assert torch.equal(first, again)


def test_embed_grad_without_tokens_and_with_bad_ones():
    rng = np.random.default_rng(2)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    g, st = saa.seacells_embed_grad(none, torch.empty(0, 6, device="cuda"), 5)
    assert flags(st) == [] and g.shape == (5, 6) and not g.any()
    tok, d_out = ids(rng, 300, 5), rows(rng, 300, 6, "f32")
    tok[7] = 5
    tok[9] = 2 ** 31 - 1
    g, st = saa.seacells_embed_grad(tok, d_out, 5)
    assert flags(st) == ["BAD_INDEX"]
    want, bound = R.embed_grad(exact(tok), exact(d_out), 5, 1.0, None, "f32")
    within(g, want, bound, "d_table")
    tok[:] = -1
    g, st = saa.seacells_embed_grad(tok, d_out, 5)
    assert flags(st) == [] and not g.any()


def test_embed_rows_beyond_4_gib():
    # two rows of a table, of an output and of a gradient, 2^31 + 5 elements apart
    far = 2 ** 31 + 5
    base = torch.empty(far + 64, dtype=torch.bfloat16, device="cuda")
    table = base.as_strided((2, 20), (far, 1))
    table.copy_(torch.arange(40, device="cuda").view(2, 20))
    tok = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
    out, _ = saa.seacells_embed(table, tok)
    assert torch.equal(out, table[tok.long()])
    saa.seacells_embed(out, tok[:2], 2.0, out=table)
    assert torch.equal(table, 2 * out[tok[:2].long()])
    table.copy_(torch.arange(40, device="cuda").view(2, 20))
    g, _ = saa.seacells_embed_grad(tok[:2], table, 3)
    assert torch.equal(g[:2], table[[1, 0]]) and not g[2].any()
    saa.seacells_embed_grad(tok[:2], out[:2], 2, d_table=table)
    assert torch.equal(table, out[[1, 0]])


# --- layer norm ---------------------------------------------------------------

NORM_SIZES = [(1, 1), (3, 2), (7, 5), (5, 16), (33, 25), (100, 64), (9, 100), (64, 256), (5, 511),
              (17, 1003), (3, 1024), (4, 2048), (2, 4099), (3, 8192), (1, 16384), (2, 40001),
              (700, 130), (1, 300000)]


def norm_input(rng, n, d, dtype, **kw):
    x = rows(rng, n, d, dtype, **kw)
    x.mul_(torch.from_numpy(np.exp(rng.normal(size=(n, 1)))).to(x))
    x.add_(torch.from_numpy(3 * rng.normal(size=(n, 1))).to(x))
    return x


@pytest.mark.parametrize("dtype,w_dtype", [("f32", "f32"), ("f16", "f16"), ("bf16", "f32"),
                                           ("bf16", "bf16"), ("f16", None)])
@pytest.mark.parametrize("n,d", NORM_SIZES)
def test_layer_norm(n, d, dtype, w_dtype):
    rng = np.random.default_rng(n + d)
    gap, start = (0, 0) if d % 2 == 0 else (3, 1)
    x = norm_input(rng, n, d, dtype, gap=gap, start=start)
    w = b = None
    we, be = np.ones(d), np.zeros(d)
    if w_dtype:
        w, b = (rows(rng, 1, d, w_dtype)[0] for _ in range(2))
        we, be = exact(w), exact(b)
    base, out = blank(n, d, dtype, gap=gap, start=start)
    eps = float(np.float32(1e-5))
    _, mean, rstd = saa.seacells_layer_norm(x, w, b, eps, out=out)
    want, bound = R.layer_norm(exact(x), we, be, eps, dtype)
    for nm, g, y, e in zip(("out", "mean", "rstd"), (out, mean, rstd), want, bound):
        within(g, y, e, nm)
    untouched(base, out)
    # in place, and one of the two vectors alone
    _, m2, _ = saa.seacells_layer_norm(x, None, b, eps, out=x)
    assert torch.equal(m2, mean)
    if w_dtype is None:
        assert torch.equal(x, out)


@pytest.mark.parametrize("dtype,w_dtype", [("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("n,d", [(140001, 9), (20001, 301), (5001, 1500), (1501, 8201)])
def test_layer_norm_of_more_rows_than_a_launch_holds(n, d, dtype, w_dtype):
    rng = np.random.default_rng(n + d)
    x = norm_input(rng, n, d, dtype, gap=1)
    w, b = (rows(rng, 1, d, w_dtype)[0] for _ in range(2))
    eps = float(np.float32(1e-5))
    got = saa.seacells_layer_norm(x, w, b, eps)
    want, bound = R.layer_norm(exact(x), exact(w), exact(b), eps, dtype)
    for nm, g, y, e in zip(("out", "mean", "rstd"), got, want, bound):
        within(g, y, e, nm)


@pytest.mark.parametrize("dtype,w_dtype", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16"),
                                           ("bf16", None)])
@pytest.mark.parametrize("n,d", NORM_SIZES + [(5000, 40), (3001, 333)])
def test_layer_norm_grad(n, d, dtype, w_dtype):
    rng = np.random.default_rng(n + d)
    gap, start = (0, 0) if d % 2 == 0 else (3, 1)
    x = norm_input(rng, n, d, dtype, gap=gap, start=start)
    dy = rows(rng, n, d, dtype, gap=gap, start=start)
    w = rows(rng, 1, d, w_dtype)[0] if w_dtype else None
    _, mean, rstd = saa.seacells_layer_norm(x)
    base, d_x = blank(n, d, dtype, gap=gap, start=start)
    _, d_w, d_b = saa.seacells_layer_norm_grad(dy, x, mean, rstd, w, d_x=d_x)
    want, bound = R.layer_norm_grad(exact(dy), exact(x), exact(mean), exact(rstd),
                                    exact(w) if w_dtype else np.ones(d), dtype, w_dtype or dtype)
    for nm, g, y, e in zip(("d_x", "d_weight", "d_bias"), (d_x, d_w, d_b), want, bound):
        within(g, y, e, nm)
    untouched(base, d_x)
    # any part alone, and in place of either input, gives the same bits
    assert torch.equal(saa.seacells_layer_norm_grad(dy, x, mean, rstd, w, d_weight=False,
                                                    d_bias=False)[0], d_x)
    none, d_w2, d_b2 = saa.seacells_layer_norm_grad(dy, x, mean, rstd, w, d_x=False)
    assert none is None and torch.equal(d_w2, d_w) and torch.equal(d_b2, d_b)
    x2 = x.clone()
    got, d_w3, none = saa.seacells_layer_norm_grad(dy, x2, mean, rstd, w, d_x=x2, d_bias=False)
    assert none is None and torch.equal(got, d_x) and torch.equal(d_w3, d_w)
    got, _, d_b3 = saa.seacells_layer_norm_grad(dy, x, mean, rstd, w, d_x=dy)
    assert torch.equal(got, d_x) and torch.equal(d_b3, d_b)


@pytest.mark.parametrize("d", [1, 25, 64, 1000, 5000, 70000])
def test_layer_norm_of_constant_rows(d):
    x = torch.full((3, d), 2.5, device="cuda")
    out, mean, rstd = saa.seacells_layer_norm(x)
    assert torch.equal(out, torch.zeros_like(x)) and bool((mean == 2.5).all())
    want = 1.0 / math.sqrt(float(np.float32(1e-5)))
    within(rstd, np.full(3, want), np.full(3, 4 * R.U * want), "rstd")


@pytest.mark.parametrize("d", [1, 3, 5, 32, 33, 64, 130, 700, 1003, 5000, 70000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_norm_grad_of_constant_rows_far_from_zero(d, dtype):
    """mean * rstd is past f32's range here, (x - mean) * rstd is 0: what a lane
    holds past the row's end must not count."""
    rng = np.random.default_rng(d)
    x = torch.full((40, d), 2.0 ** 121, dtype=DT[dtype], device="cuda")
    mean = torch.full((40,), 2.0 ** 121, device="cuda")
    rstd = torch.full((40,), 316.0, device="cuda")
    dy, w = rows(rng, 40, d, dtype), rows(rng, 1, d, "f32")[0]
    got = saa.seacells_layer_norm_grad(dy, x, mean, rstd, w)
    want, bound = R.layer_norm_grad(exact(dy), exact(x), exact(mean), exact(rstd), exact(w), dtype,
                                    "f32")
    for nm, g, y, e in zip(("d_x", "d_weight", "d_bias"), got, want, bound):
        within(g, y, e, nm)


@pytest.mark.parametrize("d", [5, 64, 700, 5000, 70000])
@pytest.mark.parametrize("dtype", TYPES)
def test_layer_norm_of_rows_that_hold_no_numbers(d, dtype):
    rng = np.random.default_rng(d)
    x = rows(rng, 4, d, dtype)
    want = saa.seacells_layer_norm(x)
    for bad in (float("nan"), INF, -INF):
        y = x.clone()
        y[1, d // 2] = bad
        out, mean, rstd = saa.seacells_layer_norm(y)
        assert bool(out[1].isnan().all()) and bool(rstd[1].isnan()) and not bool(mean[1].isfinite())
        keep = [0, 2, 3]
        for a, b in zip((out, mean, rstd), want):
            assert torch.equal(a[keep], b[keep])


def test_layer_norm_without_rows():
    x, f = torch.empty(0, 9, device="cuda"), torch.empty(0, device="cuda")
    assert saa.seacells_layer_norm(x)[0].shape == (0, 9)
    d_x, d_w, d_b = saa.seacells_layer_norm_grad(x, x, f, f)
    assert d_x.shape == (0, 9) and not d_w.any() and not d_b.any()


def test_layer_norm_rows_beyond_4_gib():
    far = 2 ** 31 + 3
    base = torch.empty(far + 512, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((2, 300), (far, 1))
    near = rows(np.random.default_rng(3), 2, 300, "bf16")
    x.copy_(near)
    out, mean, rstd = saa.seacells_layer_norm(x)
    want, m2, r2 = saa.seacells_layer_norm(near)
    assert torch.equal(out, want) and torch.equal(mean, m2) and torch.equal(rstd, r2)
    for a, b in zip(saa.seacells_layer_norm_grad(x, x, mean, rstd),
                    saa.seacells_layer_norm_grad(near, near, mean, rstd)):
        assert torch.equal(a, b)


# --- log probabilities --------------------------------------------------------

LOGP_SIZES = [(1, 1, 1), (3, 2, 5), (5, 25, 3), (200, 33, 8), (9, 64, 64), (7, 257, 20),
              (40, 1300, 5), (3, 2047, 64), (5, 4099, 16), (2, 10000, 0), (600, 700, 1),
              (4, 50001, 20), (1, 131072, 64), (300, 9001, 7)]


def logit_rows(rng, n, v, dtype, masks, gap=0, start=0):
    x = rows(rng, n, v, dtype, scale=3.0, gap=gap, start=start)
    if masks:
        x[torch.from_numpy(rng.random((n, v)) < 0.3).cuda()] = -INF
        x[torch.from_numpy(rng.random((n, v)) < 0.05).cuda()] = torch.finfo(DT[dtype]).min
        x[::4] = -INF
        if n > 1:
            x[1, 1:] = -INF
        if n > 2:
            x[2] = torch.finfo(DT[dtype]).min
    return x


def classes(rng, n, v):
    t = rng.integers(0, v, n)
    t[rng.random(n) < 0.2] = -3
    return torch.from_numpy(t.astype(np.int32)).cuda()


def check_logprobs(x, tgt, k):
    out = saa.seacells_logprobs(x, tgt, k)
    assert flags(out[5]) == []
    (lp, H, stats, idx, val), (e_lp, e_H, e_st, e_val) = R.logprobs(exact(x), exact(tgt), k)
    within(out[0], lp, e_lp, "logp")
    within(out[1], H, e_H, "entropy")
    within(out[2], stats, e_st, "stats")
    if k:
        assert np.array_equal(exact(out[3]).reshape(idx.shape), idx)
        within(out[4], val, e_val, "top_logp")
    return out


@pytest.mark.parametrize("masks", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,k", LOGP_SIZES)
def test_logprobs(n, v, k, dtype, masks):
    rng = np.random.default_rng(n + v + k)
    gap, start = (0, 0) if v % 2 == 0 else (5, 1)
    x = logit_rows(rng, n, v, dtype, masks, gap=gap, start=start)
    tgt = classes(rng, n, v)
    check_logprobs(x, tgt, k)
    # without targets, and what does not depend on them
    lp, H, stats, idx, val, _ = saa.seacells_logprobs(x, None, k)
    lp2, H2, stats2, idx2, val2, _ = saa.seacells_logprobs(x, tgt, k)
    assert lp is None and torch.equal(H, H2) and torch.equal(stats, stats2)
    assert k == 0 or (torch.equal(idx, idx2) and torch.equal(val, val2))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v,k", [(3, 2), (30, 40), (33, 0), (60, 3), (61, 30), (125, 5), (130, 0),
                                 (200, 4), (255, 9), (257, 2), (500, 1), (501, 3), (900, 1),
                                 (1001, 0)])
def test_logprobs_of_many_short_rows(v, k, dtype):
    """More rows than get a wave each: every spread of a row over lanes."""
    rng = np.random.default_rng(v + k)
    n, (gap, start) = 4103, ((0, 0) if v % 2 == 0 else (5, 1))
    x = logit_rows(rng, n, v, dtype, True, gap=gap, start=start)
    x[5, v // 2] = float("nan")
    x[6] = 1.0  # all equal
    x[7, : v // 2] = -INF
    check_logprobs(x, classes(rng, n, v), k)


@pytest.mark.parametrize("v", [6, 64, 1300, 20000, 131072])
@pytest.mark.parametrize("n", [2, 70])
def test_top_alternatives_of_ties_and_ordered_rows(n, v):
    rng = np.random.default_rng(v)
    k = min(64, v)
    base = torch.arange(v, device="cuda").float()
    kinds = {
        "all equal": torch.zeros(v, device="cuda"),
        "signed zeros": torch.where(base % 2 == 0, -0.0, 0.0),
        "few values": torch.from_numpy(rng.integers(0, 3, v)).cuda().float(),
        "ascending": base / v,
        "descending": -base / v,
        "one column in 256": torch.where(base % 256 == 5 % v, 1.0, 0.0),
        "one column in 8192": torch.where(base % 8192 == 3, 1.0 + base / v, 0.0),
        "a block": torch.where((base >= v // 3) & (base < v // 3 + 90), 2.0, 0.0),
        "ties in the last places": torch.where(base >= v - 40, 1.0, 0.0),
    }
    tgt = classes(rng, n, v)
    for name, row in kinds.items():
        print(name, flush=True)
        check_logprobs(row.expand(n, v).contiguous(), tgt, k)
        check_logprobs(row.expand(n, v).to(torch.bfloat16).contiguous(), tgt, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v", [(4, 40), (9, 3000), (5, 70000)])
def test_logprobs_of_rows_without_a_distribution(n, v, dtype):
    rng = np.random.default_rng(v)
    x = rows(rng, n, v, dtype)
    x[0, v - 1] = float("nan")
    x[1, 3] = INF
    x[2] = -INF
    x[3, :] = -INF
    x[3, 5] = float("nan")
    tgt = torch.full((n,), 7, dtype=torch.int32, device="cuda")
    tgt[1] = -1
    lp, H, stats, idx, val, _ = check_logprobs(x, tgt, 6)
    gl, ge = torch.ones(n, device="cuda"), torch.ones(n, device="cuda")
    g, _ = saa.seacells_logprobs_grad(x, tgt, stats, H, gl, ge)
    assert bool(g[[0, 1, 3]].isnan().all()) and not g[2].any()
    assert bool(g[4:].isfinite().all())


@pytest.mark.parametrize("big", [1e4, 3e38])
def test_logprobs_of_large_logits(big):
    rng = np.random.default_rng(5)
    x = rows(rng, 12, 5000, "f32") * 4
    x += big * torch.from_numpy(rng.choice([-1.0, 1.0], (12, 1))).cuda().float()
    x[3, :50] = -big
    x[4, 50:90] = big
    tgt = classes(rng, 12, 5000)
    check_logprobs(x, tgt, 9)


def test_logprobs_flags_classes_beyond_the_row():
    rng = np.random.default_rng(5)
    x, st = rows(rng, 20, 30, "f32"), saa.new_status()
    tgt = classes(rng, 20, 30)
    tgt[19] = 30
    lp = saa.seacells_logprobs(x, tgt, 0, status=st)[0]
    assert flags(st) == ["BAD_INDEX"] and lp[19] == 0
    _, H, stats = saa.seacells_logprobs(x, None)[:3]
    g, st = saa.seacells_logprobs_grad(x, tgt, stats, d_logp=torch.ones(20, device="cuda"))
    assert flags(st) == ["BAD_INDEX"] and not g[19].any()
    tgt[19] = 29
    assert flags(saa.seacells_logprobs(x, tgt, 0, status=st)[5]) == []


@pytest.mark.parametrize("n,d", [(5, 3), (32768, 2), (32769, 2), (33001, 151), (40003, 299),
                                 (33000, 300), (33003, 8200)])
@pytest.mark.parametrize("at", [0, 1, -2, -1])
def test_status_of_every_launch_that_reports_it(n, d, at):
    """Few and many ids, narrow and wide rows (one block looks over the ids, or
    the rows' lanes do), a wrong id at either end, statuses that an earlier
    call left set."""
    if d == 8200 and at not in (1, -1):
        pytest.skip("one end is enough for the large rows")
    x = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    tok = torch.zeros(n, dtype=torch.int32, device="cuda")
    bad = tok.clone()
    bad[at] = d
    table = torch.ones(d, d, dtype=torch.bfloat16, device="cuda")
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    for t in (tok, bad, tok):
        want = ["BAD_INDEX"] if t is bad else []
        if d < 8200:
            assert flags(saa.seacells_embed(table, t, status=st)[1]) == want
        _, H, stats = saa.seacells_logprobs(x, t, 0, status=st)[:3]
        assert flags(st) == want
        one = torch.ones(n, device="cuda")
        assert flags(saa.seacells_logprobs_grad(x, t, stats, d_logp=one, status=st)[1]) == want
    for t in (bad, None):  # set, then cleared without targets
        st.fill_(-1)
        stats = saa.seacells_logprobs(x, t, 0, status=st)[2]
        assert flags(st) == (["BAD_INDEX"] if t is bad else [])
        st.fill_(-1)
        one = torch.ones(n, device="cuda")
        saa.seacells_logprobs_grad(x, t, stats, d_logp=one if t is not None else None,
                                   entropy=H, d_entropy=one, status=st)
        assert flags(st) == (["BAD_INDEX"] if t is bad else [])


def test_logprobs_of_no_rows():
    x = torch.empty(0, 9, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    lp, H, stats, idx, val, st = saa.seacells_logprobs(x, none, 4)
    assert lp.shape == (0,) and idx.shape == (0, 4) and flags(st) == []
    g, st = saa.seacells_logprobs_grad(x, none, stats)
    assert g.shape == (0, 9) and flags(st) == []


@pytest.mark.parametrize("masks", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,k", LOGP_SIZES)
def test_logprobs_grad(n, v, k, dtype, masks):
    rng = np.random.default_rng(n + v + k)
    gap, start = (0, 0) if v % 2 == 0 else (5, 1)
    x = logit_rows(rng, n, v, dtype, masks, gap=gap, start=start)
    tgt = classes(rng, n, v)
    _, H, stats = saa.seacells_logprobs(x, None)[:3]
    gl, ge = (torch.from_numpy(rng.normal(size=n)).cuda().float() for _ in range(2))
    base, out = blank(n, v, dtype, gap=gap, start=start)
    _, st = saa.seacells_logprobs_grad(x, tgt, stats, H, gl, ge, d_logits=out)
    assert flags(st) == []
    a = (exact(x), exact(tgt), exact(stats), exact(H))
    want, bound = R.logprobs_grad(*a, exact(gl), exact(ge), dtype)
    within(out, want, bound, "d_logits")
    untouched(base, out)
    zero = np.zeros(n)
    want, bound = R.logprobs_grad(*a, exact(gl), zero, dtype)
    within(saa.seacells_logprobs_grad(x, tgt, stats, None, gl)[0], want, bound, "of logp")
    want, bound = R.logprobs_grad(*a, zero, exact(ge), dtype)
    within(saa.seacells_logprobs_grad(x, None, stats, H, gl, ge)[0], want, bound, "of entropy")
    saa.seacells_logprobs_grad(x, tgt, stats, H, gl, ge, d_logits=x)
    assert torch.equal(x, out)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_logits_get_no_gradient_from_infinite_ones(dtype):
    x = rows(np.random.default_rng(4), 3, 300, dtype)
    x[:, 7:90] = -INF
    x[2] = -INF
    tgt = torch.tensor([3, 8, 5], dtype=torch.int32, device="cuda")  # open, masked, empty row
    _, H, stats = saa.seacells_logprobs(x, None)[:3]
    for bad in (INF, float("nan")):
        gl = torch.full((3,), bad, device="cuda")
        g, _ = saa.seacells_logprobs_grad(x, tgt, stats, H, gl, gl)
        assert not g[:, 7:90].any() and not g[2].any()
        assert bool(g[:2, 100:].isnan().all() if bad != INF else (~g[:2, 100:].isfinite()).all())


def test_logprobs_rows_beyond_4_gib():
    far = 2 ** 31 + 7
    base = torch.empty(far + 4096, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((2, 3000), (far, 1))
    near = rows(np.random.default_rng(3), 2, 3000, "bf16")
    x.copy_(near)
    tgt = torch.tensor([5, 2999], dtype=torch.int32, device="cuda")
    a, b = saa.seacells_logprobs(x, tgt, 5), saa.seacells_logprobs(near, tgt, 5)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    one = torch.ones(2, device="cuda")
    want, _ = saa.seacells_logprobs_grad(near, tgt, a[2], a[1], one, one)
    saa.seacells_logprobs_grad(x, tgt, a[2], a[1], one, one, d_logits=x)
    assert torch.equal(x, want)


# --- streams, graphs, refusals -------------------------------------------------

def every_operator(s):
    """One pass through all of them on fixed inputs; the outputs."""
    kw = dict(stream=s.get("stream"))
    y, _ = saa.seacells_embed(s["table"], s["tok"], 2.0, **kw)
    h, mean, rstd = saa.seacells_layer_norm(y, s["w"], s["b"], **kw)
    lp, H, stats, idx, val, _ = saa.seacells_logprobs(h, s["tgt"], 4, **kw)
    g, _ = saa.seacells_logprobs_grad(h, s["tgt"], stats, H, s["one"], s["one"], **kw)
    dx, dw, db = saa.seacells_layer_norm_grad(g, y, mean, rstd, s["w"], **kw)
    dt, _ = saa.seacells_embed_grad(s["tok"], dx, 50, 2.0, **kw)
    return [y, h, mean, rstd, lp, H, stats, idx, val, g, dx, dw, db, dt]


def small_state(n=1500, d=700, seed=1):
    rng = np.random.default_rng(seed)
    return dict(table=rows(rng, 50, d, "f32"), tok=ids(rng, n, 50), w=rows(rng, 1, d, "f32")[0],
                b=rows(rng, 1, d, "f32")[0], tgt=classes(rng, n, d),
                one=torch.ones(n, device="cuda"))


def test_on_another_stream():
    s = small_state()
    want = every_operator(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = every_operator(dict(s, stream=side))
    with torch.cuda.stream(side):
        got2 = every_operator(s)
    side.synchronize()
    for a, b, c in zip(want, got, got2):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("n", [3, 1500])
def test_in_a_graph(n):
    s = small_state(n)
    every_operator(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = every_operator(s)
    for seed in (2, 3, 4):
        for k, t in small_state(n, seed=seed).items():
            s[k].copy_(t)
        want = every_operator(s)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_binding_refuses_wrong_operands():
    x = torch.zeros(4, 8, device="cuda")
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    f, st = torch.zeros(4, device="cuda"), torch.zeros(4, 2, device="cuda")
    for go in (
            lambda: saa.seacells_embed(x, t.long()),
            lambda: saa.seacells_embed(x.double(), t),
            lambda: saa.seacells_embed(x.t(), t),
            lambda: saa.seacells_embed(x, t, out=torch.empty(4, 9, device="cuda")),
            lambda: saa.seacells_embed(x[:, :4], t.cpu()),
            lambda: saa.seacells_embed(x[:1].expand(4, 8), t),
            lambda: saa.seacells_embed(x[:, :0], t),
            lambda: saa.seacells_embed_grad(t[:3], x, 5),
            lambda: saa.seacells_embed_grad(t, x, 5, d_table=torch.empty(5, 8, device="cuda").half()),
            lambda: saa.seacells_embed_grad(t, x, 5, add_to=torch.zeros(4, 8, device="cuda")),
            lambda: saa.seacells_embed_grad(t, x, 5, workspace=torch.empty(8, device="cuda")),
            lambda: saa.seacells_embed_grad(t, x, 0),
            lambda: saa.seacells_layer_norm(x, f),
            lambda: saa.seacells_layer_norm(x, torch.ones(8, device="cuda").half()),
            lambda: saa.seacells_layer_norm(x, eps=-1.0),
            lambda: saa.seacells_layer_norm(x, mean=f[:2]),
            lambda: saa.seacells_layer_norm_grad(x[:, :7], x, f, f),
            lambda: saa.seacells_layer_norm_grad(x, x, f.double(), f),
            lambda: saa.seacells_logprobs(x, t, 65),
            lambda: saa.seacells_logprobs(x, t[:2]),
            lambda: saa.seacells_logprobs(x, t, 2, top_idx=torch.empty(4, 3, device="cuda")),
            lambda: saa.seacells_logprobs_grad(x, t, f),
            lambda: saa.seacells_logprobs_grad(x, t, st, d_entropy=f),
            lambda: saa.seacells_logprobs_grad(x, t, st, d_logits=x[:, :4])):
        with pytest.raises(saa.SeacellsError):
            go()
