"""Refusals of the token operators (include/seacells_token.h): the C entry
points' host checks and the binding's, all before any GPU work."""
import pytest
import torch

import sparse_archetypal_analysis_amd as saa
from sparse_archetypal_analysis_amd import SeacellsError, native

NULL, SHAPE, WORKSPACE, TOO_LARGE, TYPE = -1, -2, -3, -4, -6
P, Q = 0x10000, 0x20000  # stand-ins for device addresses (never followed)


def call(fn, **base):
    """The entry point with the base arguments replaced by keyword."""
    entry = getattr(saa.load(), fn)
    names = list(base)

    def go(**kw):
        assert set(kw) <= set(names)
        return entry(*[kw.get(nm, base[nm]) for nm in names])
    return go


EMBED = dict(table=P, dtype=0, v=10, d=8, table_ld=8, tokens=P, n=4, scale=1.0, out=Q, out_ld=8,
             status=P, stream=None)
EMBED_GRAD = dict(tokens=P, n=4, d_out=P, d_out_type=2, d_out_ld=8, v=10, d=8, scale=1.0,
                  add_to=None, d_table=Q, d_table_type=2, d_table_ld=8, ws=P, ws_bytes=1 << 20,
                  status=P, stream=None)
NORM = dict(x=P, dtype=2, n=4, d=8, x_ld=8, weight=P, bias=P, weight_type=2, eps=1e-5, out=Q,
            out_ld=8, mean=P, rstd=P, stream=None)
NORM_GRAD = dict(d_out=P, d_out_ld=8, x=P, dtype=2, n=4, d=8, x_ld=8, mean=P, rstd=P, weight=P,
                 weight_type=2, d_x=Q, d_x_ld=8, d_weight=Q, d_bias=Q, ws=P, ws_bytes=1 << 26,
                 stream=None)
LOGP = dict(logits=P, dtype=2, n=4, v=8, ld=8, targets=P, top_k=3, logp=Q, entropy=Q, stats=Q,
            top_idx=Q, top_logp=Q, ws=P, ws_bytes=1 << 26, status=P, stream=None)
LOGP_GRAD = dict(logits=P, dtype=2, n=4, v=8, ld=8, targets=P, stats=P, entropy=P, d_logp=P,
                 d_entropy=P, d_logits=Q, d_ld=8, status=P, stream=None)

REFUSALS = [
    ("seacells_embed", EMBED, [
        (NULL, dict(table=None)), (NULL, dict(tokens=None)), (NULL, dict(out=None)),
        (NULL, dict(status=None)), (TYPE, dict(dtype=3)), (TYPE, dict(table=P + 2)),
        (TYPE, dict(out=Q + 1)), (TYPE, dict(tokens=P + 2)), (SHAPE, dict(v=0)),
        (SHAPE, dict(d=0)), (SHAPE, dict(table_ld=7)), (SHAPE, dict(out_ld=7)),
        (TOO_LARGE, dict(v=2 ** 31)), (TOO_LARGE, dict(n=2 ** 31)),
        (TOO_LARGE, dict(out_ld=2 ** 40)),
        (TOO_LARGE, dict(d=2 ** 23 + 1, table_ld=2 ** 24, out_ld=2 ** 24))]),
    ("seacells_embed_grad", EMBED_GRAD, [
        (NULL, dict(tokens=None)), (NULL, dict(d_out=None)), (NULL, dict(d_table=None)),
        (NULL, dict(status=None)), (TYPE, dict(d_out_type=9)), (TYPE, dict(d_table_type=1)),
        (TYPE, dict(d_out_type=0)), (TYPE, dict(d_out=P + 1)), (TYPE, dict(add_to=P + 1)),
        (TYPE, dict(d_table_type=0, d_table=Q + 2)), (SHAPE, dict(v=0)), (SHAPE, dict(d=0)),
        (SHAPE, dict(d_out_ld=4)), (SHAPE, dict(d_table_ld=4)), (WORKSPACE, dict(ws=None)),
        (WORKSPACE, dict(ws_bytes=8)), (WORKSPACE, dict(ws=P + 128)),
        (TOO_LARGE, dict(n=2 ** 31)), (TOO_LARGE, dict(v=2 ** 31))]),
    ("seacells_layer_norm", NORM, [
        (NULL, dict(x=None)), (NULL, dict(out=None)), (TYPE, dict(dtype=5)),
        (TYPE, dict(weight_type=1)), (TYPE, dict(x=P + 1)), (TYPE, dict(mean=P + 2)),
        (TYPE, dict(weight_type=0, weight=P + 2)), (SHAPE, dict(d=0)), (SHAPE, dict(x_ld=7)),
        (SHAPE, dict(eps=-1.0)), (SHAPE, dict(eps=float("nan"))), (SHAPE, dict(eps=float("inf"))),
        (TOO_LARGE, dict(n=2 ** 31))]),
    ("seacells_layer_norm_grad", NORM_GRAD, [
        (NULL, dict(d_out=None)), (NULL, dict(x=None)), (NULL, dict(mean=None)),
        (NULL, dict(rstd=None)), (TYPE, dict(dtype=3)), (TYPE, dict(weight_type=1)),
        (TYPE, dict(d_x=Q + 1)), (TYPE, dict(d_weight=Q + 1)), (SHAPE, dict(d=0)),
        (SHAPE, dict(d_out_ld=7)), (SHAPE, dict(d_x_ld=7)), (WORKSPACE, dict(ws=None)),
        (WORKSPACE, dict(ws_bytes=4)), (WORKSPACE, dict(ws=P + 4)), (TOO_LARGE, dict(n=2 ** 31))]),
    ("seacells_logprobs", LOGP, [
        (NULL, dict(logits=None)), (NULL, dict(targets=None)), (NULL, dict(top_idx=None)),
        (NULL, dict(top_logp=None)), (NULL, dict(status=None)), (TYPE, dict(dtype=3)),
        (TYPE, dict(logits=P + 1)), (TYPE, dict(stats=Q + 2)), (SHAPE, dict(v=0)),
        (SHAPE, dict(ld=7)), (SHAPE, dict(top_k=65)), (TOO_LARGE, dict(n=2 ** 31)),
        (TOO_LARGE, dict(v=2 ** 23 + 1, ld=2 ** 24))]),
    ("seacells_logprobs_grad", LOGP_GRAD, [
        (NULL, dict(logits=None)), (NULL, dict(stats=None)), (NULL, dict(d_logits=None)),
        (NULL, dict(entropy=None)), (NULL, dict(status=None)), (TYPE, dict(dtype=3)),
        (TYPE, dict(d_logits=Q + 1)), (SHAPE, dict(v=0)), (SHAPE, dict(ld=7)),
        (SHAPE, dict(d_ld=7)), (SHAPE, dict(d_logits=P, ld=8, d_ld=16)),
        (TOO_LARGE, dict(n=2 ** 31))]),
]


@pytest.mark.parametrize("fn,base,code,change",
                         [(fn, base, code, ch) for fn, base, rows in REFUSALS for code, ch in rows],
                         ids=lambda x: x if isinstance(x, str) else
                         "-".join(x) if isinstance(x, dict) and len(x) < 4 else "")
def test_entry_points_refuse_on_the_host(fn, base, code, change):
    assert call(fn, **base)(**change) == code


def test_few_rows_of_logits_need_their_workspace():
    need = saa.seacells_logprobs_workspace(1, 131072, 8)
    if need:
        go = call("seacells_logprobs", **dict(LOGP, n=1, v=131072, ld=131072, top_k=8))
        assert go(ws=None) == WORKSPACE and go(ws_bytes=need - 1) == WORKSPACE


def test_error_text():
    assert b"type" in saa.load().seacells_status_string(TYPE)
    assert native.ERRORS[TYPE] == "E_TYPE"


def test_workspace_queries_of_impossible_sizes_are_zero():
    assert saa.seacells_embed_grad_workspace(4, 0, 8) == 0
    assert saa.seacells_embed_grad_workspace(4, 8, 0) == 0
    assert saa.seacells_layer_norm_grad_workspace(4, 0) == 0
    assert saa.seacells_logprobs_workspace(4, 0, 0) == 0
    assert saa.seacells_logprobs_workspace(4, 8, 65) == 0
    assert saa.seacells_embed_grad_workspace(2 ** 32 + 4, 8, 8) == 0
    assert saa.seacells_layer_norm_grad_workspace(-1, 8) == 0


def test_binding_refuses_host_tensors_and_wrong_layouts():
    x, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(4)
    for go in (lambda: saa.seacells_embed(x, t), lambda: saa.seacells_embed_grad(t, x, 10),
               lambda: saa.seacells_layer_norm(x), lambda: saa.seacells_layer_norm_grad(x, x, f, f),
               lambda: saa.seacells_logprobs(x, t),
               lambda: saa.seacells_logprobs_grad(x, t, torch.zeros(4, 2)),
               lambda: saa.seacells_layer_norm(torch.zeros(2, 3, 8).transpose(0, 1))):
        with pytest.raises(SeacellsError):
            go()


def table_sizes():
    """Both sides of every step of the sort's buckets: their number and their ids."""
    steps = {1, 2, 255, 256, 511, 512, 1000, 2 ** 31 - 1}
    for s in range(22):
        for at in (1022 << s, 1023 << s, 1024 << s, 512 << s):
            steps |= {t for t in (at - 1, at, at + 1) if 0 < t < 2 ** 31}
    return sorted(steps)


@pytest.mark.parametrize("n", [1, 4096, 4097, 8192, 16383, 16384, 32768, 32769, 262144, 262145,
                               600000])
def test_every_cut_of_the_token_sort_is_written(n):
    """A chunk writes the cut of a bucket per counter, then its two totals; a
    bucket reads its own cut and the next one's."""
    for v in table_sizes():
        p = saa.seacells_debug_embed_plan(n, v, 1)
        assert (p["buckets"] - 1) << p["shift"] < v <= p["buckets"] << p["shift"], v
        assert (p["chunks"] == 0) == (n <= 4096)
        if p["chunks"] == 0:
            continue
        assert (p["chunks"] - 1) * p["chunk_len"] < n <= p["chunks"] * p["chunk_len"], v
        written = set(range(min(p["counters"], p["buckets"] + 1)))
        written |= {p["buckets"] + 1, p["buckets"] + 2}
        assert written == set(range(p["buckets"] + 3)), v
        end = p["cuts_offset"] + 4 * p["chunks"] * (p["buckets"] + 3)
        assert end <= saa.seacells_embed_grad_workspace(n, v, 1), v


def test_the_plan_of_the_token_sort_refuses():
    with pytest.raises(SeacellsError):
        saa.seacells_debug_embed_plan(4, 0, 8)
    with pytest.raises(SeacellsError):
        saa.seacells_debug_embed_plan(4, 2 ** 31, 8)
    assert saa.load().seacells_debug_embed_plan(4, 8, 8, None) == NULL


@pytest.mark.parametrize("d", [2 ** 31, 2 ** 32 + 5])
def test_binding_refuses_rows_whose_length_32_bits_cannot_hold(d):
    """A length is passed in 32 bits, where 2^32 + 5 elements would count as 5."""
    one = torch.empty(1, d, dtype=torch.bfloat16, device="meta")
    f = torch.empty(1)
    for go in (lambda: saa.seacells_embed(one, torch.zeros(1, dtype=torch.int32)),
               lambda: saa.seacells_embed_grad(torch.zeros(1, dtype=torch.int32), one, 3),
               lambda: saa.seacells_layer_norm(one), lambda: saa.seacells_layer_norm(one[0]),
               lambda: saa.seacells_layer_norm_grad(one, one, f, f),
               lambda: saa.seacells_logprobs(one),
               lambda: saa.seacells_logprobs_grad(one, None, torch.empty(1, 2))):
        with pytest.raises(SeacellsError, match=r"2\^31 - 1 elements"):
            go()


@pytest.mark.parametrize("fn,base,change,code", [
    ("seacells_layer_norm", dict(NORM, n=2 ** 31, out=P, out_ld=16), dict(x_ld=16), TOO_LARGE),
    ("seacells_layer_norm", dict(NORM, n=2 ** 31, out=P, x_ld=9), dict(out_ld=9), TOO_LARGE),
    ("seacells_layer_norm_grad", dict(NORM_GRAD, ws_bytes=4, d_x=P, x=Q, d_x_ld=16),
     dict(d_out_ld=16), WORKSPACE),
    ("seacells_layer_norm_grad", dict(NORM_GRAD, ws_bytes=4, d_x=P, d_out=Q, x_ld=9),
     dict(d_x_ld=9), WORKSPACE),
    ("seacells_layer_norm_grad", dict(NORM_GRAD, ws_bytes=4, d_x=P, d_x_ld=16), dict(n=1),
     WORKSPACE)], ids=lambda x: x if isinstance(x, str) else "")
def test_in_place_norms_refuse_two_strides(fn, base, change, code):
    """An output row would lie on input rows that other blocks have still to
    read. (The base has a second fault, which alone is left with one stride
    or one row: no call here comes to a launch.)"""
    assert call(fn, **base)() == SHAPE
    assert call(fn, **base)(**change) == code
