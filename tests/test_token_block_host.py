"""Refusals of the gated block and of the log probabilities from hidden rows
(include/seacells_token.h): the C entry points' host checks and the binding's,
all before any GPU work; the workspace queries; and the 64-bit forms that the
GPU tests compare against, by differences."""
import numpy as np
import pytest
import torch

import sparse_archetypal_analysis_amd as saa
from sparse_archetypal_analysis_amd import SeacellsError
from tests import block_reference as R
from tests.test_token_host import NULL, SHAPE, TOO_LARGE, TYPE, WORKSPACE, P, Q, call

FFN = dict(x=P, dtype=2, n=4, d=8, x_ld=8, w_in=P, w_in_ld=8, f=16, w_out=P, w_out_ld=16, m=8, act=0,
           out=Q, out_ld=8, pre=Q, pre_ld=32, ws=P, ws_bytes=1 << 20, stream=None)
FFN_GRAD = dict(d_out=P, d_out_ld=8, x=P, dtype=2, n=4, d=8, x_ld=8, pre=P, pre_ld=32, w_in=P, w_in_ld=8,
                f=16, w_out=P, w_out_ld=16, m=8, act=0, d_x=Q, d_x_ld=8, d_w_in=Q, d_w_in_ld=8,
                d_w_out=Q, d_w_out_ld=16, ws=P, ws_bytes=1 << 22, stream=None)
LOSS = dict(x=P, dtype=2, n=4, d=8, x_ld=8, table=P, table_ld=8, v=10, bias=P, targets=P, logp=Q,
            entropy=Q, stats=Q, ws=P, ws_bytes=1 << 20, status=P, stream=None)
LOSS_GRAD = dict(x=P, dtype=2, n=4, d=8, x_ld=8, table=P, table_ld=8, v=10, bias=P, targets=P, stats=P,
                 entropy=P, d_logp=P, d_entropy=P, d_x=Q, d_x_ld=8, d_table=Q, d_table_ld=8, d_bias=Q,
                 ws=P, ws_bytes=1 << 22, status=P, stream=None)

REFUSALS = [
    ("seacells_gated_ffn", FFN, [
        (NULL, dict(x=None)), (NULL, dict(w_in=None)), (NULL, dict(w_out=None)), (NULL, dict(out=None)),
        (TYPE, dict(dtype=3)), (TYPE, dict(x=P + 1)), (TYPE, dict(w_in=P + 1)), (TYPE, dict(w_out=P + 1)),
        (TYPE, dict(out=Q + 1)), (TYPE, dict(pre=Q + 1)), (TYPE, dict(dtype=0, x=P + 2)),
        (SHAPE, dict(d=0)), (SHAPE, dict(f=0)), (SHAPE, dict(m=0)), (SHAPE, dict(act=3)),
        (SHAPE, dict(x_ld=7)), (SHAPE, dict(w_in_ld=7)), (SHAPE, dict(w_out_ld=15)),
        (SHAPE, dict(out_ld=7)), (SHAPE, dict(pre_ld=31)), (WORKSPACE, dict(ws=None)),
        (WORKSPACE, dict(ws_bytes=16)), (WORKSPACE, dict(ws=P + 16)), (TOO_LARGE, dict(n=2 ** 31)),
        (TOO_LARGE, dict(f=2 ** 20 + 1, w_out_ld=2 ** 21, pre_ld=2 ** 22)),
        (TOO_LARGE, dict(d=2 ** 20 + 1, x_ld=2 ** 21, w_in_ld=2 ** 21)),
        (TOO_LARGE, dict(m=2 ** 20 + 1, out_ld=2 ** 21)), (TOO_LARGE, dict(x_ld=2 ** 40)),
        (TOO_LARGE, dict(d=2 ** 15, x_ld=2 ** 15, w_in_ld=2 ** 15, f=2 ** 15, w_out_ld=2 ** 15,
                         pre_ld=2 ** 16))]),
    ("seacells_gated_ffn_grad", FFN_GRAD, [
        (NULL, dict(d_out=None)), (NULL, dict(x=None)), (NULL, dict(pre=None)), (NULL, dict(w_in=None)),
        (NULL, dict(w_out=None)), (TYPE, dict(dtype=3)), (TYPE, dict(d_out=P + 1)), (TYPE, dict(pre=P + 1)),
        (TYPE, dict(d_x=Q + 1)), (TYPE, dict(d_w_in=Q + 1)), (TYPE, dict(d_w_out=Q + 1)),
        (SHAPE, dict(d=0)), (SHAPE, dict(f=0)), (SHAPE, dict(m=0)), (SHAPE, dict(act=9)),
        (SHAPE, dict(d_out_ld=7)), (SHAPE, dict(pre_ld=31)), (SHAPE, dict(d_x_ld=7)),
        (SHAPE, dict(d_w_in_ld=7)), (SHAPE, dict(d_w_out_ld=15)), (WORKSPACE, dict(ws=None)),
        (WORKSPACE, dict(ws_bytes=16)), (WORKSPACE, dict(ws=P + 128)), (TOO_LARGE, dict(n=2 ** 31))]),
    ("seacells_linear_logprobs", LOSS, [
        (NULL, dict(x=None)), (NULL, dict(table=None)), (NULL, dict(targets=None)),
        (NULL, dict(status=None)), (TYPE, dict(dtype=7)), (TYPE, dict(x=P + 1)), (TYPE, dict(table=P + 1)),
        (TYPE, dict(bias=P + 2)), (TYPE, dict(targets=P + 1)), (TYPE, dict(logp=Q + 2)),
        (TYPE, dict(entropy=Q + 2)), (TYPE, dict(stats=Q + 2)), (SHAPE, dict(v=0)), (SHAPE, dict(d=0)),
        (SHAPE, dict(x_ld=7)), (SHAPE, dict(table_ld=7)), (WORKSPACE, dict(ws=None)),
        (WORKSPACE, dict(ws_bytes=16)), (WORKSPACE, dict(ws=P + 8)), (TOO_LARGE, dict(n=2 ** 31)),
        (TOO_LARGE, dict(v=2 ** 23 + 1)),
        (TOO_LARGE, dict(d=2 ** 20 + 1, x_ld=2 ** 21, table_ld=2 ** 21))]),
    ("seacells_linear_logprobs_grad", LOSS_GRAD, [
        (NULL, dict(x=None)), (NULL, dict(table=None)), (NULL, dict(stats=None)),
        (NULL, dict(entropy=None)), (NULL, dict(status=None)), (TYPE, dict(dtype=7)),
        (TYPE, dict(d_x=Q + 1)), (TYPE, dict(d_table=Q + 1)), (TYPE, dict(d_bias=Q + 2)),
        (TYPE, dict(stats=P + 2)), (TYPE, dict(d_logp=P + 1)), (SHAPE, dict(v=0)), (SHAPE, dict(d=0)),
        (SHAPE, dict(d_x_ld=7)), (SHAPE, dict(d_table_ld=7)), (WORKSPACE, dict(ws=None)),
        (WORKSPACE, dict(ws_bytes=16)), (WORKSPACE, dict(ws=P + 4)), (TOO_LARGE, dict(n=2 ** 31)),
        (TOO_LARGE, dict(v=2 ** 23 + 1))]),
]


@pytest.mark.parametrize("fn,base,code,change",
                         [(fn, base, code, ch) for fn, base, rows in REFUSALS for code, ch in rows],
                         ids=lambda x: x if isinstance(x, str) else
                         "-".join(x) if isinstance(x, dict) and len(x) < 4 else "")
def test_entry_points_refuse_on_the_host(fn, base, code, change):
    assert call(fn, **base)(**change) == code


QUERIES = [(saa.seacells_gated_ffn_workspace, 4), (saa.seacells_gated_ffn_grad_workspace, 4),
           (saa.seacells_linear_logprobs_workspace, 3), (saa.seacells_linear_logprobs_grad_workspace, 3)]


@pytest.mark.parametrize("query,count", QUERIES)
def test_workspace_queries(query, count):
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        for n in (1, 64, 65, 500):
            some = query(dtype, n, *[64] * (count - 1))
            there = query(dtype, n, *[64] * (count - 1), on_16_bytes=True)
            assert 0 < there <= some
            if n > 64:  # copies only where rows do not start on 16 bytes, or elements are f32
                assert (there == some) == (dtype == torch.float32)
        assert query(dtype, *[60] * count, on_16_bytes=True) > 0
        assert query(dtype, 0, *[64] * (count - 1)) == 0
        for i in range(1, count):
            sizes = [64] * count
            sizes[i] = 0
            assert query(dtype, *sizes) == 0
            sizes[i] = 2 ** 32 + 64
            assert query(dtype, *sizes) == 0
    with pytest.raises(SeacellsError):
        query(torch.float64, *[64] * count)


def test_binding_refuses_host_tensors():
    x, w, o = torch.zeros(4, 8), torch.zeros(12, 8), torch.zeros(5, 6)
    t = torch.zeros(4, dtype=torch.int32)
    for go in (lambda: saa.seacells_gated_ffn(x, w, o),
               lambda: saa.seacells_gated_ffn_grad(torch.zeros(4, 5), x, torch.zeros(4, 12), w, o),
               lambda: saa.seacells_linear_logprobs(x, w, t),
               lambda: saa.seacells_linear_logprobs_grad(x, w, t, torch.zeros(4, 2))):
        with pytest.raises(SeacellsError):
            go()


def slopes(f, args, which, step=1e-6):
    """Central differences of a scalar f to every entry of args[which]."""
    out = np.zeros_like(args[which])
    for at in np.ndindex(*out.shape):
        vals = []
        for s in (step, -step):
            moved = [a.copy() for a in args]
            moved[which][at] += s
            vals.append(f(*moved))
        out[at] = (vals[0] - vals[1]) / (2 * step)
    return out


@pytest.mark.parametrize("name", ["silu", "gelu", "relu"])
def test_reference_block_gradients_by_differences(name):
    rng = np.random.default_rng(5)
    n, d, f, m = 3, 4, 5, 2
    x, wi, wo, dy = (rng.normal(size=s) for s in ((n, d), (2 * f, d), (m, f), (n, m)))
    args = [x, wi, wo]

    def value(x, wi, wo):
        return (R.ffn(x, wi, wo, name, "f32")[0][0] * dy).sum()

    got, _ = R.ffn_grad(dy, x, x @ wi.T, wi, wo, name, "f32")
    for i in range(3):
        assert np.allclose(got[i], slopes(value, args, i), rtol=1e-6, atol=1e-7)


def test_reference_loss_gradients_by_differences():
    rng = np.random.default_rng(5)
    n, d, v = 4, 3, 6
    x, table, bias = (rng.normal(size=s) for s in ((n, d), (v, d), (v,)))
    bias[2] = -np.inf
    t = np.array([1, -1, 5, 0])
    gl, ge = rng.normal(size=n), rng.normal(size=n)

    def value(x, table, b):
        b = b.copy()
        b[2] = -np.inf
        (logp, H, _), _ = R.loss(x, table, b, t, "f32")
        return (gl * logp + ge * H).sum()

    (_, H, stats), _ = R.loss(x, table, bias, t, "f32")
    got, _ = R.loss_grad(x, table, bias, t, stats, H, gl, ge, "f32")
    flat = np.where(bias == -np.inf, 0.0, bias)
    for i in range(3):
        assert np.allclose(got[i], slopes(value, [x, table, flat], i), rtol=1e-6, atol=1e-7)
