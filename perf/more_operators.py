"""Measured cases of the token model's block and head: the gated feed-forward
block and its gradient, and log probabilities of given classes straight from
hidden rows and the class table, in pieces of the classes, with their gradient.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, where ``own`` is true, through the
library's entry points. ``exact`` computes the same outputs in 64 bits from
the operators' definitions, apart from both.

Definitions (n rows of d elements, f the block's inner width, v classes):

  ffn         pre = x w_in^T, w_in [2f, d]: f gate rows, then f up rows;
              h = act(pre[:, :f]) * pre[:, f:], y = h w_out^T, w_out [m, f].
              act: silu g / (1 + e^-g), gelu g Phi(g) or relu. A training pass
              keeps pre, rounded to x's type; a serving pass returns y alone
  ffn_grad    with dh = d_y w_out, g and u the halves of the pre that the
              forward pass left, d_pre = [dh u act'(g), dh act(g)]:
              d_x = d_pre w_in, d_w_in = d_pre^T x, d_w_out = d_y^T h
  loss        z = x table^T + bias; m = max z, s = log sum exp(z - m) per row,
              logp = z[target] - m - s, entropy = -sum p log p, stats (m, s).
              A class whose bias is -inf is masked (p = 0). A negative target
              is ignored: logp 0
  loss_grad   d_z = d_logp (1[target] - p) - d_entropy p (log p + H), 0 at
              masked classes; d_x = d_z table, d_table = d_z^T x,
              d_bias = column sums of d_z
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def _ffn(name, op, n, d, f, m, dtype, act, keep, gap):
    return {"name": name, "op": op, "n": n, "d": d, "f": f, "m": m, "dtype": dtype, "act": act,
            "keep": keep, "gap": gap}


def _loss(name, op, n, d, v, dtype, bias, mask, gap):
    return {"name": name, "op": op, "n": n, "d": d, "v": v, "dtype": dtype, "bias": bias,
            "mask": mask, "gap": gap}


def listed():
    return [
        # a serving step: the newest token of one request through a small block
        _ffn("ffn_token", "ffn", 1, 1024, 4096, 1024, "bf16", "silu", False, 0),
        # a serving step of 32 requests
        _ffn("ffn_step", "ffn", 32, 4096, 8192, 4096, "bf16", "silu", False, 0),
        # a training pass over ragged rows, odd widths and rows in padded buffers
        _ffn("ffn_odd", "ffn", 5003, 1003, 2731, 1003, "f16", "gelu", True, 5),
        # a training batch of a wide model
        _ffn("ffn_batch", "ffn", 8192, 4096, 16384, 4096, "bf16", "silu", True, 0),
        # a block over a batch of cells, f32 as the example's model
        _ffn("ffn_grad_cells", "ffn_grad", 8192, 256, 1000, 256, "f32", "gelu", True, 0),
        # a training batch's gradient
        _ffn("ffn_grad_batch", "ffn_grad", 16384, 2048, 8192, 2048, "bf16", "silu", True, 0),
        # a scoring step of 4 requests over many classes
        _loss("loss_step", "loss", 4, 2048, 131072, "bf16", False, 0.0, 0),
        # archetypes of 100k cells (k = 1300) from rows of 100 elements
        _loss("loss_cells", "loss", 100000, 100, 1300, "f32", True, 0.0, 0),
        # a training batch's loss, nothing kept but two numbers a row
        _loss("loss_batch", "loss", 8192, 2048, 131072, "bf16", False, 0.0, 0),
        # a batch of cells in f32 as the example trains it
        _loss("loss_grad_cells", "loss_grad", 8192, 64, 1300, "f32", True, 0.0, 0),
        # odd counts, masked classes, rows in padded buffers
        _loss("loss_grad_odd", "loss_grad", 3001, 520, 50001, "f16", True, 0.2, 8),
        # a training batch's gradient
        _loss("loss_grad_batch", "loss_grad", 8192, 2048, 65536, "bf16", False, 0.0, 0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row's length: three in four a multiple of 64, as models have them."""
    w = _log_int(rng, lo, hi)
    return w if rng.random() < 0.25 else max(64, w // 64 * 64)


def draw(rng):
    """One more case: sizes log-uniform over the range, types, activations and
    masks mixed; rows are cut so that no case computes more than the largest
    listed one (f32 a sixth of that)."""
    op = rng.choice(["ffn", "ffn_grad", "loss", "loss_grad"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    most = 3.2e12 / (6 if dtype == "f32" else 1) / (1 if op in ("ffn", "loss") else 2)
    gap = rng.choice([0, 0, rng.randint(1, 64)])
    if op in ("ffn", "ffn_grad"):
        d, f = _width(rng, 16, 4096), _width(rng, 16, 16384)
        m = d if rng.random() < 0.8 else _width(rng, 16, 4096)
        n = min(_log_int(rng, 1, 65536), max(1, int(most / (2 * f * (2 * d + m)))))
        keep = op == "ffn_grad" or rng.random() < 0.6
        c = _ffn("", op, n, d, f, m, dtype, rng.choice(["silu", "gelu", "relu"]), keep, gap)
    else:
        d, v = _width(rng, 16, 4096), _log_int(rng, 2, 131072)
        n = min(_log_int(rng, 1, 131072), 2 ** 30 // v, max(1, int(most / (2 * v * d))))
        bias = rng.random() < 0.5
        c = _loss("", op, n, d, v, dtype, bias, rng.choice([0.0, 0.3]) if bias else 0.0, gap)
    del c["name"]
    return c


# ---------------------------------------------------------------- definitions

def _act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return torch.where(g > 0, g, 0.0)


def _act_grad(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
                + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi))
    return torch.where(g > 0, 1.0, 0.0)


def _lse(z):
    """Row maximum, log sum exp(z - max) and z - max, rows with nothing left (-inf, 0)."""
    m = z.max(dim=1, keepdim=True).values
    left = m > -math.inf
    t = torch.where(left, z - m, -math.inf)
    s = torch.exp(t).sum(dim=1, keepdim=True)
    return m, torch.where(left, torch.log(s), 0.0), t


def _entropy(t, ls):
    lp = t - ls
    return -torch.where(t > -math.inf, torch.exp(lp) * lp, 0.0).sum(dim=1)


def _logits(x, table, bias):
    z = x.float() @ table.float().t()
    return z if bias is None else z + bias


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, n, d, dt = case["op"], case["n"], case["d"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def rows(count, width, spread=1.0):
        """Rows in a buffer that may be wider than they are."""
        base = torch.empty(count, width + case["gap"], dtype=dt, device="cuda")
        out = base[:, :width]
        return out.copy_(spread * normal(count, width))

    s = {"op": op, "ws": None, "x": rows(n, d)}
    if op in ("ffn", "ffn_grad"):
        f, m = case["f"], case["m"]
        s["act"], s["keep"] = case["act"], case["keep"]
        s["w_in"] = (normal(2 * f, d) / math.sqrt(d)).to(dt)
        s["w_out"] = (normal(m, f) / math.sqrt(f)).to(dt)
        if op == "ffn":
            s["out"] = torch.empty(n, m, dtype=dt, device="cuda")
            s["pre"] = torch.empty(n, 2 * f, dtype=dt, device="cuda") if case["keep"] else False
        else:
            # what the forward pass left, and the gradient of a mean over rows
            s["pre"] = (s["x"].float() @ s["w_in"].float().t()).to(dt)
            s["d_out"] = rows(n, m, 0.1)
            s["d_x"] = torch.empty(n, d, dtype=dt, device="cuda")
            s["d_w_in"], s["d_w_out"] = torch.empty_like(s["w_in"]), torch.empty_like(s["w_out"])
        return s
    v = case["v"]
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    # logits of a trained head spread by a few units
    s["table"] = rows(v, d, 2.5 / math.sqrt(d))
    s["bias"] = None
    if case["bias"]:
        s["bias"] = 0.5 * normal(v)
        if case["mask"]:
            # classes that may not be answered with
            hide = torch.rand(v, generator=gen, device="cuda") < case["mask"]
            hide[0] = False
            s["bias"].masked_fill_(hide, -math.inf)
    targets = torch.randint(0, v, (n,), generator=gen, device="cuda")
    targets = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.05, -1, targets)
    s["targets"] = targets.to(torch.int32)
    s["stats"] = torch.empty(n, 2, device="cuda")
    s["entropy"] = torch.empty(n, device="cuda")
    if op == "loss":
        s["logp"] = torch.empty(n, device="cuda")
        return s
    step = max(1, 2 ** 28 // v)
    for i in range(0, n, step):  # what the forward pass left
        mx, ls, t = _lse(_logits(s["x"][i:i + step], s["table"], s["bias"]))
        s["stats"][i:i + step] = torch.cat([mx, ls], dim=1)
        s["entropy"][i:i + step] = _entropy(t, ls)
    # a mean over the rows and an entropy term, scaled as training in f16 scales its loss
    mean = (4096.0 if case["dtype"] == "f16" else 1.0) / n
    s["d_logp"] = -mean * (1.0 + 0.1 * normal(n))
    s["d_entropy"] = -0.01 * mean * (1.0 + 0.1 * normal(n))
    s["d_x"] = torch.empty(n, d, dtype=dt, device="cuda")
    s["d_table"] = torch.empty(v, d, dtype=dt, device="cuda")
    s["d_bias"] = torch.empty(v, device="cuda") if s["bias"] is not None else None
    return s


def _kept(s, size):
    """The workspace that a program keeps from call to call."""
    if s["ws"] is None:
        s["ws"] = torch.empty(max(256, size), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_own(s):
    import sparse_archetypal_analysis_amd as saa
    op, x = s["op"], s["x"]
    n, d = x.shape
    if op in ("ffn", "ffn_grad"):
        m, f = s["w_out"].shape
        if op == "ffn":
            ws = s["ws"]
            if ws is None:
                ws = _kept(s, saa.seacells_gated_ffn_workspace(x.dtype, n, d, f, m))
            out, pre = saa.seacells_gated_ffn(x, s["w_in"], s["w_out"], s["act"], out=s["out"],
                                              pre=s["pre"], workspace=ws)
            return (out, pre) if s["keep"] else out
        ws = s["ws"]
        if ws is None:
            ws = _kept(s, saa.seacells_gated_ffn_grad_workspace(x.dtype, n, d, f, m))
        return saa.seacells_gated_ffn_grad(s["d_out"], x, s["pre"], s["w_in"], s["w_out"], s["act"],
                                           d_x=s["d_x"], d_w_in=s["d_w_in"], d_w_out=s["d_w_out"],
                                           workspace=ws)
    v = s["table"].shape[0]
    ws = s["ws"]
    if op == "loss":
        if ws is None:
            ws = _kept(s, saa.seacells_linear_logprobs_workspace(x.dtype, n, d, v))
        return saa.seacells_linear_logprobs(x, s["table"], s["targets"], s["bias"], logp=s["logp"],
                                            entropy=s["entropy"], stats=s["stats"], workspace=ws,
                                            status=s["status"])[:3]
    if ws is None:
        ws = _kept(s, saa.seacells_linear_logprobs_grad_workspace(x.dtype, n, d, v))
    got = saa.seacells_linear_logprobs_grad(x, s["table"], s["targets"], s["stats"], s["entropy"],
                                            s["d_logp"], s["d_entropy"], s["bias"], d_x=s["d_x"],
                                            d_table=s["d_table"], d_bias=s["d_bias"], workspace=ws,
                                            status=s["status"])
    return got[:2] if s["bias"] is None else got[:3]


def run(s):
    if own:
        return _run_own(s)
    op, x = s["op"], s["x"]
    dt = x.dtype
    if op == "ffn":
        pre = x.float() @ s["w_in"].float().t()
        g, u = pre.chunk(2, dim=1)
        y = ((_act(g, s["act"]) * u) @ s["w_out"].float().t()).to(dt)
        return (y, pre.to(dt)) if s["keep"] else y
    if op == "ffn_grad":
        g, u = s["pre"].float().chunk(2, dim=1)
        dy, act = s["d_out"].float(), s["act"]
        a = _act(g, act)
        dh = dy @ s["w_out"].float()
        d_pre = torch.cat([dh * u * _act_grad(g, act), dh * a], dim=1)
        return ((d_pre @ s["w_in"].float()).to(dt), (d_pre.t() @ x.float()).to(dt),
                (dy.t() @ (a * u)).to(dt))
    z = _logits(x, s["table"], s["bias"])
    t = s["targets"].long()
    if op == "loss":
        m, ls, c = _lse(z)
        at = c.gather(1, t.clamp(min=0)[:, None]) - ls
        return torch.where(t >= 0, at[:, 0], 0.0), _entropy(c, ls), torch.cat([m, ls], dim=1)
    m, ls = s["stats"][:, :1], s["stats"][:, 1:]
    lp = torch.where(z > -math.inf, z - m - ls, -math.inf)
    p = torch.exp(lp)
    hit = torch.arange(z.shape[1], device=z.device) == t[:, None]
    dz = torch.where(t >= 0, s["d_logp"], 0.0)[:, None] * (hit.float() - p)
    dz = dz - s["d_entropy"][:, None] * p * (torch.where(lp > -math.inf, lp, 0.0)
                                             + s["entropy"][:, None])
    dz = torch.where(z > -math.inf, dz, 0.0)
    out = ((dz @ s["table"].float()).to(dt), (dz.t() @ x.float()).to(dt))
    return out if s["bias"] is None else (*out, dz.sum(dim=0))


def work(case):
    op, n, d, e = case["op"], case["n"], case["d"], SIZE[case["dtype"]]
    if op in ("ffn", "ffn_grad"):
        f, m = case["f"], case["m"]
        weights = e * f * (2 * d + m)
        if op == "ffn":
            rows = e * n * (d + m + (2 * f if case["keep"] else 0))
            return {"bytes": rows + weights, "flops": 2 * n * f * (2 * d + m)}
        return {"bytes": e * n * (m + 2 * d + 2 * f) + 2 * weights, "flops": 4 * n * f * (2 * d + m)}
    v = case["v"]
    vector = 4 * v if case["bias"] else 0
    if op == "loss":
        return {"bytes": e * d * (n + v) + vector + 20 * n, "flops": 2 * n * v * d}
    return {"bytes": 2 * e * d * (n + v) + 2 * vector + 24 * n, "flops": 6 * n * v * d}


# ------------------------------------------------------------ 64-bit outcome

def _gate64(g, act):
    """act(g) and its derivative in 64 bits."""
    if act == "relu":
        return g.clamp(min=0.0), (g > 0).double()
    if act == "gelu":
        phi = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5
    s = 1.0 / (1.0 + torch.exp(-g))
    return g * s, s + g * s * (1.0 - s)


def _exact_ffn(s):
    w_in, w_out, f = s["w_in"].double(), s["w_out"].double(), s["w_out"].shape[1]
    n = s["x"].shape[0]
    step = max(1, 2 ** 27 // (2 * f))
    if s["op"] == "ffn":
        ys, pres = [], []
        for i in range(0, n, step):
            x = s["x"][i:i + step].double()
            g, u = x @ w_in[:f].t(), x @ w_in[f:].t()
            ys.append((_gate64(g, s["act"])[0] * u) @ w_out.t())
            if s["keep"]:
                pres.append(torch.cat([g, u], dim=1))
        return (torch.cat(ys), torch.cat(pres)) if s["keep"] else torch.cat(ys)
    d_x, d_in, d_out = [], torch.zeros_like(w_in), torch.zeros_like(w_out)
    for i in range(0, n, step):
        x, dy = s["x"][i:i + step].double(), s["d_out"][i:i + step].double()
        g, u = s["pre"][i:i + step, :f].double(), s["pre"][i:i + step, f:].double()
        a, da = _gate64(g, s["act"])
        dh = dy @ w_out
        dg, du = dh * u * da, dh * a
        d_x.append(dg @ w_in[:f] + du @ w_in[f:])
        d_in[:f] += dg.t() @ x
        d_in[f:] += du.t() @ x
        d_out += dy.t() @ (a * u)
    return torch.cat(d_x), d_in, d_out


def _exact_loss(s):
    table = s["table"].double()
    v = table.shape[0]
    bias = torch.zeros(v, dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"].double()
    shut = bias == -math.inf
    n = s["x"].shape[0]
    step = max(1, 2 ** 28 // v)
    rows, d_table, d_bias = [], torch.zeros_like(table), torch.zeros_like(bias)
    for i in range(0, n, step):
        x, t = s["x"][i:i + step].double(), s["targets"][i:i + step].long()
        z = torch.addmm(bias, x, table.t())
        top = z.amax(dim=1)
        e = (z - top[:, None]).exp_()
        total = e.sum(dim=1)
        known = (t >= 0).nonzero()[:, 0]
        if s["op"] == "loss":
            p = e / total[:, None]
            z.sub_((top + total.log())[:, None])
            got = torch.zeros_like(top)
            got[known] = z[known, t[known]]
            rows.append((got, -torch.where(p > 0, z, 0.0).mul_(p).sum(dim=1),
                         torch.stack([top, total.log()], dim=1)))
            continue
        e.div_(total[:, None])
        ent = -torch.special.xlogy(e, e).sum(dim=1)
        dl, de = s["d_logp"][i:i + step].double(), s["d_entropy"][i:i + step].double()
        dz = -e * (dl * (t >= 0) + de * ent)[:, None] - de[:, None] * torch.special.xlogy(e, e)
        dz[known, t[known]] += dl[known]
        dz[:, shut] = 0.0
        rows.append((dz @ table,))
        d_table += dz.t() @ x
        d_bias += dz.sum(dim=0)
    out = tuple(torch.cat(r) for r in zip(*rows))
    if s["op"] == "loss":
        return out
    return (*out, d_table) if s["bias"] is None else (*out, d_table, d_bias)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_ffn(s) if s["op"] in ("ffn", "ffn_grad") else _exact_loss(s)
