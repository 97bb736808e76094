"""The example that runs the token operators together: its gradients against
64-bit autograd of the same formulas, and that it learns."""
import math

import numpy as np
import pytest
import torch

from examples import archetype_tokens as E

pytestmark = pytest.mark.gpu


def reference(model, cells, archetypes, beta):
    """Loss and gradients in 64 bits on the CPU, by autograd of the formulas."""
    p = {k: t.detach().cpu().double().requires_grad_() for k, t in model.parameters().items()}
    c, t = cells.cpu().long(), archetypes.cpu().long()
    x = p["table"][c] * model.scale
    mean = x.mean(dim=1, keepdim=True)
    var = (x - mean).square().mean(dim=1, keepdim=True)
    h = (x - mean) / (var + float(np.float32(1e-5))).sqrt() * p["weight"] + p["bias"]
    lp = (h @ p["head"].t()).log_softmax(dim=1)
    kept = t >= 0
    loss = -lp[kept, t[kept]].sum() / kept.sum().clamp(min=1)
    loss = loss + beta * (lp.exp() * lp).sum(dim=1).mean()
    loss.backward()
    return loss.item(), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("n,k,d,batch", [(40, 7, 24, 300), (500, 1300, 64, 77), (9, 25, 5, 1)])
def test_a_training_step_gives_the_formulas_gradients(n, k, d, batch):
    gen = torch.Generator().manual_seed(n + k)
    model = E.Model(n, k, d, seed=3)
    cells = torch.randint(0, n, (batch,), generator=gen).to(torch.int32).cuda()
    archetypes = torch.randint(0, k, (batch,), generator=gen).to(torch.int32)
    archetypes[::5] = -1
    if batch == 1:
        archetypes[0] = k - 1
    loss, grads, status = E.training_step(model, cells, archetypes.cuda(), beta=0.05)
    assert [int(s) for s in status] == [0, 0, 0, 0]
    want, want_grads = reference(model, cells, archetypes, 0.05)
    # f32 products over d and k terms, sums over the batch: a few hundred
    # roundings on values near the largest gradient
    tol = 64.0 * 2.0 ** -24 * math.sqrt(max(d, k, batch))
    assert abs(loss.item() - want) <= tol * max(1.0, abs(want))
    for name, g in grads.items():
        w = want_grads[name]
        assert g.shape == w.shape
        assert float((g.cpu().double() - w).abs().max()) <= tol * float(w.abs().max()), name


@pytest.mark.parametrize("steps", [1, 3, 5])
def test_the_command_runs_any_number_of_steps(monkeypatch, capsys, steps):
    monkeypatch.setattr("sys.argv", ["archetype_tokens", "--steps", str(steps), "--batch", "500"])
    E.main()
    out = capsys.readouterr().out
    assert "ms per step" in out and "loss" in out and out.count("archetypes [") == 4


def test_the_command_refuses_no_steps(monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["archetype_tokens", "--steps", "0"])
    with pytest.raises(SystemExit):
        E.main()
    assert "--steps" in capsys.readouterr().err


def test_the_model_learns_and_answers():
    rng = np.random.default_rng(0)
    n, k = 300, 12
    of = torch.from_numpy(rng.integers(0, k, n).astype(np.int32)).cuda()
    model = E.Model(n, k, 32, seed=1)
    losses = []
    for step in range(60):
        cells = torch.from_numpy(rng.integers(0, n, 2048).astype(np.int32)).cuda()
        loss, grads, status = E.training_step(model, cells, of[cells.long()])
        for name, value in model.parameters().items():
            value.sub_(grads[name], alpha=20.0 if name == "table" else 0.5)
        losses.append(loss)
    assert [int(s) for s in status] == [0, 0, 0, 0]
    losses = [float(v) for v in losses]
    assert losses[0] > 1.5 and losses[-1] < 0.5 * losses[0]
    every = torch.arange(n, dtype=torch.int32, device="cuda")
    top, logp, _ = E.answer(model, every, top_k=3)
    assert top.shape == (n, 3) and bool((logp[:, :1] >= logp).all())
    assert float((top[:, 0] == of).float().mean()) > 0.8
