"""A small model over a fit: cells are tokens, K's neighbour pairs are the
training pairs, and the archetype of the neighbour is the class to predict.

    logits = layer_norm(scale * table[cell]) @ head^T
    loss   = mean over pairs of -log p[archetype] - beta * entropy

It runs the token operators (include/seacells_token.h) as a training step does,
forward and backward, and as a serving step does, with the top alternatives of
a few cells. The matrix products are torch's.

    python -m examples.archetype_tokens [--config c1] [--width 64] [--steps 200]
"""
import argparse
import math
import time

import numpy as np
import torch

import sparse_archetypal_analysis_amd as saa


class Model:
    """Parameters in f32 on the GPU; rows of the table and of the head are
    cells and archetypes."""

    def __init__(self, cells, archetypes, width, seed=0, device="cuda"):
        gen = torch.Generator(device="cpu").manual_seed(seed)
        self.scale = math.sqrt(width)
        self.table = (torch.randn(cells, width, generator=gen) / self.scale).to(device)
        self.weight = torch.ones(width, device=device)
        self.bias = torch.zeros(width, device=device)
        self.head = (torch.randn(archetypes, width, generator=gen) / self.scale).to(device)

    def parameters(self):
        return {"table": self.table, "weight": self.weight, "bias": self.bias, "head": self.head}


def forward(model, cells):
    """(embedded rows, normalised rows, mean, rstd, logits, status) of int32 cells."""
    x, status = saa.seacells_embed(model.table, cells, model.scale)
    h, mean, rstd = saa.seacells_layer_norm(x, model.weight, model.bias)
    return x, h, mean, rstd, h @ model.head.t(), status


def training_step(model, cells, archetypes, beta=0.0):
    """Loss (on the device), gradients by parameter and the step's status words.
    A negative archetype leaves its pair out of the loss' first term."""
    x, h, mean, rstd, logits, s0 = forward(model, cells)
    logp, entropy, stats, _, _, s1 = saa.seacells_logprobs(logits, archetypes)
    kept = (archetypes >= 0).sum().clamp(min=1).float()
    loss = -logp.sum() / kept - beta * entropy.mean()
    d_logp = (-1.0 / kept).expand(cells.numel()).contiguous()
    d_entropy = torch.full_like(d_logp, -beta / max(cells.numel(), 1))
    d_logits, s2 = saa.seacells_logprobs_grad(logits, archetypes, stats, entropy, d_logp, d_entropy,
                                              d_logits=logits)
    d_x, d_weight, d_bias = saa.seacells_layer_norm_grad(d_logits @ model.head, x, mean, rstd,
                                                         model.weight)
    d_table, s3 = saa.seacells_embed_grad(cells, d_x, model.table.shape[0], model.scale)
    grads = {"table": d_table, "weight": d_weight, "bias": d_bias, "head": d_logits.t() @ h}
    return loss, grads, (s0, s1, s2, s3)


def answer(model, cells, top_k=5):
    """The top_k likeliest archetypes of a few cells and their log probabilities."""
    _, _, _, _, logits, status = forward(model, cells)
    _, _, _, top, logp, s1 = saa.seacells_logprobs(logits, None, top_k)
    return top, logp, (status, s1)


def neighbour_pairs(w):
    """(cell, archetype of its neighbour) for every off-diagonal entry of K."""
    import workloads as W
    K = W.kernel_matrix(w).tocoo()
    of = np.asarray(w.a_prev_t.argmax(axis=1)).ravel()  # the archetype with the largest weight
    off = K.row != K.col
    return K.row[off].astype(np.int32), of[K.col[off]].astype(np.int32)


def main():
    import workloads as W
    p = argparse.ArgumentParser()
    p.add_argument("--config", default="c1")
    p.add_argument("--width", type=int, default=64)
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--batch", type=int, default=8192)
    p.add_argument("--rate", type=float, default=0.3)
    a = p.parse_args()
    if a.steps < 1:
        p.error("--steps must be at least 1")
    w = W.make(a.config)
    cells, archetypes = (torch.from_numpy(t).cuda() for t in neighbour_pairs(w))
    model = Model(w.n, w.k, a.width)
    gen = torch.Generator(device="cuda").manual_seed(1)
    seen = []
    first = min(3, a.steps - 1)  # the steps before load the kernels and are not timed
    for step in range(a.steps):
        pick = torch.randint(0, cells.numel(), (a.batch,), generator=gen, device="cuda")
        if step == first:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
        loss, grads, status = training_step(model, cells[pick], archetypes[pick], beta=0.01)
        for name, value in model.parameters().items():
            # (a row of the table meets a few of the batch's pairs only)
            value.sub_(grads[name], alpha=a.rate * (w.n / 64 if name == "table" else 1.0))
        seen.append(loss)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) / (a.steps - first) * 1e3
    for s in status:
        saa.raise_on_status(s)
    some = torch.arange(0, w.n, w.n // 4, dtype=torch.int32, device="cuda")[:4]
    top, logp, _ = answer(model, some)
    print("%d cells, %d archetypes, %d pairs; %.3f ms per step" % (w.n, w.k, cells.numel(), ms))
    print("loss %.3f -> %.3f (log k = %.3f)" % (seen[0], seen[-1], math.log(w.k)))
    for i in range(4):
        print("cell %d: archetypes %s, log p %s" % (int(some[i]), top[i].tolist(),
                                                   ["%.2f" % v for v in logp[i].tolist()]))


if __name__ == "__main__":
    main()
