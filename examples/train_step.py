#!/usr/bin/env python3
"""Whole training steps of a small model in this library's calls: embedding,
norm with the activation quantizer, a Sparse-BitLinear layer, norm, the output
head that shares the embedding's table, every gradient back, and AdamW.

A step:
  masters (BF16)   -> quant_weights -> packed ternary 6:8 weights, beta
  ids              -> embed (tied table) -> x (fp32)
  x                -> norm_quant -> int8, gamma (and the normed x);  linear -> y
  x + y            -> norm -> h (BF16);  head_ce(h, table) -> per-token losses
  backward         -> head_ce_backward -> dh, dtable
                      norm_backward -> d(x + y);  sbl_linear_backward -> dx of the layer, dw
                      norm_backward -> dx;  embed_backward adds the lookup's part to dtable
  all weights      -> sbl_adamw_batch: masters and table in BF16 with their low
                      bits (the table's states in 8 bits), norm weights in fp32

The data are synthetic: every token is followed by a fixed other one, a tenth
of the targets is taken out, the ends of the sequences are padding.

  python examples/train_step.py [--steps 40] [--tokens 512] [--width 256] [--vocab 1000]
"""

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from sparse_linear_layers_absmean_amd import sbl  # noqa: E402

N, M, FMT = 6, 8, sbl.SBL_FMT_DENSE2
ADAM = dict(beta1=0.9, beta2=0.99, eps=1e-8)


def model(width, vocab, seed=0):
    """Weights with their optimizer states, as the dicts that AdamWItems takes (gradients still to come)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def master(*shape, bits):
        w, low = sbl.split_master(torch.randn(*shape, generator=g, device="cuda") / shape[-1] ** 0.5)
        return dict(w=w, w_low=low, weight_decay=0.01, **sbl.adamw_state(w, bits))

    def vector(value):
        w = torch.full((width,), value, device="cuda")
        return dict(w=w, **sbl.adamw_state(w))

    return dict(table=master(vocab, width, bits=8), layer=master(width, width, bits=32), norm1=vector(1.0),
                bias1=vector(0.0), norm2=vector(1.0), bias2=vector(0.0))


def data(tokens, vocab, seed=0):
    """(ids, targets) of one batch: -1 and -100 where there is none."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    after = torch.randperm(vocab, generator=g, device="cuda")
    rank = torch.rand(tokens, generator=g, device="cuda") ** 3         # some ids often, most seldom
    ids = (rank * vocab).long().clamp(max=vocab - 1)
    target = after[ids]
    target[torch.rand(tokens, generator=g, device="cuda") < 0.1] = -100
    ids[-tokens // 16:] = -1
    target[-tokens // 16:] = -100
    return ids, target


def gradients(p, ids, target):
    """One forward and backward: (mean loss, gradients by name, what the forward left)."""
    vocab, width = p["table"]["w"].shape
    table, scale = p["table"]["w"], width ** 0.5
    q = sbl.quant_weights(p["layer"]["w"], N, M, FMT, want_codes=True)

    x = sbl.embed(ids, table, scale=scale, dtype=torch.float32)
    xq, gamma, xn, mean1, rstd1 = sbl.norm_quant(x, p["norm1"]["w"], p["bias1"]["w"])
    y, _ = sbl.linear(q["packed"], q["meta"], FMT, N, M, q["beta"], xq, gamma, width)
    r = x + y
    h, mean2, rstd2 = sbl.norm(r, p["norm2"]["w"], p["bias2"]["w"], dtype=torch.bfloat16)
    loss, lse = sbl.head_ce(h, table, target)
    kept = (target >= 0).sum().clamp(min=1)

    dh, dtable = sbl.head_ce_backward(h, table, target, lse, torch.ones_like(loss) / kept)
    dr, dnorm2, dbias2 = sbl.norm_backward(dh, r, mean2, rstd2, p["norm2"]["w"], want_bias=True)
    dxn, dlayer = torch.empty_like(xn), torch.empty((width, width), device="cuda")
    dy = dr.bfloat16()
    sbl.sbl_linear_backward(dy, q["packed"], q["meta"], FMT, N, M, q["beta"], xn, xq, gamma, dx=dxn, dw=dlayer)
    dx, dnorm1, dbias1 = sbl.norm_backward(dxn, x, mean1, rstd1, p["norm1"]["w"], want_bias=True)
    sbl.embed_backward(ids, dx + dr, vocab, scale=scale, add_to=dtable)
    grads = dict(table=dtable, layer=dlayer, norm1=dnorm1, bias1=dbias1, norm2=dnorm2, bias2=dbias2)
    return loss.sum() / kept, grads, dict(x=x, xq=xq, gamma=gamma, xn=xn, r=r, h=h, dh=dh, dy=dy, codes=q["codes"],
                                          beta=q["beta"], lse=lse)


def train(steps=40, tokens=512, width=256, vocab=1000, rate=5e-3, clip=1.0, seed=0):
    """Mean loss of every step."""
    p, (ids, target) = model(width, vocab, seed), data(tokens, vocab, seed)
    items, schedule, losses = None, torch.zeros(5, device="cuda"), []
    for step in range(1, steps + 1):
        loss, grads, _ = gradients(p, ids, target)
        losses.append(loss)
        if items is None:
            items = sbl.AdamWItems([dict(e, g=grads[name]) for name, e in p.items()])
        for i, name in enumerate(p):
            items.set_gradient(i, grads[name])
        # the clipping factor stays on the GPU: the step reads it from the schedule
        norm = torch.stack([g.float().norm() for g in grads.values()]).norm()
        schedule.copy_(sbl.adamw_schedule(rate, ADAM["beta1"], ADAM["beta2"], step))
        schedule[3] = clip / norm.clamp(min=clip)
        sbl.sbl_adamw_batch(items, rate, **ADAM, step=step, schedule=schedule)
    return [float(x) for x in losses]


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    a.add_argument("--steps", type=int, default=40)
    a.add_argument("--tokens", type=int, default=512)
    a.add_argument("--width", type=int, default=256)
    a.add_argument("--vocab", type=int, default=1000)
    a = a.parse_args()
    for i, loss in enumerate(train(a.steps, a.tokens, a.width, a.vocab)):
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i:3d}  cross entropy {loss:.4f}", flush=True)


if __name__ == "__main__":
    main()
