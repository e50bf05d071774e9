#!/usr/bin/env python3
"""Training steps of a Sparse-BitLinear layer under an output head: the layer's
forward, the head's cross entropy and its distillation from a teacher's top
logits, and the gradients of both back into the head and the layer's masters.

A step:
  masters (BF16)  -> quant_weights -> packed ternary 6:8 weights, beta
  x (fp32)        -> quant_acts    -> int8, gamma;  linear -> y (fp32), h = y in BF16
  head            -> head_ce, head_kd -> per-token losses; the logits are never stored
  backward        -> head_ce_backward, head_kd_backward -> dh, dw of the head
                     sbl_linear_backward(dh)            -> gradient of the masters
  both            -> a step of the optimizer on fp32 copies

The data are synthetic: x is random, the teacher is a dense linear map of x,
the targets are its most likely ids, and a tenth of the tokens is taken out.

  python examples/train_head.py [--steps 40] [--tokens 512] [--width 256] [--vocab 1000]
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


def train(steps=40, tokens=512, width=256, vocab=1000, top=8, tau=2.0, mix=0.5, rate=5e-3, seed=0):
    """[(mean cross entropy, mean distillation loss)] of every step."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    x = normal(tokens, width)
    z = x @ (normal(vocab, width) * (3.0 / width ** 0.5)).T
    teacher, index = z.topk(top, dim=1)
    target = index[:, 0].contiguous()
    gone = torch.rand(tokens, generator=g, device="cuda") < 0.1
    target[gone] = -100
    index = torch.where(gone[:, None], torch.full_like(index, -1), index)
    kept = (~gone).sum().clamp(min=1)

    layer = normal(width, width) / width ** 0.5      # fp32 copies of the masters and of the head
    head = normal(vocab, width) * (0.5 / width ** 0.5)
    optimizer = torch.optim.Adam([layer, head], lr=rate)
    # scratch, kept from step to step
    forward = sbl.new_head_workspace(tokens, vocab, width, top)
    backward = sbl.new_head_workspace(tokens, vocab, width, top, backward=True)
    layer_ws = sbl.new_backward_workspace(tokens, width, width)
    share = torch.full((tokens,), 1.0, device="cuda") / kept        # of each token in the mean
    dlayer = torch.empty_like(layer)

    xq, gamma = sbl.quant_acts(x)
    losses = []
    for _ in range(steps):
        q = sbl.quant_weights(layer.bfloat16(), N, M, FMT)
        y, _ = sbl.linear(q["packed"], q["meta"], FMT, N, M, q["beta"], xq, gamma, width)
        h, w = y.bfloat16(), head.bfloat16()

        ce, ce_lse = sbl.head_ce(h, w, target, workspace=forward)
        kd, kd_lse = sbl.head_kd(h, w, index, teacher, tau, workspace=forward)
        losses.append((ce.sum() / kept, kd.sum() / kept))

        dh1, dw1 = sbl.head_ce_backward(h, w, target, ce_lse, (1.0 - mix) * share, workspace=backward)
        dh2, dw2 = sbl.head_kd_backward(h, w, index, teacher, tau, kd_lse, mix * share, workspace=backward)
        sbl.sbl_linear_backward(dh1 + dh2, None, None, FMT, N, M, None, None, xq, gamma, dw=dlayer,
                                workspace=layer_ws)
        layer.grad, head.grad = dlayer, dw1.float() + dw2.float()
        optimizer.step()
    return [(float(a), float(b)) for a, b in losses]


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--steps", type=int, default=40)
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--width", type=int, default=256)
    p.add_argument("--vocab", type=int, default=1000)
    a = p.parse_args()
    losses = train(a.steps, a.tokens, a.width, a.vocab)
    for i, (ce, kd) in enumerate(losses):
        if i % 5 == 0 or i == len(losses) - 1:
            print(f"step {i:3d}  cross entropy {ce:.4f}  distillation {kd:.4f}", flush=True)


if __name__ == "__main__":
    main()
