"""Embedding, norm with quantizer, Sparse-BitLinear layer, norm, tied head, all
backwards and AdamW together, as examples/train_step.py runs them: every
gradient against the formulas in 64 bits, the update against the oracle."""

import importlib.util
import math
import os

import numpy as np
import pytest

from conftest import ROOT
from gpu_util import oracle_weight_rows, say, to_np
from oracle import head_oracle as H
from oracle import sbl_oracle as O
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _np(t):
    return to_np(t.double())


@pytest.mark.parametrize("tokens,width,vocab", [(40, 64, 100), (300, 256, 1003), (1100, 320, 517)])
def test_gradients_of_a_step(example, tokens, width, vocab):
    """Against the formulas in 64 bits, with the roundings to BF16 that the step makes (h, dh, dy) at the same
    places: what is left are fp32 sums, some 1e-6 of each norm, and the BF16 values that these carry to the other
    neighbour, a step of 2^-7 for a share of some 1e-6 / 2^-9 of the values: in the norm 2^-7 sqrt(5e-4) = 1.8e-4 for
    each of the three.  The table's own rounding comes twice (the head's part, then the sum), 2^-8 each, after a dz in
    16 bits, 2^-8.  Above 64 tokens the head rounds dz for dh too: 2^-8 of dh in the norm, and the roundings of dh and
    dy then fall elsewhere, 2^-8 each."""
    import torch
    say(f"train_step gradients tokens={tokens} width={width} vocab={vocab}")
    p, (ids, target) = example.model(width, vocab, 3), example.data(tokens, vocab, 3)
    g = torch.Generator(device="cuda").manual_seed(5)
    for name in ("norm1", "bias1", "norm2", "bias2"):
        p[name]["w"] += 0.3 * torch.randn(width, generator=g, device="cuda")
    loss, grads, kept = example.gradients(p, ids, target)
    torch.cuda.synchronize()
    k = {name: _np(v) for name, v in kept.items()}
    w = {name: _np(e["w"]) for name, e in p.items()}
    t, goal, scale = to_np(ids), to_np(target), width ** 0.5

    def bf16(x):
        return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().double().numpy()

    # forward
    x = S.embed(t, w["table"], scale).astype(np.float64)
    assert np.array_equal(x, k["x"]) and not x[t < 0].any()
    m1, r1 = S.norm_stats(x, 1e-5)
    xn = (x - m1[:, None]) * r1[:, None] * w["norm1"] + w["bias1"]
    assert np.abs(xn - k["xn"]).max() <= 8 * S.U32 * (np.abs(xn).max() + np.abs(w["bias1"]).max())
    q, gamma = O.quant_acts(k["xn"].astype(np.float32))
    assert np.array_equal(q, k["xq"]) and np.array_equal(gamma, k["gamma"].astype(np.float32))
    master = to_np(p["layer"]["w"].view(torch.int16)).view(np.uint16)
    _, codes = oracle_weight_rows(master, O.absmean_beta(master), example.N, example.M)
    assert np.array_equal(codes, k["codes"])
    beta = float(O.beta_eff(O.absmean_beta(master)))
    xh = k["xq"] * np.maximum(k["gamma"], 1e-5)[:, None] / 128.0
    r = x + xh @ (codes.astype(np.float64) * beta).T
    m2, r2 = S.norm_stats(r, 1e-5)
    h = bf16((r - m2[:, None]) * r2[:, None] * w["norm2"] + w["bias2"])
    assert np.linalg.norm(h - k["h"]) <= 1.8e-4 * np.linalg.norm(h)
    want, row = H.wanted_ce(goal, vocab)
    rl, lse, _ = H.forward(h, w["table"], want, row, np.zeros(tokens))
    count = max(1, int(row.sum()))
    assert abs(float(loss) - rl.sum() / count) < 1e-3 * rl.sum() / count

    # backward
    dh, dt, _, _ = H.backward(h, w["table"], want, row, lse, np.full(tokens, 1.0 / count), None, dtype="bfloat16")
    dh = bf16(dh)
    (dr, dn2, db2), _ = S.norm_backward(dh, r, m2, r2, w["norm2"])
    dy = bf16(dr)
    passed = O.clip_pass(k["xn"].astype(np.float32), k["gamma"].astype(np.float32))
    dxn = beta * (dy @ codes.astype(np.float64)) * passed
    dl = dy.T @ xh
    (dx, dn1, db1), _ = S.norm_backward(dxn, x, m1, r1, w["norm1"])
    back = dx + dr
    total, _ = S.embed_backward(t, back, vocab, scale)
    for name, ref in dict(table=dt + total, layer=dl, norm1=dn1, bias1=db1, norm2=dn2, bias2=db2).items():
        got, norm = _np(grads[name]), np.linalg.norm(ref)
        off = np.linalg.norm(got - ref) / norm
        allowed = 3 * 1.8e-4 + 1e-5 + 3 * 2.0 ** -8 * ((name == "table") + (tokens > 64))
        assert off <= allowed, (name, off, allowed)
        assert norm > 0


def test_updates_of_steps(example):
    """Three steps: every update is the oracle's, bit for bit, from the gradients that the step computed; the next
    step's ternary codes are those of the new masters."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    p, (ids, target) = example.model(128, 300, 4), example.data(200, 300, 4)
    items = None
    for step in range(1, 4):
        _, grads, kept = example.gradients(p, ids, target)
        master = to_np(p["layer"]["w"].view(torch.int16)).view(np.uint16)
        assert np.array_equal(to_np(kept["codes"]), oracle_weight_rows(master, O.absmean_beta(master), 6, 8)[1])
        before = {n: {f: (v.clone() if isinstance(v, torch.Tensor) else v) for f, v in e.items()} for n, e in p.items()}
        if items is None:
            items = sbl.AdamWItems([dict(e, g=grads[n]) for n, e in p.items()])
        for i, name in enumerate(p):
            items.set_gradient(i, grads[name])
        sbl.sbl_adamw_batch(items, 1e-2, **example.ADAM, step=step)
        torch.cuda.synchronize()
        s = S.schedule(1e-2, example.ADAM["beta1"], example.ADAM["beta2"], step)
        for name, e in p.items():
            b = before[name]
            flat = lambda v: to_np(v.reshape(-1))                                                   # noqa: E731
            small = "m_scale" in b
            args = dict(m_scale=flat(b["m_scale"]), v_scale=flat(b["v_scale"])) if small else {}
            m, v = ((flat(b[f].view(torch.uint8)) if small else flat(b[f])) for f in ("m", "v"))
            w = flat(sbl.join_master(b["w"], b["w_low"])) if "w_low" in b else flat(b["w"])
            got = S.adamw(w, flat(grads[name].float()), m, v, s, example.ADAM["beta1"], example.ADAM["beta2"],
                          example.ADAM["eps"], 1.0, b.get("weight_decay", 0.0), **args)
            now = flat(sbl.join_master(e["w"], e["w_low"])) if "w_low" in e else flat(e["w"])
            assert np.array_equal(now, got[0]), name
            for f, x in zip(("m", "v", "m_scale", "v_scale"), got[1:]):
                assert np.array_equal(flat(e[f].view(torch.uint8)) if x.dtype == np.uint8 else flat(e[f]), x), (name, f)


def test_example_runs_and_repeats(example):
    losses = example.train(steps=6, tokens=200, width=128, vocab=300)
    assert len(losses) == 6 and all(math.isfinite(x) for x in losses)
    assert losses == example.train(steps=6, tokens=200, width=128, vocab=300)
