"""The losses of the output head, measured: softmax cross entropy over a large
vocabulary and distillation from a teacher's top logits, each taken straight
from the hidden states and the head's weights (the logits are not an input),
forward and backward.

With z[t][v] = sum_d h[t][d] w[v][d]:

  cross entropy   lse[t] = log sum_v exp z[t][v],  loss[t] = lse[t] - z[t][target[t]]
                  dz = (dloss + dlse) softmax(z) - dloss [v = target]
                  a negative target takes its row out: loss = lse = 0, no gradient
  distillation    p[t] = softmax over the listed entries of teacher[t] / tau,
                  lse[t] = log sum_v exp(z[t][v] / tau),
                  loss[t] = tau^2 sum_k p[t][k] (log p[t][k] - z[t][index[t][k]] / tau + lse[t])
                  dz = dloss tau (softmax(z / tau) - sum_k p[k] [v = index[k]])
                  a negative index is no entry; a row without entries is taken out
  both            dh = dz w,  dw = dz^T h

Where `own` is false, `run` is the plain form: elementary torch operations in
32 bits, rounded once at the end.  Where it is true, `run` makes the calls of
this repository's package.
"""

import math
import random

import torch

own = False

OPS = ("ce_fwd", "ce_bwd", "kd_fwd", "kd_bwd")
MOST_WORK = 8.0e12          # products (tokens x vocab x width, three more times backward) of the largest case


def listed():
    """Hidden sizes are those of the transformer blocks this repository works
    on (256, 1536, 3200, 5120, 8192); vocabularies are a small one, two usual
    ones and an odd one."""
    return [
        # a unit-sized head: the latency of a call
        dict(name="ce_fwd_unit", op="ce_fwd", tokens=16, vocab=1000, width=256, dtype="bfloat16", out=0.0),
        # the likelihood of one token after a decode step: the head's weights are read once
        dict(name="ce_fwd_1tok", op="ce_fwd", tokens=1, vocab=32000, width=3200, dtype="bfloat16", out=0.0),
        # scoring a ragged batch: odd sizes, half of it prompt (taken out)
        dict(name="ce_fwd_ragged", op="ce_fwd", tokens=777, vocab=50257, width=1536, dtype="float16", out=0.5),
        # a training step's forward at a middle size
        dict(name="ce_fwd_block", op="ce_fwd", tokens=2048, vocab=32000, width=3200, dtype="bfloat16", out=0.02),
        dict(name="ce_bwd_unit", op="ce_bwd", tokens=16, vocab=1000, width=256, dtype="bfloat16", out=0.0),
        # per-token weights and a gradient into lse (a penalty on it), odd sizes
        dict(name="ce_bwd_ragged", op="ce_bwd", tokens=777, vocab=50257, width=1544, dtype="float16", out=0.25),
        dict(name="ce_bwd_block", op="ce_bwd", tokens=2048, vocab=32000, width=3200, dtype="bfloat16", out=0.02),
        # a training step's backward with a large vocabulary
        dict(name="ce_bwd_large", op="ce_bwd", tokens=4096, vocab=128256, width=5120, dtype="bfloat16", out=0.02),
        # a few tokens of an online student
        dict(name="kd_fwd_few", op="kd_fwd", tokens=64, vocab=32000, width=1536, dtype="bfloat16", out=0.0, top=8, tau=1.0),
        # forward with a wide head and a large vocabulary
        dict(name="kd_fwd_large", op="kd_fwd", tokens=4096, vocab=128256, width=8192, dtype="bfloat16", out=0.02, top=64, tau=2.0),
        # a handful of tokens, odd sizes, backward
        dict(name="kd_bwd_few", op="kd_bwd", tokens=37, vocab=32003, width=1536, dtype="bfloat16", out=0.1, top=20, tau=1.0),
        dict(name="kd_bwd_block", op="kd_bwd", tokens=2048, vocab=32000, width=3200, dtype="bfloat16", out=0.02, top=64, tau=2.0),
    ]


def _products(case):
    return float(case["tokens"]) * case["vocab"] * case["width"] * (3 if case["op"].endswith("bwd") else 1)


def draw(rng):
    def log_uniform(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    case = dict(op=rng.choice(OPS), tokens=log_uniform(1, 4096), vocab=log_uniform(500, 128256),
                width=8 * log_uniform(8, 1024), dtype=rng.choice(("bfloat16", "bfloat16", "float16")),
                out=rng.choice((0.0, 0.02, 0.5)))
    if case["op"].startswith("kd"):
        case.update(top=log_uniform(1, 128), tau=rng.choice((1.0, 2.0, 4.0)))
    while _products(case) > MOST_WORK:
        case["tokens"] = case["tokens"] // 2
    return case


def prepare(case, seed):
    """Hidden states as a final normalisation leaves them, head weights whose
    logits have a standard deviation of 2, and tokens that the head has in
    part learned: a random share of each target's row (cross entropy) is in
    its token's hidden state."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, v, d = case["tokens"], case["vocab"], case["width"]
    dtype = getattr(torch, case["dtype"])
    w32 = torch.randn(v, d, generator=g, device="cuda") * (2.0 / math.sqrt(d))
    h32 = torch.randn(t, d, generator=g, device="cuda")
    learned = torch.rand(t, 1, generator=g, device="cuda") * 3.0
    out = torch.rand(t, generator=g, device="cuda") < case["out"]
    s = dict(op=case["op"], dtype=dtype)
    if case["op"].startswith("ce"):
        target = torch.randint(0, v, (t,), generator=g, device="cuda")
        h32 += learned * w32[target]
        s["target"] = torch.where(out, torch.full_like(target, -100), target)
    else:
        top = case["top"]
        gap = max(1, v // top)          # distinct entries: one in each of `top` stretches of the vocabulary
        start = torch.randint(0, v, (t, 1), generator=g, device="cuda")
        inside = torch.randint(0, gap, (t, top), generator=g, device="cuda")
        index = (start + gap * torch.arange(top, device="cuda") + inside) % v
        h32 += learned * w32[index[:, 0]]
        teacher = torch.randn(t, top, generator=g, device="cuda") * 2.0
        teacher = 6.0 + teacher.sort(dim=1, descending=True).values
        listed_ = torch.randint(1, top + 1, (t, 1), generator=g, device="cuda")
        some = torch.rand(t, 1, generator=g, device="cuda") < 0.25    # a quarter of the rows list fewer entries
        absent = some & (torch.arange(top, device="cuda") >= listed_)
        s["index"] = torch.where(absent | out[:, None], torch.full_like(index, -1), index).contiguous()
        s["teacher"] = teacher.contiguous()
        s["tau"] = case["tau"]
    s["h"], s["w"] = h32.to(dtype), w32.to(dtype)
    del w32, h32
    if case["op"].endswith("bwd"):
        kept = (~out).sum().clamp(min=1)
        scale = 1024.0 if dtype == torch.float16 else 1.0              # loss scaling, as 16-bit training uses it
        weight = torch.ones(t, device="cuda")
        if t % 2:                                                      # odd token counts: per-token weights
            weight = 0.25 + torch.rand(t, generator=g, device="cuda")
        s["dloss"] = weight * (scale / kept)
        z = s["h"].float() @ s["w"].float().T
        if case["op"] == "ce_bwd":
            s["lse"] = torch.where(out, torch.zeros(()).cuda(), torch.logsumexp(z, 1))
            s["dlse"] = 2e-3 * s["lse"] * s["dloss"] if t % 2 else None
        else:
            s["lse"] = torch.where(out, torch.zeros(()).cuda(), torch.logsumexp(z / case["tau"], 1))
    return s


# ------------------------------------------------------------------ the plain form

def _lse(z):
    top = z.max(dim=1, keepdim=True).values
    return (top + (z - top).exp().sum(dim=1, keepdim=True).log())[:, 0]


def _teacher(s):
    has = s["index"] >= 0
    row = has.any(dim=1)
    a = torch.where(has, s["teacher"] / s["tau"], torch.full_like(s["teacher"], -math.inf))
    top = torch.where(row[:, None], a.max(dim=1, keepdim=True).values, torch.zeros_like(a[:, :1]))
    e = (a - top).exp()
    total = torch.where(row[:, None], e.sum(dim=1, keepdim=True), torch.ones_like(a[:, :1]))
    return has, row, e / total, torch.where(has, a - top - total.log(), torch.zeros_like(a))


def _plain(s):
    h, w, op = s["h"].float(), s["w"].float(), s["op"]
    z = h @ w.T
    if op.startswith("ce"):
        row = s["target"] >= 0
        at = s["target"].clamp(min=0)[:, None]
        if op == "ce_fwd":
            lse = _lse(z)
            loss = lse - z.gather(1, at)[:, 0]
            return torch.where(row, loss, torch.zeros_like(loss)), torch.where(row, lse, torch.zeros_like(lse))
        dloss = s["dloss"]
        both = dloss if s["dlse"] is None else dloss + s["dlse"]
        dz = (z - s["lse"][:, None]).exp() * both[:, None]
        dz = dz.scatter_add(1, at, -dloss[:, None])
    else:
        has, row, p, logp = _teacher(s)
        at = s["index"].clamp(min=0)
        z = z / s["tau"]
        if op == "kd_fwd":
            lse = _lse(z)
            each = p * (logp - z.gather(1, at) + lse[:, None])
            loss = s["tau"] ** 2 * torch.where(has, each, torch.zeros_like(each)).sum(dim=1)
            return torch.where(row, loss, torch.zeros_like(loss)), torch.where(row, lse, torch.zeros_like(lse))
        dz = (z - s["lse"][:, None]).exp().scatter_add(1, at, -p) * (s["dloss"] * s["tau"])[:, None]
    dz = torch.where(row[:, None], dz, torch.zeros_like(dz))
    return (dz @ w).to(s["dtype"]), (dz.T @ h).to(s["dtype"])


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    if not own:
        return _plain(s)
    from sparse_linear_layers_absmean_amd import sbl
    if s["op"] == "ce_fwd":
        return sbl.head_ce(s["h"], s["w"], s["target"])
    if s["op"] == "ce_bwd":
        return sbl.head_ce_backward(s["h"], s["w"], s["target"], s["lse"], s["dloss"], dlse=s["dlse"])
    if s["op"] == "kd_fwd":
        return sbl.head_kd(s["h"], s["w"], s["index"], s["teacher"], s["tau"])
    return sbl.head_kd_backward(s["h"], s["w"], s["index"], s["teacher"], s["tau"], s["lse"], s["dloss"])


def work(case):
    # rows that are taken out need no work: the expected number of others counts
    t, v, d = max(1, round(case["tokens"] * (1.0 - case["out"]))), case["vocab"], case["width"]
    small = t * (8 + 4 + 4) if case["op"].startswith("ce") else t * (12 * case["top"] + 8)
    if case["op"].endswith("bwd"):
        # the logits once more, then the two gradients; h, w, dh and dw once each
        return {"bytes": 2 * (2 * t * d + 2 * v * d) + small, "flops": 6 * t * v * d}
    return {"bytes": 2 * (t * d + v * d) + small, "flops": 2 * t * v * d}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    """Row block by row block, from log-probabilities (not from the plain form's exponentials)."""
    s = prepare(case, seed)
    h, w = s["h"].double(), s["w"].double()
    t, v = h.shape[0], w.shape[0]
    tau = float(case.get("tau", 1.0))
    backward = case["op"].endswith("bwd")
    loss, lse = torch.zeros(t, dtype=torch.float64, device="cuda"), torch.zeros(t, dtype=torch.float64, device="cuda")
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    for r in range(0, t, 1024):
        b = slice(r, min(t, r + 1024))
        logq = (h[b] @ w.t()) / tau
        norm = torch.logsumexp(logq, dim=1) if not backward else s["lse"][b].double()
        logq -= norm[:, None]
        # the wanted distribution over the vocabulary, and its entropy term
        want = torch.zeros_like(logq)
        if case["op"].startswith("ce"):
            row = s["target"][b] >= 0
            n = torch.nonzero(row)[:, 0]
            want[n, s["target"][b][n]] = 1.0
            entropy = torch.zeros_like(norm)
        else:
            idx = s["index"][b]
            row = (idx >= 0).sum(dim=1) > 0
            logp = torch.log_softmax((s["teacher"][b].double() / tau).masked_fill(idx < 0, -math.inf), dim=1)
            n, k = torch.nonzero(idx >= 0, as_tuple=True)
            want.index_put_((n, idx[n, k]), logp[n, k].exp(), accumulate=True)
            entropy = torch.zeros_like(norm).index_put_((n,), logp[n, k].exp() * logp[n, k], accumulate=True)
        if not backward:
            loss[b] = tau * tau * (entropy - (want * logq).sum(dim=1)) * row
            lse[b] = norm * row
            continue
        weight = s["dloss"][b].double()[:, None] * tau
        more = s["dlse"][b].double()[:, None] if s.get("dlse") is not None else 0.0
        dz = (weight * (logq.exp() - want) + more * logq.exp()) * row[:, None]
        dh[b] = dz @ w
        dw += dz.t() @ h[b]
    return (dh, dw) if backward else (loss, lse)


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c, work(c))
