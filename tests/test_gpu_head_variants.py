"""Losses of the output head on the GPU at sizes that reach every variant of its
products (tiles, loads and stores past the caches, shares of dh, several ranges
of the vocabulary), element by element against 64 bits on the GPU within the
oracle's bounds (oracle/head_oracle.py has their derivation).  Every tile of ids
holds some token's target or listed ids, so that none can be left out unseen."""

import pytest

from gpu_util import say
from oracle import head_oracle as H

pytestmark = pytest.mark.gpu

BLOCK = 16384                          # ids at a time of the reference


def _tokens(t, d, v, dtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(t, d, generator=g, device="cuda").to(getattr(torch, dtype))
    w = (torch.randn(v, d, generator=g, device="cuda") * (2.0 / d ** 0.5)).to(getattr(torch, dtype))
    gone = torch.rand(t, generator=g, device="cuda") < 0.1
    gone[0] = gone[t - 1] = False
    h[gone] = float("nan")
    return g, h, w, gone


def _spread(g, n, v):
    """n ids, one in each of n equal stretches of the vocabulary (the last id among
    them), in random order."""
    import torch
    ids = (torch.arange(n, device="cuda") * v) // n + torch.randint(0, max(1, v // n), (n,), generator=g, device="cuda")
    ids[-1] = v - 1
    return ids[torch.randperm(n, generator=g, device="cuda")]


def _within(got, want, bound, name):
    import torch
    got = got.double()
    off = (got - want).abs() - bound
    assert bool(torch.isfinite(got).all()), name
    assert not bool((off > 0).any()), (name, float(off.max()), int((off > 0).sum()))


def _check(h, w, keep, rows, ids, share, entropy, tau, got, dloss, dlse, dtype, slack):
    """got = (loss, lse, dh, dw); (rows, ids, share): the wanted distribution's entries,
    rows among those kept; slack: error of each share relative to it."""
    import torch
    loss, lse, dh, dw = got
    u, tiny, few = H.U16[dtype], H.TINY16[dtype], len(h) <= 64
    hk, n, d, v = h[keep].double(), int(keep.sum()), h.shape[1], w.shape[0]
    s, g = lse[keep].double(), dloss[keep].double() * tau
    more = torch.zeros_like(g) if dlse is None else dlse[keep].double() * tau
    zero = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")
    rh, eh, top, ez_top, wz, total = zero(n, d), zero(n, d), zero(n), zero(n), zero(n), zero(n, 0)
    base = float(g.abs().max() + (g + more).abs().max())
    sums = []
    for i in range(0, v, BLOCK):
        wi = w[i:i + BLOCK].double()
        wa = wi.abs()
        z = hk @ wi.t() / tau
        ez = (d + 1) * H.U32 * (hk.abs() @ wa.t()) / tau
        want, err = zero(n, len(wi)), zero(n, len(wi))
        here = (ids >= i) & (ids < i + len(wi))
        want.index_put_((rows[here], ids[here] - i), share[here], accumulate=True)
        err.index_put_((rows[here], ids[here] - i), share[here] * slack[rows[here]], accumulate=True)
        sums.append(torch.logsumexp(z, 1))
        top = torch.maximum(top, z.abs().max(1).values)
        ez_top = torch.maximum(ez_top, ez.max(1).values)
        wz += (want * z).sum(1)
        first = (g + more)[:, None] * torch.exp(z - s[:, None])
        second = g[:, None] * want
        dz = first - second
        # the rounding of dz to 16 bits; up to 64 tokens a second part holds what it left
        e = (u * u if few else u) * dz.abs()
        e += first.abs() * (2 * ez + 64 * H.U32 * (1 + s.abs()[:, None] + z.abs()))
        e += 64 * H.U32 * (first.abs() + second.abs()) + g.abs()[:, None] * err + 2.0 ** -38 * base
        e *= 1 + 2 * u
        rh += dz @ wi
        eh += e @ wa + (v + 8) * H.U32 * ((dz.abs() + e) @ wa)
        rw = dz.t() @ hk
        ew = e.t() @ hk.abs() + (n + 8) * H.U32 * ((dz.abs() + e).t() @ hk.abs())
        _within(dw[i:i + BLOCK], rw, ew + u * (rw.abs() + ew) + tiny, f"dw from {i}")
    _within(dh[keep], rh, eh + u * (rh.abs() + eh) + tiny, "dh")
    assert not dh[~keep].any() and not loss[~keep].any() and not lse[~keep].any()
    ref = torch.logsumexp(torch.stack(sums, 1), 1)
    bound = 2 * ez_top + 64 * H.U32 * (1 + ref.abs() + top)
    _within(lse[keep], ref, bound, "lse")
    _within(loss[keep], tau * tau * (entropy - wz + ref), tau * tau * (bound + slack), "loss")


# tokens, ids, features: which variant
SIZES = [
    (20, 140001, 1024),     # up to 32 tokens; w, dw and the loads past the caches
    (50, 140001, 1024),     # up to 64
    (40, 140001, 1032),     # rows of dw that are no whole lines
    (64, 33000, 1032),      # the 128 x 64 logits tile, 17 steps
    (128, 33000, 1032),     # the 256 x 128 one
    (1500, 20000, 1032),    # dh on 256 x 128
    (777, 50257, 328),      # an odd vocabulary, a last step of 8 features
    (4100, 70007, 520),     # two ranges, dh on 256 x 256 added to, dw on 128 x 128
    (4100, 70007, 1032),    # both gradients in one launch, two ranges
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("t,v,d", SIZES)
def test_cross_entropy_variants(t, v, d, dtype):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"head_ce variants t={t} v={v} d={d} {dtype}")
    g, h, w, gone = _tokens(t, d, v, dtype, 31)
    target = torch.where(gone, torch.full((t,), -100, device="cuda"), _spread(g, t, v))
    up = 512.0 if dtype == "float16" else 1.0
    dloss = (torch.rand(t, generator=g, device="cuda") + 0.5) * up / t
    dlse = torch.randn(t, generator=g, device="cuda") * 0.1 * up / t
    loss, lse = sbl.head_ce(h, w, target)
    dh, dw = sbl.head_ce_backward(h, w, target, lse, dloss, dlse=dlse)
    torch.cuda.synchronize()
    n = int((~gone).sum())
    ones, none = torch.ones(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    _check(h, w, ~gone, torch.arange(n, device="cuda"), target[~gone], ones, none, 1.0, (loss, lse, dh, dw), dloss, dlse,
           dtype, none)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("t,v,d,crowd", [(*size, 0) for size in SIZES + [(4100, 70007, 128)]] +
                         # a later range's tile with more listed ids than it keeps apart: 512 up to 64 tokens, then 1024
                         [(40, 2500000, 64, 2400000), (4100, 70007, 128, 50000)])
def test_distillation_variants(t, v, d, crowd, dtype):
    """20 listed ids, some absent (by id or by logit, past the vocabulary too), some listed
    twice; spread over the vocabulary, or all among 128 ids from `crowd` on."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    top, tau = 20, 2.0
    say(f"head_kd variants t={t} v={v} d={d} crowd={crowd} {dtype}")
    g, h, w, gone = _tokens(t, d, v, dtype, 32)
    index = crowd + _spread(g, t * top, 128 if crowd else v).view(t, top)
    index[:, 7] = index[:, 3]
    teacher = torch.randn(t, top, generator=g, device="cuda") * 2
    absent = torch.rand(t, top, generator=g, device="cuda") < 0.2
    absent[:, 0] = False
    absent |= gone[:, None]
    by_id = torch.rand(t, top, generator=g, device="cuda") < 0.5
    index[absent & by_id] = -1
    index[absent & ~by_id] += v // 2
    teacher[absent & ~by_id] = -float("inf")
    up = 512.0 if dtype == "float16" else 1.0
    dloss = (torch.rand(t, generator=g, device="cuda") + 0.5) * up / t
    loss, lse = sbl.head_kd(h, w, index, teacher, tau)
    dh, dw = sbl.head_kd_backward(h, w, index, teacher, tau, lse, dloss)
    torch.cuda.synchronize()
    keep = ~gone
    logp = torch.log_softmax((teacher.double() / tau).masked_fill(absent, -float("inf"))[keep], 1)
    p = logp.exp()
    rows, k = torch.nonzero(~absent[keep], as_tuple=True)
    entropy = torch.zeros(len(p), dtype=torch.float64, device="cuda").index_put_(
        (rows,), p[rows, k] * logp[rows, k], accumulate=True)
    # the teacher's probabilities are fp32: differences of logits, an exponential, a sum, a quotient
    slack = 64 * H.U32 * (1 + logp.masked_fill(absent[keep], 0.0).abs().max(1).values)
    _check(h, w, keep, rows, index[keep][rows, k], p[rows, k], entropy, tau, (loss, lse, dh, dw), dloss, None, dtype, slack)
