"""Losses of the output head on the GPU where their sizes end: vocabularies of
tens of millions of ids, launches of more workgroups than one grid holds, and
the gradients of an empty batch."""

import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu


def test_gradients_of_a_vocabulary_of_tens_of_millions():
    """One token, 40 million ids.  Every id but the target has features 0 or 1/2
    (the target none), so each feature of dh is a sum of positive terms: in fp32,
    of fewer than 1000 roundings one after the other, with logit gradients of
    2^-16 or better, it is off by less than 2^-12, and its rounding to BF16 by 2^-9."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    t, v, d, y = 1, 40000000, 8, 17
    say(f"head_ce wide vocabulary t={t} v={v} d={d}")
    g = torch.Generator(device="cuda").manual_seed(21)
    w = torch.randint(0, 2, (v, d), generator=g, device="cuda", dtype=torch.int8).bfloat16() * 0.5
    n = torch.arange(v, device="cuda")
    w[:, 5] = (n >= (1 << 25)) * 0.5                 # where features of the first ids say nothing
    w[:, 6] = (n < 512) * 0.5
    w[:, 7] = (n >= v - 100) * 0.5
    w[y] = 0
    h = torch.tensor([[1.0, -2.0, 0.5, 3.0, -1.0, 2.0, 1.5, -0.5]], device="cuda").bfloat16()
    target = torch.tensor([y], device="cuda")
    loss, lse = sbl.head_ce(h, w, target)
    dloss = torch.ones(1, device="cuda")
    dh, dw = sbl.head_ce_backward(h, w, target, lse, dloss)
    torch.cuda.synchronize()
    z = torch.zeros(v, dtype=torch.float64, device="cuda")
    for i in range(d):
        z += w[:, i].double() * h[0, i].double()
    ref = torch.logsumexp(z, 0)
    assert abs(float(lse[0].double() - ref)) < 1e-4 and abs(float(loss[0].double() - ref)) < 1e-4
    q = torch.exp(z - lse[0].double())
    for i in range(d):
        want = (q * w[:, i].double()).sum()
        assert abs(float(dh[0, i].double() - want)) <= 2.0 ** -8 * float(want), (i, float(dh[0, i]), float(want))
    q[y] -= 1
    for i in range(d):
        want = q * h[0, i].double()
        assert bool(((dw[:, i].double() - want).abs() <= 2.0 ** -8 * want.abs()).all()), i


def test_a_product_of_more_workgroups_than_one_grid():
    """2^18 tokens over more than 2^21 ids: over 2^32 threads in all.  64 of the rows
    against 64 bits, within the oracle's bound of a 32-bit evaluation."""
    import torch
    from oracle import head_oracle as H
    from sparse_linear_layers_absmean_amd import sbl
    t, v, d = 1 << 18, (1 << 21) + 77, 8
    say(f"head_ce many tiles t={t} v={v} d={d}")
    g = torch.Generator(device="cuda").manual_seed(22)
    h = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    w = torch.randn(v, d, generator=g, device="cuda").bfloat16()
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    rows = torch.cat([torch.tensor([0, 1, t - 2, t - 1], device="cuda"),
                      torch.randint(0, t, (60,), generator=g, device="cuda")])
    target[rows[:4]] = torch.tensor([0, v - 1, v - 77, v - 78], device="cuda")
    loss, lse = sbl.head_ce(h, w, target)
    torch.cuda.synchronize()
    assert bool(lse.isfinite().all()) and bool(loss.isfinite().all())
    hr, wd = h[rows].double(), w.double()
    z = hr @ wd.t()
    ref = torch.logsumexp(z, 1)
    picked = z.gather(1, target[rows][:, None])[:, 0]
    ez = (d + 1) * H.U32 * (hr.abs() @ wd.abs().t()).max(dim=1).values
    bound = 2 * ez + 64 * H.U32 * (1 + ref.abs() + z.abs().max(dim=1).values)
    assert bool(((lse[rows].double() - ref).abs() <= bound).all())
    assert bool(((loss[rows].double() - (ref - picked)).abs() <= bound).all())


def test_no_tokens_zero_a_large_gradient_quickly():
    """An empty batch's dw (525 MB): zero everywhere, nothing beside it written, and at
    no less than a tenth of what a fill of the same size takes."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v, d = 64001, 4104
    say(f"head_ce no tokens v={v} d={d}")
    h = torch.empty((0, d), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((v, d), dtype=torch.bfloat16, device="cuda")
    none = torch.empty((0,), dtype=torch.float32, device="cuda")
    target = torch.empty((0,), dtype=torch.int64, device="cuda")
    room = torch.full((v + 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = sbl.new_head_workspace(0, v, d, backward=True)

    def call():
        sbl.sbl_head_ce_backward(h, w, target, none, none, None, room[1:v + 1], ws)

    def took(f):
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            f()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    call()
    torch.cuda.synchronize()
    assert not room[1:v + 1].any() and bool((room[0] == 7).all()) and bool((room[v + 1] == 7).all())
    mine, fill = took(call), took(lambda: w.fill_(0.0))
    say(f"zeroed in {mine * 1e3:.0f} us, a fill takes {fill * 1e3:.0f}")
    assert mine < 10 * fill


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_the_most_tokens(dtype):
    """2^22 tokens: logit gradients of 2 GiB in each of two ranges of the vocabulary,
    hidden states read in 65536 steps.  Every row of dh and dw within the oracle's
    bounds; a sum over the tokens has one rounding per 32 of them, and 40 more."""
    import torch
    from oracle import head_oracle as H
    from sparse_linear_layers_absmean_amd import sbl
    t, v, d = 1 << 22, 300, 16
    say(f"head_ce many tokens t={t} v={v} d={d} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(23)
    h = torch.randn(t, d, generator=g, device="cuda").to(getattr(torch, dtype))
    w = (torch.randn(v, d, generator=g, device="cuda") * 0.5).to(getattr(torch, dtype))
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    target[torch.rand(t, generator=g, device="cuda") < 0.01] = -1
    target[0], target[t - 1] = v - 1, 0
    # FP16: a scale at which the sum over the tokens stays in its range
    dloss = (torch.rand(t, generator=g, device="cuda") + 0.5) * (2.0 ** -10 if dtype == "float16" else 2.0 ** -22)
    lse = sbl.head_ce(h, w, target)[1]
    dh, dw = sbl.head_ce_backward(h, w, target, lse, dloss)
    torch.cuda.synchronize()
    u, tiny = H.U16[dtype], H.TINY16[dtype]
    wd, base = w.double(), 2 * float(dloss.max())
    rw, sizes = torch.zeros(v, d, dtype=torch.float64, device="cuda"), torch.zeros(v, d, dtype=torch.float64, device="cuda")
    errors = torch.zeros_like(rw)
    for i in range(0, t, 1 << 18):
        b = slice(i, i + (1 << 18))
        hd, keep = h[b].double(), (target[b] >= 0).double()
        z = hd @ wd.t()
        ez = (d + 1) * H.U32 * (hd.abs() @ wd.abs().t())
        ref = torch.logsumexp(z, 1)
        bound = 2 * ez.max(1).values + 64 * H.U32 * (1 + ref.abs() + z.abs().max(1).values)
        s = lse[b].double()
        assert bool(((s - ref * keep).abs() <= bound).all())
        first = (dloss[b].double() * keep)[:, None] * torch.exp(z - s[:, None] - 100.0 * (1 - keep)[:, None])
        second = torch.zeros_like(first).scatter_(1, target[b].clamp(min=0)[:, None], (dloss[b].double() * keep)[:, None])
        dz = first - second
        e = u * dz.abs() + first * (2 * ez + 64 * H.U32 * (1 + s.abs()[:, None] + z.abs()))
        e = (e + 64 * H.U32 * (first + second) + 2.0 ** -38 * base * keep[:, None]) * (1 + 2 * u)
        want = dz @ wd
        err = e @ wd.abs() + (v + 8) * H.U32 * ((dz.abs() + e) @ wd.abs())
        off = (dh[b].double() - want).abs() - (err + u * (want.abs() + err) + tiny)
        assert not bool((off > 0).any()), (i, float(off.max()))
        rw += dz.t() @ hd
        errors += e.t() @ hd.abs()
        sizes += (dz.abs() + e).t() @ hd.abs()
    err = errors + (t / 32 + 40) * H.U32 * sizes
    off = (dw.double() - rw).abs() - (err + u * (rw.abs() + err) + tiny)
    assert bool(dw.isfinite().all()) and not bool((off > 0).any()), float(off.max())
