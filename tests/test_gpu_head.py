"""Losses of the output head on the GPU against the 64-bit oracle: loss, lse, dh
and dw within the oracle's elementwise bounds, over tile edges, both 16-bit
types, rows that are taken out (with NaN in them), duplicate and absent
teacher entries, several ranges of the vocabulary, strides, streams, graphs
and dirty workspaces."""

import numpy as np
import pytest

from gpu_util import say, to_np
from oracle import head_oracle as H

pytestmark = pytest.mark.gpu

# tokens around the tile variants' edges (32, 64, 128, 256), vocabularies around
# 32, 128 and 256, features with and without a whole last step of 64
SHAPES = [(1, 1, 8), (1, 1000, 256), (3, 130, 72), (32, 500, 64), (33, 31, 136), (64, 1003, 128), (65, 257, 264),
          (128, 385, 72), (129, 640, 136), (257, 300, 64), (300, 1003, 200), (513, 777, 328),
          # vocabularies large enough for the larger tiles of each product
          (70, 33001, 136), (500, 32700, 72), (600, 9001, 1032)]
TYPES = ["bfloat16", "float16"]


def _half(x, dtype):
    """numpy -> GPU tensor of the 16-bit type, and its values back in float64."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(getattr(torch, dtype))
    return t.cuda(), t.double().numpy()


def _f32(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()


def _i64(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int64)).cuda()


def _inputs(t, v, d, dtype, seed, out=0.25):
    rng = np.random.default_rng(seed)
    h, hv = _half(rng.standard_normal((t, d)), dtype)
    w, wv = _half(rng.standard_normal((v, d)) * (2.0 / np.sqrt(d)), dtype)
    gone = rng.random(t) < out
    if t > 2:
        gone[1] = True
        gone[0] = False
    else:
        gone[:] = False
    h[_i64(np.nonzero(gone)[0])] = float("nan")      # must reach nothing
    return rng, h, hv, w, wv, gone


def _teacher(rng, t, v, top, gone):
    index = np.stack([rng.integers(0, v, top) for _ in range(t)])     # duplicates happen
    index[rng.random((t, top)) < 0.2] = -1
    index[~(index >= 0).any(axis=1), 0] = 0
    teacher = (rng.standard_normal((t, top)) * 3).astype(np.float32)
    low = rng.random((t, top)) < 0.1
    low[:, 0] = False
    index[:, 0] = np.maximum(index[:, 0], 0)
    teacher[low] = -np.inf
    index[gone] = -1 - (np.arange(top) % 3)
    return index, teacher


def _dirty(nbytes):
    import torch
    return torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")


def _near(got, want, bound, name):
    got = got.astype(np.float64)
    assert np.isfinite(got).all(), (name, int((~np.isfinite(got)).sum()))
    bad = np.abs(got - want) > bound
    assert not bad.any(), (name, int(bad.sum()), float((np.abs(got - want) - bound)[bad].max()),
                           [tuple(int(v) for v in x) for x in np.argwhere(bad)[:4]])


def _np(t):
    return to_np(t.float())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,v,d", SHAPES)
def test_cross_entropy_matches_oracle(t, v, d, dtype):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"head_ce t={t} v={v} d={d} {dtype}")
    rng, h, hv, w, wv, gone = _inputs(t, v, d, dtype, [70, t, v, d])
    target = rng.integers(0, v, t)
    target[gone] = -100
    want, row = H.wanted_ce(target, v)
    loss, lse = sbl.head_ce(h, w, _i64(target), workspace=_dirty(sbl.sbl_head_workspace_bytes(t, v, d)))
    torch.cuda.synchronize()
    rl, rs, bound = H.forward(hv, wv, want, row, np.zeros(t))
    _near(_np(loss), rl, bound * row, "loss")
    _near(_np(lse), rs, bound * row, "lse")
    up = 512.0 if dtype == "float16" else 1.0
    dloss = (rng.random(t) + 0.5) * up / t
    dlse = rng.standard_normal(t) * up / t
    dloss[gone] = np.nan                             # not used either
    for dl in (None, dlse):
        ws = _dirty(sbl.sbl_head_workspace_bytes(t, v, d, backward=True))
        dh, dw = sbl.head_ce_backward(h, w, _i64(target), lse, _f32(dloss), dlse=None if dl is None else _f32(dl),
                                      workspace=ws)
        torch.cuda.synchronize()
        rh, rw, eh, ew = H.backward(hv, wv, want, row, _np(lse), dloss.astype(np.float32),
                                    None if dl is None else dl.astype(np.float32), dtype=dtype)
        _near(_np(dh), rh, eh, "dh")
        _near(_np(dw), rw, ew, "dw")
        assert not _np(dh)[gone].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("top,tau", [(1, 1.0), (5, 2.0), (64, 4.0), (200, 0.5)])
@pytest.mark.parametrize("t,v,d", [(1, 1, 8), (3, 130, 72), (40, 1003, 128), (65, 257, 264), (300, 1003, 200),
                                   (500, 32700, 72)])
def test_distillation_matches_oracle(t, v, d, top, tau, dtype):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"head_kd t={t} v={v} d={d} top={top} tau={tau} {dtype}")
    rng, h, hv, w, wv, gone = _inputs(t, v, d, dtype, [71, t, v, d, top])
    index, teacher = _teacher(rng, t, v, top, gone)
    p, logp = H.teacher_probabilities(index, teacher, tau)
    want, row = H.wanted_kd(index, p, v)
    assert np.array_equal(row, ~gone)
    loss, lse = sbl.head_kd(h, w, _i64(index), _f32(teacher), tau,
                            workspace=_dirty(sbl.sbl_head_workspace_bytes(t, v, d, top)))
    torch.cuda.synchronize()
    rl, rs, bound = H.forward(hv, wv, want, row, H.entropy_of(p, logp), tau)
    # the teacher's logarithms: differences of fp32 logits, an exponential and a logarithm
    spread = np.abs(np.where(p > 0, logp, 0.0)).max(axis=1)
    _near(_np(loss), rl, tau * tau * (bound + 64 * H.U32 * (1 + spread)) * row, "loss")
    _near(_np(lse), rs, bound * row, "lse")
    up = 512.0 if dtype == "float16" else 1.0
    dloss = (rng.random(t) + 0.5) * up / t
    ws = _dirty(sbl.sbl_head_workspace_bytes(t, v, d, top, True))
    dh, dw = sbl.head_kd_backward(h, w, _i64(index), _f32(teacher), tau, lse, _f32(dloss), workspace=ws)
    torch.cuda.synchronize()
    # the teacher's probabilities are fp32 themselves: 64 U32 (1 + spread) of each
    rh, rw, eh, ew = H.backward(hv, wv, want, row, _np(lse), dloss.astype(np.float32), tau=tau, dtype=dtype)
    s = (tau * np.abs(dloss) * row * 64 * H.U32 * (1 + spread))[:, None] * want
    hz = np.where(row[:, None], np.abs(hv), 0.0)
    _near(_np(dh), rh, eh + 2 * s @ np.abs(wv), "dh")
    _near(_np(dw), rw, ew + 2 * s.T @ hz, "dw")


def _reference64(h, w, target, lse, dloss, dlse=None):
    """Cross entropy in 64 bits on the GPU, for sizes the NumPy oracle is slow at."""
    import torch
    z = h.double() @ w.double().t()
    q = torch.exp(z - lse.double()[:, None])
    dz = (dloss + (0 if dlse is None else dlse)).double()[:, None] * q
    dz[torch.arange(len(target)), target] -= dloss.double()
    return torch.logsumexp(z, 1), dz @ w.double(), dz.t() @ h.double()


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_several_ranges_of_the_vocabulary():
    """More than 2^28 logits: the backward takes the vocabulary in two ranges,
    and the last one is not a whole number of tiles."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    t, v, d = 4100, 70007, 128
    say(f"head_ce ranges t={t} v={v} d={d}")
    g = torch.Generator(device="cuda").manual_seed(5)
    h = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    w = (torch.randn(v, d, generator=g, device="cuda") * 0.2).bfloat16()
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    loss, lse = sbl.head_ce(h, w, target)
    dloss = torch.full((t,), 1.0 / t, device="cuda")
    dh, dw = sbl.head_ce_backward(h, w, target, lse, dloss)
    torch.cuda.synchronize()
    ref, rh, rw = _reference64(h, w, target, lse, dloss)
    assert float((lse.double() - ref).abs().max()) < 1e-4
    # one rounding of dz and one of the result, each at most 2^-8 relative, and
    # never all of them at once: 2^-8 in the norm
    assert _rel(dh, rh) < 2.0 ** -8 and _rel(dw, rw) < 2.0 ** -8


def test_weights_past_32_bit_offsets():
    """A head of more than 2^31 bytes (and 2^30 values): few tokens, every id
    of the far end present among the targets."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    t, v, d = 6, 140001, 8192
    say(f"head_ce wide t={t} v={v} d={d}")
    g = torch.Generator(device="cuda").manual_seed(6)
    h = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    w = torch.empty(v, d, dtype=torch.bfloat16, device="cuda")
    w.normal_(0, 0.02, generator=g)
    target = torch.tensor([0, v - 1, v - 2, 131071, 131072, 70000], device="cuda")
    loss, lse = sbl.head_ce(h, w, target)
    dloss = torch.full((t,), 0.25, device="cuda")
    dh, dw = sbl.head_ce_backward(h, w, target, lse, dloss)
    torch.cuda.synchronize()
    z = torch.cat([h.double() @ w[i:i + 16384].double().t() for i in range(0, v, 16384)], 1)
    ref = torch.logsumexp(z, 1)
    assert float((lse.double() - ref).abs().max()) < 1e-4
    assert float((loss.double() - (ref - z[torch.arange(t), target])).abs().max()) < 1e-4
    dz = 0.25 * torch.exp(z - lse.double()[:, None])
    dz[torch.arange(t), target] -= 0.25
    rh = sum(dz[:, i:i + 16384] @ w[i:i + 16384].double() for i in range(0, v, 16384))
    assert _rel(dh, rh) < 2.0 ** -8
    for i in range(0, v, 16384):
        assert _rel(dw[i:i + 16384], dz[:, i:i + 16384].t() @ h.double()) < 2.0 ** -8


@pytest.mark.parametrize("t", [5, 300])
def test_all_rows_taken_out(t):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    h = torch.full((t, 64), float("nan"), device="cuda").bfloat16()
    w = torch.randn(300, 64, device="cuda").bfloat16()
    target = torch.full((t,), -1, device="cuda")
    loss, lse = sbl.head_ce(h, w, target)
    dh, dw = sbl.head_ce_backward(h, w, target, lse, torch.ones(t, device="cuda"))
    assert not loss.any() and not lse.any() and not dh.any() and not dw.any()
    index = torch.full((t, 3), 7, device="cuda")
    teacher = torch.full((t, 3), -float("inf"), device="cuda")         # listed, but nothing left
    loss, lse = sbl.head_kd(h, w, index, teacher, 2.0)
    dh, dw = sbl.head_kd_backward(h, w, index, teacher, 2.0, lse, torch.ones(t, device="cuda"))
    assert not loss.any() and not lse.any() and not dh.any() and not dw.any()


def test_no_tokens():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    h = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.randn(300, 64, device="cuda").bfloat16()
    target = torch.empty((0,), dtype=torch.int64, device="cuda")
    loss, lse = sbl.head_ce(h, w, target)
    assert loss.shape == (0,)
    dh, dw = sbl.head_ce_backward(h, w, target, lse, loss)
    assert dh.shape == (0, 64) and dw.shape == w.shape and not dw.any()


@pytest.mark.parametrize("t", [7, 300])
def test_ids_past_the_vocabulary_show(t):
    """Their rows' loss is NaN and they leave the gradients; other rows are as if they were not there."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    h = torch.randn(t, 64, device="cuda").bfloat16()
    w = torch.randn(300, 64, device="cuda").bfloat16()
    target = torch.arange(t, device="cuda") % 300
    bad = target.clone()
    bad[3] = 300
    bad[5] = 2 ** 40
    out = target.clone()
    out[3] = out[5] = -1
    g = torch.ones(t, device="cuda")
    loss, lse = sbl.head_ce(h, w, bad)
    want, wlse = sbl.head_ce(h, w, out)
    keep = torch.ones(t, dtype=torch.bool, device="cuda")
    keep[3] = keep[5] = False
    assert loss[3].isnan() and loss[5].isnan() and torch.equal(loss[keep], want[keep])
    a, b = sbl.head_ce_backward(h, w, bad, lse, g), sbl.head_ce_backward(h, w, out, wlse, g)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and not a[0][~keep].any()
    index = torch.stack([target, (target + 9) % 300], 1)
    teacher = torch.randn(t, 2, device="cuda")
    bad, out = index.clone(), index.clone()
    bad[3, 1] = 300
    out[3] = -1
    loss, lse = sbl.head_kd(h, w, bad, teacher, 1.0)
    keep[5] = True
    want, wlse = sbl.head_kd(h, w, out, teacher, 1.0)
    assert loss[3].isnan() and torch.equal(loss[keep], want[keep])
    a = sbl.head_kd_backward(h, w, bad, teacher, 1.0, lse, g)
    b = sbl.head_kd_backward(h, w, out, teacher, 1.0, wlse, g)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("t", [20, 300])
def test_extreme_logits(t):
    """Logits of thousands (their exponentials would overflow), one id far above
    the rest, the teacher's lowest finite logits."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v, d = 500, 64
    g = torch.Generator(device="cuda").manual_seed(9)
    h = (torch.randn(t, d, generator=g, device="cuda") * 40).bfloat16()
    w = (torch.randn(v, d, generator=g, device="cuda") * 10).bfloat16()
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    loss, lse = sbl.head_ce(h, w, target)
    z = h.double() @ w.double().t()
    ref = torch.logsumexp(z, 1)
    # z of thousands, 64 exact products: 65 2^-24 sum|hw|, as the oracle's bound has it
    bound = 2 * 65 * H.U32 * (h.double().abs() @ w.double().abs().t()).max() + 64 * H.U32 * z.abs().max()
    assert float((lse.double() - ref).abs().max()) < float(bound)
    assert float((loss.double() - (ref - z.gather(1, target[:, None])[:, 0])).abs().max()) < float(bound)
    dh, dw = sbl.head_ce_backward(h, w, target, lse, torch.ones(t, device="cuda"))
    assert dh.isfinite().all() and dw.isfinite().all()
    index = target[:, None].repeat(1, 3)
    index[:, 1] = (target + 1) % v
    index[:, 2] = (target + 2) % v
    low = torch.finfo(torch.float32).min
    teacher = torch.full((t, 3), low, device="cuda")
    teacher[: t // 2, 0] = 1.0                        # one listed logit far above; else all equal and lowest
    loss, _ = sbl.head_kd(h, w, index, teacher, 0.5)
    q = torch.log_softmax(z / 0.5, 1).gather(1, index)
    p = torch.full((t, 3), 1 / 3, dtype=torch.float64, device="cuda")
    p[: t // 2] = torch.tensor([1.0, 0.0, 0.0], dtype=torch.float64, device="cuda")
    want = 0.25 * (torch.where(p > 0, p * (p.clamp(min=1e-300).log() - q), torch.zeros_like(p))).sum(1)
    assert float((loss.double() - want).abs().max()) < 0.25 * 2 * float(bound)


@pytest.mark.parametrize("t,k", [(5, 64), (300, 72)])
def test_row_stride_and_either_output(t, k):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v = 300
    wide = torch.randn(t, 2 * k + 8, device="cuda").bfloat16()
    wide[:, k:] = float("nan")
    h, hc = wide[:, :k], wide[:, :k].contiguous()
    w = torch.randn(v, k, device="cuda").bfloat16()
    target = torch.randint(0, v, (t,), device="cuda")
    a, b = sbl.head_ce(h, w, target), sbl.head_ce(hc, w, target)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    g = torch.rand(t, device="cuda")
    dh, dw = sbl.head_ce_backward(h, w, target, a[1], g)
    eh, ew = sbl.head_ce_backward(hc, w, target, a[1], g)
    assert torch.equal(dh, eh) and torch.equal(dw, ew)
    ws = sbl.new_head_workspace(t, v, k, backward=True)
    oh, ow = torch.full_like(hc, 7.0), torch.full_like(w, 7.0)
    sbl.sbl_head_ce_backward(h, w, target, a[1], g, oh, None, ws)
    assert torch.equal(oh, dh)
    sbl.sbl_head_ce_backward(h, w, target, a[1], g, None, ow, ws)
    assert torch.equal(ow, dw)
    # dw of the taken-in rows only, into the middle of a buffer whose edges stay as they are
    room = torch.full((v + 2, k), 7.0, device="cuda").bfloat16()
    sbl.sbl_head_ce_backward(h, w, target, a[1], g, None, room[1:v + 1], ws)
    assert torch.equal(room[1:v + 1], dw) and bool((room[0] == 7).all()) and bool((room[v + 1] == 7).all())


def test_other_stream_and_repeats():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    t, v, k = 300, 1003, 136
    h, w = torch.randn(t, k, device="cuda").half(), torch.randn(v, k, device="cuda").half() * 0.2
    index = torch.randint(0, v, (t, 9), device="cuda")
    teacher = torch.randn(t, 9, device="cuda")
    g = torch.rand(t, device="cuda")
    first = None
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        stream = s if i % 2 else None
        loss, lse = sbl.head_kd(h, w, index, teacher, 2.0, stream=stream)
        out = (loss, lse) + sbl.head_kd_backward(h, w, index, teacher, 2.0, lse, g, stream=stream)
        torch.cuda.synchronize()
        first = first or [x.clone() for x in out]
        assert all(torch.equal(x, y) for x, y in zip(first, out))


@pytest.mark.parametrize("t", [6, 300])
def test_graph_replays(t):
    """Captured calls with new inputs in place: every replay equals the eager call."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v, k = 700, 128
    h, w = torch.randn(t, k, device="cuda").bfloat16(), (torch.randn(v, k, device="cuda") * 0.2).bfloat16()
    target = torch.randint(0, v, (t,), device="cuda")
    g = torch.rand(t, device="cuda")
    fw, bw = sbl.new_head_workspace(t, v, k), sbl.new_head_workspace(t, v, k, backward=True)
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)

    def step():
        sbl.sbl_head_ce_forward(h, w, target, loss, lse, fw)
        sbl.sbl_head_ce_backward(h, w, target, lse, g, dh, dw, bw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        h.copy_(torch.randn(t, k, device="cuda"))
        target.copy_(torch.randint(0, v, (t,), device="cuda"))
        if i == 2:
            target[::2] = -1
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (loss, lse, dh, dw)]
        el, es = sbl.head_ce(h, w, target)
        eh, ew = sbl.head_ce_backward(h, w, target, es, g)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, (el, es, eh, ew)))


def test_refusals_of_the_binding():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    h, w = torch.randn(4, 64, device="cuda").bfloat16(), torch.randn(10, 64, device="cuda").bfloat16()
    target = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        sbl.head_ce(h.float(), w, target)
    with pytest.raises(TypeError):
        sbl.head_ce(h, w.half(), target)
    with pytest.raises(TypeError):
        sbl.head_ce(h, w, target.int())
    with pytest.raises(ValueError):
        sbl.head_ce(h, w[:, :56].contiguous(), target)
    with pytest.raises(ValueError):
        sbl.head_ce(h, w, target[:3])
    with pytest.raises(ValueError):
        sbl.head_ce(h.t().contiguous().t(), w, target)
    with pytest.raises(ValueError):
        sbl.head_ce(h.cpu(), w, target)
    with pytest.raises(ValueError):
        sbl.head_kd(h, w, target[:, None], torch.zeros(4, 2, device="cuda"), 1.0)
    with pytest.raises(sbl.SblError):
        sbl.head_kd(h, w, target[:, None], torch.zeros(4, 1, device="cuda"), 0.0)
    with pytest.raises(sbl.SblError):                 # a workspace one byte short
        n = sbl.sbl_head_workspace_bytes(4, 10, 64)
        sbl.head_ce(h, w, target, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))


def _grid(rng, shape, step, top):
    """Multiples of `step` up to `top`: exact in 16 bits, and so is a step from them."""
    return np.clip(np.round(rng.standard_normal(shape) / step * 0.5), -top / step, top / step) * step


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t", [7, 40, 150])
@pytest.mark.parametrize("kind,tau", [("ce", 1.0), ("kd", 1.0), ("kd", 2.0)])
def test_gradients_are_the_forwards_differences(kind, tau, t, dtype):
    """dh and dw along a direction against the central difference of the forward's
    own losses, whose inputs (the point and both steps from it) are exact in 16
    bits.  Allowed: the forward's bound twice, the gradients' bounds along the
    direction, and what a central difference leaves out, which is the same
    difference and derivative taken in 64 bits."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"head differences {kind} tau={tau} t={t} {dtype}")
    v, d, top = 300, 64, 6
    rng = np.random.default_rng([72, t, int(2 * tau)])
    step_h, step_w = 2.0 ** -5, 2.0 ** -7
    hv, wv = _grid(rng, (t, d), step_h, 3.0), _grid(rng, (v, d), step_w, 0.75) * 0.5
    gone = rng.random(t) < 0.2
    gone[0] = False
    dloss = (rng.integers(1, 9, t) / 8.0).astype(np.float32)
    if kind == "ce":
        target = np.where(gone, -1, rng.integers(0, v, t))
        want, row = H.wanted_ce(target, v)
        entropy, slack = np.zeros(t), np.zeros(t)
        forward = lambda h, w: sbl.head_ce(h, w, _i64(target))
        backward = lambda h, w, lse: sbl.head_ce_backward(h, w, _i64(target), lse, _f32(dloss))
    else:
        index, teacher = _teacher(rng, t, v, top, gone)
        p, logp = H.teacher_probabilities(index, teacher, tau)
        want, row = H.wanted_kd(index, p, v)
        entropy = H.entropy_of(p, logp)
        slack = 64 * H.U32 * (1 + np.abs(np.where(p > 0, logp, 0.0)).max(axis=1))
        forward = lambda h, w: sbl.head_kd(h, w, _i64(index), _f32(teacher), tau)
        backward = lambda h, w, lse: sbl.head_kd_backward(h, w, _i64(index), _f32(teacher), tau, lse, _f32(dloss))
    put = lambda x: _half(x, dtype)[0]
    h, w = put(hv), put(wv)
    assert np.array_equal(_half(hv, dtype)[1], hv) and np.array_equal(_half(wv, dtype)[1], wv)
    lse = forward(h, w)[1]
    dh, dw = (_np(x).astype(np.float64) for x in backward(h, w, lse))
    rh, rw, eh, ew = H.backward(hv, wv, want, row, _np(lse), dloss, tau=tau, dtype=dtype)
    rounded = (tau * np.abs(dloss) * row * slack)[:, None] * want
    eh = eh + 2 * rounded @ np.abs(wv)
    ew = ew + 2 * rounded.T @ np.where(row[:, None], np.abs(hv), 0.0)

    def total(hx, wx):
        loss64, _, bound = H.forward(hx, wx, want, row, entropy, tau)
        loss = _np(forward(put(hx), put(wx))[0]).astype(np.float64)
        return (dloss * loss).sum(), (dloss * loss64 * row).sum(), (dloss * row * (tau * tau) * (bound + slack)).sum()

    for grad, exact, err, step, at in ((dh, rh, eh, step_h, "h"), (dw, rw, ew, step_w / 2, "w")):
        e = np.sign(exact) * step                    # the steepest direction: every difference has one sign
        up = total(hv + e, wv) if at == "h" else total(hv, wv + e)
        down = total(hv - e, wv) if at == "h" else total(hv, wv - e)
        left_out = abs((up[1] - down[1]) / 2 - (exact * e).sum())
        allowed = left_out + (up[2] + down[2]) / 2 + (err * np.abs(e)).sum()
        got, slope = (up[0] - down[0]) / 2, (grad * e).sum()
        assert abs(got - slope) <= allowed, (at, got, slope, allowed)
        assert allowed < 0.1 * abs(slope), (at, slope, allowed)        # the comparison says something


@pytest.mark.parametrize("t,v,d", [(20, 700, 64), (64, 33000, 128), (300, 9000, 64), (520, 33000, 72)])
def test_many_listed_ids_in_one_tile(t, v, d):
    """Every token lists 40 ids of the same 128: more than a tile keeps apart."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"head_kd crowded t={t} v={v} d={d}")
    top, tau, dtype = 40, 2.0, "bfloat16"
    rng, h, hv, w, wv, gone = _inputs(t, v, d, dtype, [73, t])
    index = np.stack([512 + rng.permutation(128)[:top] for _ in range(t)])
    teacher = rng.standard_normal((t, top)).astype(np.float32)
    index[gone] = -1
    p, logp = H.teacher_probabilities(index, teacher, tau)
    want, row = H.wanted_kd(index, p, v)
    loss, lse = sbl.head_kd(h, w, _i64(index), _f32(teacher), tau)
    rl, rs, bound = H.forward(hv, wv, want, row, H.entropy_of(p, logp), tau)
    spread = np.abs(np.where(p > 0, logp, 0.0)).max(axis=1)
    _near(_np(loss), rl, tau * tau * (bound + 64 * H.U32 * (1 + spread)) * row, "loss")
    dloss = (rng.random(t) + 0.5) / t
    dh, dw = sbl.head_kd_backward(h, w, _i64(index), _f32(teacher), tau, lse, _f32(dloss))
    rh, rw, eh, ew = H.backward(hv, wv, want, row, _np(lse), dloss.astype(np.float32), tau=tau, dtype=dtype)
    s = (tau * np.abs(dloss) * row * 64 * H.U32 * (1 + spread))[:, None] * want
    _near(_np(dh), rh, eh + 2 * s @ np.abs(wv), "dh")
    _near(_np(dw), rw, ew + 2 * s.T @ np.where(row[:, None], np.abs(hv), 0.0), "dw")


@pytest.mark.parametrize("t", [1, 20, 40, 70, 300])
def test_an_id_of_no_probability(t):
    """A weight of -infinity on a feature that is positive in every token: its id
    has probability 0, and its row of dw is exactly zero, at every token count."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v, d = 300, 64
    g = torch.Generator(device="cuda").manual_seed(11)
    h, w = torch.randn(t, d, generator=g, device="cuda"), torch.randn(v, d, generator=g, device="cuda") * 0.2
    h[:, 5] = h[:, 5].abs() + 0.5
    w[17, 5] = -float("inf")
    h, w = h.bfloat16(), w.bfloat16()
    target = torch.full((t,), 20, device="cuda")
    loss, lse = sbl.head_ce(h, w, target)
    z = h.double() @ w.double().t()
    assert float((lse.double() - torch.logsumexp(z, 1)).abs().max()) < 1e-4
    assert float((loss.double() - (torch.logsumexp(z, 1) - z[:, 20])).abs().max()) < 1e-4
    dw = torch.empty_like(w)
    sbl.sbl_head_ce_backward(h, w, target, lse, torch.ones(t, device="cuda"), None, dw,
                             _dirty(sbl.sbl_head_workspace_bytes(t, v, d, backward=True)))
    assert dw.isfinite().all() and not dw[17].any()


@pytest.mark.parametrize("t,v,d,kept", [(100, 70001, 256, 0.5), (200, 33001, 520, 0.1), (777, 20011, 392, 0.25),
                                        (777, 20011, 392, 1.0), (130, 70001, 72, 0.01), (100, 140001, 8192, 0.3)])
def test_dh_where_many_rows_are_taken_out(t, v, d, kept):
    """dh is shared over the vocabulary by how many rows take part: few of many,
    all, one; and (the last) in two ranges of the vocabulary."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"head_ce kept={kept} t={t} v={v} d={d}")
    g = torch.Generator(device="cuda").manual_seed(12)
    h = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    w = (torch.randn(v, d, generator=g, device="cuda") * (2.0 / d ** 0.5)).bfloat16()
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    gone = torch.rand(t, generator=g, device="cuda") >= kept
    gone[t // 2] = False
    target[gone] = -1
    h[gone] = float("nan")
    lse = sbl.head_ce(h, w, target)[1]
    dloss = torch.rand(t, generator=g, device="cuda") + 0.5
    dh, dw = torch.full_like(h, 7.0), torch.empty_like(w)
    sbl.sbl_head_ce_backward(h, w, target, lse, dloss, dh, dw,
                             _dirty(sbl.sbl_head_workspace_bytes(t, v, d, backward=True)))
    torch.cuda.synchronize()
    keep = ~gone
    n, hk = int(keep.sum()), h[keep].double()
    rh = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    for i in range(0, v, 16384):
        wi = w[i:i + 16384].double()
        dz = dloss[keep].double()[:, None] * torch.exp(hk @ wi.t() - lse[keep].double()[:, None])
        here = (target[keep] >= i) & (target[keep] < i + len(wi))
        rows = torch.nonzero(here)[:, 0]
        dz[rows, target[keep][rows] - i] -= dloss[keep].double()[rows]
        rh += dz @ wi
        # one rounding of dz and one of the result, each 2^-8 relative at most and never all at once
        assert _rel(dw[i:i + 16384], dz.t() @ hk) < 2.0 ** -8
    assert _rel(dh[keep], rh) < 2.0 ** -8
    assert not dh[gone].any()


@pytest.mark.parametrize("t,top", [(7, 4), (60, 20), (300, 4), (300, 40), (1500, 12)])
def test_absent_entries_hold_any_id(t, top):
    """A teacher logit of -infinity makes its entry absent whatever its id, past the
    vocabulary too (lists padded with the vocabulary's size, say), in both directions."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v, d = 300, 64
    g = torch.Generator(device="cuda").manual_seed(13)
    h = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    w = (torch.randn(v, d, generator=g, device="cuda") * 0.2).bfloat16()
    index = torch.randint(0, v, (t, top), generator=g, device="cuda")
    teacher = torch.randn(t, top, generator=g, device="cuda")
    absent = torch.rand(t, top, generator=g, device="cuda") < 0.4
    absent[:, 0] = False
    absent[t // 2] = True                            # nothing left of this row
    dloss = torch.rand(t, generator=g, device="cuda") + 0.5
    results = []
    for far in (-1, v, 2 ** 40):
        i = torch.where(absent, torch.full_like(index, far), index)
        x = torch.where(absent, torch.full_like(teacher, -float("inf")), teacher)
        loss, lse = sbl.head_kd(h, w, i, x, 2.0)
        results.append((loss, lse, *sbl.head_kd_backward(h, w, i, x, 2.0, lse, dloss)))
    torch.cuda.synchronize()
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))
    assert bool(results[0][2].any(dim=1).sum() == t - 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", ["inf", "-inf", "nan"])
@pytest.mark.parametrize("t,top", [(7, 4), (300, 4), (1500, 12)])
def test_a_gradient_that_is_not_finite_stays_in_its_row(t, top, bad, dtype):
    """dloss or dlse of one row infinite or NaN (an overflow under loss scaling): every
    other row of dh is what it is with an ordinary value there."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v, d, row = 300, 64, t // 2
    g = torch.Generator(device="cuda").manual_seed(14)
    h = torch.randn(t, d, generator=g, device="cuda").to(getattr(torch, dtype))
    w = (torch.randn(v, d, generator=g, device="cuda") * 0.2).to(getattr(torch, dtype))
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    index = torch.randint(0, v, (t, top), generator=g, device="cuda")
    teacher = torch.randn(t, top, generator=g, device="cuda")
    dloss = torch.rand(t, generator=g, device="cuda") + 0.5
    dlse = torch.randn(t, generator=g, device="cuda").clamp(-1, 1) * 0.25
    dloss[0] = 2.0                                   # the largest coefficient is another row's
    spoilt = dloss.clone()
    spoilt[row] = float(bad)
    spoilt_lse = dlse.clone()
    spoilt_lse[row] = float(bad)
    others = torch.arange(t, device="cuda") != row
    lse = sbl.head_ce(h, w, target)[1]
    want = sbl.head_ce_backward(h, w, target, lse, dloss, dlse=dlse)[0]
    for a, b in ((spoilt, dlse), (dloss, spoilt_lse)):
        dh = sbl.head_ce_backward(h, w, target, lse, a, dlse=b)[0]
        assert torch.equal(dh[others], want[others]) and not dh[row].isfinite().any()
    lse = sbl.head_kd(h, w, index, teacher, 2.0)[1]
    want = sbl.head_kd_backward(h, w, index, teacher, 2.0, lse, dloss)[0]
    dh = sbl.head_kd_backward(h, w, index, teacher, 2.0, lse, spoilt)[0]
    assert torch.equal(dh[others], want[others]) and not dh[row].isfinite().any()


def test_refusals_of_the_bindings_lists():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    h, w = torch.randn(4, 64, device="cuda").bfloat16(), torch.randn(10, 64, device="cuda").bfloat16()
    index, teacher = torch.zeros((4, 2), dtype=torch.int64, device="cuda"), torch.zeros((4, 2), device="cuda")
    f = torch.zeros(4, device="cuda")
    for i, x, error in [(None, teacher, TypeError), (index, None, TypeError), (index, [[0.0] * 2] * 4, TypeError),
                        (index[:, 0].contiguous(), teacher, ValueError), (index[:3], teacher[:3], ValueError),
                        (index.int(), teacher, TypeError), (index, teacher.double(), TypeError),
                        (index.t().contiguous().t(), teacher, ValueError)]:
        with pytest.raises(error):
            sbl.head_kd(h, w, i, x, 1.0)
        with pytest.raises(error):
            sbl.head_kd_backward(h, w, i, x, 1.0, f, f)
