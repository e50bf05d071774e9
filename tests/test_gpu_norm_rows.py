"""The norm with the quantizer in every form that a call can ask for (centered
or not, with weight and bias or without), and rows that are not finite: they
show it in everything that is computed from them, up to the next layer's
products."""

import numpy as np
import pytest

from gpu_util import say, to_np
from oracle import sbl_oracle as O
from test_gpu_step import PAIRS, Guarded, _check_norm, _dev, _f32, _norm_inputs, _same, _type

pytestmark = pytest.mark.gpu

# one token, few and many rows, rows in one to eight vectors a thread, held weights and weights read again, whole
# lines past the caches, the kernel for the longest rows
SIZES = [(1, 64), (1, 3200), (5, 256), (3, 4096), (2, 8192), (2, 28672), (2, 40000), (1, 131072), (1025, 320),
         (1650, 5120), (1100, 8640), (1030, 13824)]
FORMS = [(True, True, True), (False, True, False), (True, False, True), (False, False, False)]


@pytest.mark.parametrize("tx,ty", PAIRS)
@pytest.mark.parametrize("t,k", SIZES)
def test_norm_with_quantizer_in_every_form(t, k, tx, ty):
    """y, mean and rstd against the oracle; gamma and the codes are the quantizer's of the fp32 y, bit for bit."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    rng, x, xv, w, b = _norm_inputs(t, k, tx, [91, t, k])
    for center, weight, bias in FORMS:
        say(f"norm_quant t={t} k={k} {tx}->{ty} center={center} weight={weight} bias={bias}")
        wt, bt = w if weight else None, b if bias else None
        args = (x, _f32(w) if weight else None, _f32(b) if bias else None, 1e-5, center)
        y32, mean32, rstd32 = sbl.norm(*args, dtype=torch.float32)
        _check_norm(xv, wt, bt, center, y32, "float32", mean32, rstd32)
        rq, rg = O.quant_acts(to_np(y32))
        out = Guarded()
        y, xq = out.new((t, k), ty), out.new((t, k), "int8")
        gamma, mean, rstd = (out.new((t,), "float32") for _ in range(3))
        for want_y in (y, None):
            sbl.sbl_norm_forward(*args, y=want_y, xq=xq, gamma=gamma, mean=mean, rstd=rstd)
            torch.cuda.synchronize()
            _same(gamma, torch.from_numpy(rg), "gamma")
            _same(xq, torch.from_numpy(rq), "xq")
            _same(mean, mean32.cpu(), "mean")
            _same(rstd, rstd32.cpu(), "rstd")
            xq.zero_()
            gamma.zero_()
        _same(y, y32.to(_type(ty)).cpu(), "y")
        out.check()


@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("tx,ty", [("bfloat16", "float32"), ("float32", "bfloat16"), ("float16", "float16")])
@pytest.mark.parametrize("t,k", [(5, 64), (3, 4096), (2, 28672), (3, 39936), (1500, 512), (1650, 5120), (1100, 8192),
                                 (1100, 8640), (1030, 13824)])
def test_rows_that_are_not_finite_show_it(t, k, tx, ty, center, bad):
    """y, rstd and gamma of such a row are NaN wherever its value lies; the other rows keep their bits."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"not finite t={t} k={k} {tx}->{ty} center={center} {bad}")
    rng, x, _, w, b = _norm_inputs(t, k, tx, [92, t, k])
    dy = _dev(rng.standard_normal((t, k)), ty)[0]
    args = (_f32(w), _f32(b), 1e-5, center, _type(ty))
    want = sbl.norm_quant(x, *args)
    gx = sbl.norm_backward(dy, x, want[3], want[4], args[0], center=center)[0]
    at = sorted({(0, 0), (1, k // 2 + 1), (t - 1, k - 1)})
    for row, col in at:
        x[row, col] = float(bad)
    rows = torch.tensor(sorted({r for r, _ in at}), device="cuda")
    keep = torch.ones(t, dtype=torch.bool, device="cuda")
    keep[rows] = False
    got = sbl.norm_quant(x, *args)
    for a, r in zip(got, want):
        assert torch.equal(a[keep], r[keep])
    xq, gamma, y, mean, rstd = got
    for a in (gamma, y, rstd):
        assert torch.isnan(a[rows]).all()
    if center:
        assert not torch.isfinite(mean[rows]).any()
    else:
        assert not mean.any()
    none = sbl.norm_quant(x, *args[:4], want_y=False)
    assert none[2] is None and torch.isnan(none[1][rows]).all() and torch.equal(none[1][keep], gamma[keep])
    dx = sbl.norm_backward(dy, x, mean, rstd, args[0], center=center)[0]
    assert torch.equal(dx[keep], gx[keep]) and torch.isnan(dx[rows]).all()


@pytest.mark.parametrize("t,k", [(3, 256), (2, 39936), (1650, 5120)])
def test_weights_that_are_not_finite_show_in_gamma(t, k):
    """A NaN in weight or bias makes its column NaN, and the gamma of every row; a y past fp32's range, an infinite one."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"weights not finite t={t} k={k}")
    _, x, _, w, b = _norm_inputs(t, k, "bfloat16", [93, t, k])
    others = [j for j in range(k) if j != k // 3]
    for center in (True, False):
        want = sbl.norm(x, _f32(w), _f32(b), center=center, dtype=torch.float32)[0]
        for which in range(2):
            p = [w.copy(), b.copy()]
            p[which][k // 3] = np.nan
            _, gamma, y, _, rstd = sbl.norm_quant(x, _f32(p[0]), _f32(p[1]), center=center, dtype=torch.float32)
            assert torch.isnan(gamma).all() and torch.isnan(y[:, k // 3]).all() and torch.isfinite(rstd).all()
            assert torch.equal(y[:, others], want[:, others])
        p = b.copy()
        p[k // 3] = np.inf
        assert torch.isinf(sbl.norm_quant(x, _f32(w), _f32(p), center=center)[1]).all()
