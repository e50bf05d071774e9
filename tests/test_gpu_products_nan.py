"""A token whose gamma is NaN (the norm's of a row that is not finite) shows it in every product, and in no other token's."""

import numpy as np
import pytest

import synth
from gpu_util import FMT_DENSE2, FMT_NM, say, to_dev

pytestmark = pytest.mark.gpu

KINDS = [(FMT_DENSE2, 6, 8), (FMT_NM, 6, 8), (FMT_NM, 2, 4), (FMT_NM, 5, 8)]


def _rows(got, want, bad):
    import torch
    keep = torch.ones(got.shape[0], dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[bad]).all() and torch.isfinite(want).all()


@pytest.mark.parametrize("fmt,n,m", KINDS)
@pytest.mark.parametrize("t", [1, 5, 16, 17, 300])
def test_products_of_a_row_that_is_not_finite(t, fmt, n, m):
    """Norm and quantizer, then the product as GEMV, GEMM, sparse GEMM and in the generic kernel, one beta or several."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    n_out, k, rpg = 300, 640, 64
    say(f"products of a NaN row t={t} {n}:{m} fmt={fmt}")
    rng = np.random.default_rng([97, t, fmt, n])
    w = sbl.quant_weights(to_dev(synth.gaussian_masters(rng, n_out, k)), n, m, fmt)
    x = torch.from_numpy(rng.standard_normal((t, k)).astype(np.float32)).cuda()
    xq, gamma = sbl.norm_quant(x, center=False, want_y=False)[:2]
    want = sbl.linear(w["packed"], w["meta"], fmt, n, m, w["beta"], xq, gamma, n_out)[0]
    x[t // 2, 7] = float("nan")
    xq2, gamma2 = sbl.norm_quant(x, center=False, want_y=False)[:2]
    _rows(sbl.linear(w["packed"], w["meta"], fmt, n, m, w["beta"], xq2, gamma2, n_out)[0], want, t // 2)
    beta = w["beta"].repeat(-(-n_out // rpg)).contiguous()
    groups = [torch.empty((t, n_out), device="cuda") for _ in range(2)]
    for y, q, g in zip(groups, (xq2, xq), (gamma2, gamma)):
        sbl.sbl_linear_grouped(w["packed"], w["meta"], fmt, n, m, beta, rpg, q, g, n_out, y)
    _rows(groups[0], groups[1], t // 2)


def test_products_with_activation_groups():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    t, n_out, k, kg = 5, 100, 640, 320
    rng = np.random.default_rng(98)
    w = sbl.quant_weights(to_dev(synth.gaussian_masters(rng, n_out, k)), 6, 8, FMT_NM)
    x = torch.from_numpy(rng.standard_normal((t, k)).astype(np.float32)).cuda()
    xq, gamma = torch.empty((t, k), dtype=torch.int8, device="cuda"), torch.empty((t, k // kg), device="cuda")
    sbl.sbl_quant_acts_kgrouped(x, kg, xq, gamma)
    y = [torch.empty((t, n_out), device="cuda") for _ in range(2)]
    for out in y:
        sbl.sbl_linear_kgrouped(w["packed"], w["meta"], FMT_NM, 6, 8, w["beta"], n_out, xq, gamma, kg, n_out, out)
        gamma[3, 1] = float("nan")
    _rows(y[1], y[0], 3)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("t", [1, 40, 300])
def test_weight_gradient_of_a_row_that_is_not_finite(t, workspace):
    """Every weight's gradient sums over the tokens: all are NaN."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    n_out, k = 200, 320
    say(f"dw of a NaN row t={t} workspace={workspace}")
    rng = np.random.default_rng([99, t])
    w = sbl.quant_weights(to_dev(synth.gaussian_masters(rng, n_out, k)), 6, 8, FMT_DENSE2)
    x = torch.from_numpy(rng.standard_normal((t, k)).astype(np.float32)).cuda()
    dy = torch.from_numpy(rng.standard_normal((t, n_out)).astype(np.float32)).cuda().bfloat16()
    ws = sbl.new_backward_workspace(t, n_out, k) if workspace else None
    for bad in (False, True):
        if bad:
            x[t // 2, 0] = float("nan")
        xq, gamma, y, _, _ = sbl.norm_quant(x, center=False)
        dw = torch.zeros((n_out, k), device="cuda")
        sbl.sbl_linear_backward(dy, w["packed"], w["meta"], FMT_DENSE2, 6, 8, w["beta"], y, xq, gamma, dw=dw, workspace=ws)
        assert torch.isnan(dw).all() if bad else torch.isfinite(dw).all()
