"""A token with a NaN or an infinity shows it in its gamma, by every quantizer, and in no other token's values."""

import numpy as np
import pytest

import synth
from gpu_util import FMT_DENSE2, say, to_dev

pytestmark = pytest.mark.gpu

# NaNs of either sign, infinities
BAD = [0x7FC00000, 0xFFC00000, 0x7F800001, 0x7F800000, 0xFF800000]


def _inputs(t, k, seed):
    import torch
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal((t, k)).astype(np.float32)).cuda()


def _spoil(x, row, col, bits):
    import torch
    x.view(torch.int32)[row, col] = bits - (1 << 32) if bits >> 31 else bits


def _shows(gamma, bits):
    import torch
    return torch.isinf(gamma).all() if bits & 0x7FFFFFFF == 0x7F800000 else torch.isnan(gamma).all()


# one wave's row to the longest, few tokens and many: each variant of the quantizer
@pytest.mark.parametrize("t,k", [(1, 64), (3, 640), (2, 8192), (2, 16384), (1, 32768), (2, 40000), (200, 320), (130, 8192),
                                 (128, 13824), (129, 28672)])
def test_gamma_of_a_token_that_is_not_finite(t, k):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"quant_acts not finite t={t} k={k}")
    x = _inputs(t, k, [101, t, k])
    q, g = sbl.quant_acts(x)
    keep = torch.arange(t, device="cuda") != t // 2
    for bits in BAD:
        for col in (0, k // 3, k - 1):
            y = x.clone()
            _spoil(y, t // 2, col, bits)
            q2, g2 = sbl.quant_acts(y)
            assert _shows(g2[t // 2], bits) and torch.equal(g2[keep], g[keep]) and torch.equal(q2[keep], q[keep])


def test_gamma_of_a_group_that_is_not_finite():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    t, k, kg = 3, 1280, 320
    x = _inputs(t, k, 102)
    out = lambda: (torch.empty((t, k), dtype=torch.int8, device="cuda"), torch.empty((t, k // kg), device="cuda"))  # noqa: E731
    (q, g), (q2, g2) = out(), out()
    sbl.sbl_quant_acts_kgrouped(x, kg, q, g)
    for bits in BAD:
        y = x.clone()
        _spoil(y, 1, 2 * kg + 5, bits)
        sbl.sbl_quant_acts_kgrouped(y, kg, q2, g2)
        keep = torch.ones((t, k // kg), dtype=torch.bool, device="cuda")
        keep[1, 2] = False
        assert _shows(g2[1, 2], bits) and torch.equal(g2[keep], g[keep])
        wide = keep.repeat_interleave(kg, 1)
        assert torch.equal(q2[wide], q[wide])


@pytest.mark.parametrize("t,k", [(1, 1024), (4, 640), (16, 1024)])
def test_products_that_quantize_within(t, k):
    """The product's own quantizer (up to 16 tokens): gamma and y of the token, the other tokens' as they were."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"linear_acts not finite t={t} k={k}")
    n_out = 320
    w = sbl.quant_weights(to_dev(synth.gaussian_masters(np.random.default_rng(103), n_out, k)), 6, 8, FMT_DENSE2)
    x = _inputs(t, k, [104, t, k])

    def run(x):
        xq, gamma = torch.empty((t, k), dtype=torch.int8, device="cuda"), torch.empty(t, device="cuda")
        y = torch.empty((t, n_out), device="cuda")
        sbl.sbl_linear_acts_batch(x, xq, gamma, [dict(packed=w["packed"], meta=w["meta"], beta=w["beta"], n_out=n_out, y=y)],
                                  FMT_DENSE2, 6, 8)
        return xq, gamma, y

    want = run(x)
    keep = torch.arange(t, device="cuda") != t // 2
    for bits in BAD:
        y = x.clone()
        _spoil(y, t // 2, 7, bits)
        got = run(y)
        assert _shows(got[1][t // 2], bits) and not torch.isfinite(got[2][t // 2]).any()
        for a, b in zip(got, want):
            assert torch.equal(a[keep], b[keep])
