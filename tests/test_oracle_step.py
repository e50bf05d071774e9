"""The oracle of the norm, the embedding and AdamW against independent
formulas: gradients against central differences, 8-bit codes against torch's
own float8 type, the update against the textbook formula in 64 bits."""

import math

import numpy as np
import pytest
import torch

from oracle import sbl_oracle as O
from oracle import step_oracle as S


@pytest.mark.parametrize("center", [True, False])
def test_norm_backward_is_the_derivative(center):
    rng = np.random.default_rng(1)
    x, w, b = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal(7)
    dy, eps, h = rng.standard_normal((3, 7)), 1e-3, 1e-6

    def loss(x, w, b):
        mean, rstd = S.norm_stats(x, eps, center)
        return (((x - mean[:, None]) * rstd[:, None] * w + b) * dy).sum()

    mean, rstd = S.norm_stats(x, eps, center)
    got, bounds = S.norm_backward(dy, x, mean, rstd, w, center)
    for i, (at, grad) in enumerate(zip((x, w, b), got)):
        for j in np.ndindex(at.shape):
            args = [a.copy() for a in (x, w, b)]
            args[i][j] += h
            up = loss(*args)
            args[i][j] -= 2 * h
            assert abs((up - loss(*args)) / (2 * h) - grad[j]) < 1e-7
    assert all((e >= 0).all() and e.max() < 1e-4 for e in bounds)


@pytest.mark.parametrize("center", [True, False])
def test_norm_forward_is_near_the_formula(center):
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((5, 300)) * 3 + 2).astype(np.float32)
    w, b = rng.standard_normal(300).astype(np.float32), rng.standard_normal(300).astype(np.float32)
    y, mean, rstd = S.norm_forward(x, w, b, 1e-5, center)
    x64 = torch.from_numpy(x).double()
    if center:
        want = torch.nn.functional.layer_norm(x64, (300,), torch.from_numpy(w).double(), torch.from_numpy(b).double(), 1e-5)
    else:
        want = x64 / (x64.square().mean(1, keepdim=True) + 1e-5).sqrt() * torch.from_numpy(w) + torch.from_numpy(b)
        assert not mean.any()
    want = want.numpy()
    # d, rstd and their product, the product with w: 4 roundings of n w, then one of the sum
    assert (np.abs(y - want) <= 5 * S.U32 * (np.abs(want) + 2 * np.abs(b)) + 1e-12).all()
    assert y.dtype == rstd.dtype == np.float32


def test_norm_keeps_a_far_mean():
    """A mean 10^5 times the spread: the differences are exact in 64 bits, rounded once."""
    x = (np.arange(64, dtype=np.float32) / 64 + np.float32(1e5))[None]
    y, _, _ = S.norm_forward(x, None, None, 1e-12)
    d = x.astype(np.float64) - x.astype(np.float64).mean()
    assert np.abs(y - d / np.sqrt((d * d).mean())).max() < 4 * S.U32 * np.abs(y).max()


def test_embedding_and_its_gradient():
    rng = np.random.default_rng(3)
    table = rng.standard_normal((6, 4)).astype(np.float32)
    ids = np.array([2, -1, 5, 2, 6, 0, 2, -100])
    out = S.embed(ids, table, 2.0)
    assert np.array_equal(out[0], 2 * table[2]) and not out[1].any() and np.isnan(out[4]).all() and not out[7].any()
    dout = rng.standard_normal((8, 4))
    got, bound = S.embed_backward(ids, dout, 6, 2.0)
    want = np.zeros((6, 4))
    np.add.at(want, [2, 5, 2, 0, 2], 2.0 * dout[[0, 2, 3, 5, 6]])
    assert np.allclose(got, want, rtol=1e-14, atol=0) and not bound[1].any() and (bound[2] > 0).all()
    more, _ = S.embed_backward(ids, dout, 6, 2.0, old=table)
    assert np.allclose(more, want + table, rtol=1e-14, atol=1e-14)


def test_e4m3_codes_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    codes = codes[(codes & 127) != 127]
    values = S.e4m3_decode(codes)
    assert np.array_equal(values, torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy())
    assert np.array_equal(S.e4m3_nearest(values), codes)
    rng = np.random.default_rng(4)
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 0.01, 2.0 ** rng.uniform(-12, 9, 4000)])
    mids = (S.e4m3_values()[:126] + S.e4m3_values()[1:127]) / 2        # ties
    x = np.clip(np.concatenate([x, mids, -mids]), -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(S.e4m3_nearest(x), want)


def test_e4m3_cut_rounds_in_proportion():
    values = S.e4m3_values()[:127]
    t = np.array([0.0, 1e-6, 2.0 ** -10, 0.003, 0.0149, 0.0157, 0.3, 1.0, 1.06, 5.3, 440.0, 448.0], np.float32)
    for x in t:
        random = np.arange(65536)
        got = values[S.e4m3_cut(np.full(65536, x, np.float32), random, x > 0)]
        lo = values[np.searchsorted(values, x, side="right") - 1]
        hi = values[min(np.searchsorted(values, x, side="right"), 126)]
        assert set(got) <= {lo, hi, 2.0 ** -9 if x > 0 else 0.0}
        if x >= 2.0 ** -9:
            # the share of random bits that go up is the place between the neighbours, to one in 65536 (and below
            # 2^-6 the rounding of one fp32 addition, 2^-30 of 2^-9)
            assert abs(got.mean() - x) <= (hi - lo) / 65536 + 2.0 ** -30
        assert (got > 0).all() or x == 0


def test_dither_is_spread():
    d = S.dither(1 << 16, 7)
    assert d.min() >= 0 and d.max() < 65536 and abs(d.mean() / 65536 - 0.5) < 0.01
    assert np.histogram(d, 16, (0, 65536))[0].std() < 300                  # 64 expected of a Poisson count of 4096
    assert (S.dither(1 << 10, 8) != d[:1 << 10]).mean() > 0.99 and np.array_equal(S.dither(5, 7), d[:5])
    assert abs(np.corrcoef(d[0::2], d[1::2])[0, 1]) < 0.03


def test_split_master_is_the_fp32_weight():
    rng = np.random.default_rng(5)
    bits = rng.integers(0, 1 << 32, 20000, dtype=np.uint32)
    bits = bits[((bits >> 23) & 255) < 254]
    special = np.array([0x3F808000, 0x3F807FFF, 0x3F818000, 0xBF808000, 0, 0x80000000, 0x8000, 0x7FFF], np.uint32)
    w = np.concatenate([bits, special]).view(np.float32)
    high, low = S.split_master(w)
    assert np.array_equal(S.join_master(high, low).view(np.uint32), w.view(np.uint32))
    near = O.bf16_to_f32(high).astype(np.float64)
    step = np.abs(O.bf16_to_f32(high + np.uint16(1)).astype(np.float64) - near)
    assert (np.abs(near - w) <= step / 2 * (1 + 1e-9)).all()


@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_adamw_is_the_textbook_step(decay):
    rng = np.random.default_rng(6)
    n, lr, b1, b2, eps = 1000, 1e-2, 0.9, 0.99, 1e-8
    w, m, v = rng.standard_normal(n), np.zeros(n), np.zeros(n)
    got = (w.astype(np.float32), np.zeros(n, np.float32), np.zeros(n, np.float32))
    p = torch.nn.Parameter(torch.from_numpy(w.copy()))
    optimizer = torch.optim.AdamW([p], lr=lr, betas=(b1, b2), eps=eps, weight_decay=decay)
    for t in range(1, 6):
        g = rng.standard_normal(n).astype(np.float32)
        got = S.adamw(got[0], g, got[1], got[2], S.schedule(lr, b1, b2, t), b1, b2, eps, weight_decay=decay)
        p.grad = torch.from_numpy(g).double()
        optimizer.step()
    # a dozen roundings a step of a weight of order one
    assert np.abs(got[0] - p.detach().numpy()).max() < 5 * 12 * S.U32 * 5
    state = optimizer.state[p]
    assert np.allclose(got[1], state["exp_avg"], rtol=0, atol=1e-6) and np.allclose(got[2], state["exp_avg_sq"], atol=1e-6)


def test_adamw_in_8_bits_follows_the_32_bit_states():
    """v must follow its average although a step moves it far less than half a code.

    How far the held root may be from the true one: a step moves it by d = |g^2 / v - 1| / (2 T) of itself, T the
    steps that v averages over (t at first, 1 / (1 - b2) later), and pulls an error e back by e / T.  Rounding
    at random adds a variance of d times the codes' distance, E|chi^2 - 1| / (2 T) * 0.090 (e4m3's distance over
    the value is 1/8 to 1/16, 0.090 in the mean of its logarithm) = 0.0437 / T.  At rest that is e's
    variance times 2 / T: 0.0218, a deviation of 0.148, and a median of |e| of 0.6745 * 0.148 = 0.0996 in the first
    order of e; the second, -e^2 / 2 in the logarithm, moves it by up to 0.148^2 / 2 = 0.011, and the median of
    2048 values has a deviation of 0.0025 (4 of them: 0.010)."""
    rng = np.random.default_rng(7)
    n, b1, b2 = 2048, 0.9, 0.999
    size = np.exp(rng.standard_normal(n))
    a = (np.zeros(n, np.float32), np.zeros(n, np.float32), np.zeros(n, np.float32))
    blocks = n // 256
    b = (a[0], np.zeros(n, np.uint8), np.zeros(n, np.uint8), np.zeros(blocks, np.float32), np.zeros(blocks, np.float32))
    for t in range(1, 401):
        g = (size * rng.standard_normal(n)).astype(np.float32)
        s = S.schedule(1e-3, b1, b2, t)
        a = S.adamw(a[0], g, a[1], a[2], s, b1, b2, 1e-8)
        b = S.adamw(b[0], g, b[1], b[2], s, b1, b2, 1e-8, m_scale=b[3], v_scale=b[4])
    root = S.e4m3_decode(b[2]) * np.repeat(b[4], 256)
    assert abs(math.log((root.astype(np.float64) ** 2).sum() / a[2].astype(np.float64).sum())) < 0.05
    away = np.abs(np.log(root / np.sqrt(a[2])))
    assert np.median(away) < 0.0996 + 0.011 + 0.010
    assert np.corrcoef(a[0], b[0])[0, 1] > 0.98
