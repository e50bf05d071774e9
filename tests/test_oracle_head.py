"""The oracle of the output head's losses against independent formulas: the
losses against their definitions written as sums over dictionaries, and the
gradients against central differences of the losses."""

import math

import numpy as np
import pytest

from oracle import head_oracle as H


def _inputs(seed, t=5, v=11, d=7, top=4):
    rng = np.random.default_rng(seed)
    h, w = rng.standard_normal((t, d)), rng.standard_normal((v, d))
    target = rng.integers(0, v, t)
    target[1] = -1
    index = np.stack([rng.permutation(v)[:top] for _ in range(t)])
    index[0, 2] = -1
    index[3, 1] = index[3, 0]                       # listed twice
    index[2] = -7                                   # nothing listed
    teacher = rng.standard_normal((t, top)) * 3
    teacher[4, 0] = -np.inf
    return rng, h, w, target, index, teacher


def _ce(h, w, target):
    row = target >= 0
    want, _ = H.wanted_ce(target, w.shape[0])
    return H.forward(h, w, want, row, np.zeros(len(target)))


def _kd(h, w, index, teacher, tau):
    p, logp = H.teacher_probabilities(index, teacher, tau)
    want, row = H.wanted_kd(index, p, w.shape[0])
    return H.forward(h, w, want, row, H.entropy_of(p, logp), tau)


def test_cross_entropy_is_minus_log_probability():
    _, h, w, target, _, _ = _inputs(1)
    loss, lse, _ = _ce(h, w, target)
    for t in range(h.shape[0]):
        if target[t] < 0:
            assert loss[t] == 0 and lse[t] == 0
            continue
        z = [float(h[t] @ w[v]) for v in range(w.shape[0])]
        s = math.fsum(math.exp(x) for x in z)
        assert loss[t] == pytest.approx(-math.log(math.exp(z[target[t]]) / s), rel=1e-12)
        assert lse[t] == pytest.approx(math.log(s), rel=1e-12)


@pytest.mark.parametrize("tau", [1.0, 2.0, 0.7])
def test_distillation_is_the_divergence_on_the_listed_ids(tau):
    _, h, w, _, index, teacher = _inputs(2)
    loss, _, _ = _kd(h, w, index, teacher, tau)
    for t in range(h.shape[0]):
        has = [k for k in range(index.shape[1]) if index[t, k] >= 0 and teacher[t, k] != -np.inf]
        if not has:
            assert loss[t] == 0
            continue
        e = [math.exp(teacher[t, k] / tau) for k in has]
        p = [x / math.fsum(e) for x in e]
        z = [math.exp(float(h[t] @ w[v]) / tau) for v in range(w.shape[0])]
        s = math.fsum(z)
        want = tau ** 2 * math.fsum(p[i] * math.log(p[i] / (z[index[t, k]] / s)) for i, k in enumerate(has))
        assert loss[t] == pytest.approx(want, rel=1e-10)


@pytest.mark.parametrize("kind,tau", [("ce", 1.0), ("kd", 1.0), ("kd", 2.5)])
def test_gradients_are_the_losses_differences(kind, tau):
    rng, h, w, target, index, teacher = _inputs(3)
    dloss = rng.standard_normal(h.shape[0])
    dlse = rng.standard_normal(h.shape[0]) if kind == "ce" else np.zeros(h.shape[0])

    def total(h, w):
        loss, lse, _ = _ce(h, w, target) if kind == "ce" else _kd(h, w, index, teacher, tau)
        return float((dloss * loss + dlse * lse).sum())

    if kind == "ce":
        row, (want, _) = target >= 0, H.wanted_ce(target, w.shape[0])
        _, lse, _ = _ce(h, w, target)
    else:
        want, row = H.wanted_kd(index, H.teacher_probabilities(index, teacher, tau)[0], w.shape[0])
        _, lse, _ = _kd(h, w, index, teacher, tau)
    dh, dw, _, _ = H.backward(h, w, want, row, lse, dloss, dlse, tau)
    step = 1e-5                                     # differences are off by step^2 of third derivatives
    for x, g in ((h, dh), (w, dw)):
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + step
            up = total(h, w)
            x[i] = keep - step
            down = total(h, w)
            x[i] = keep
            assert g[i] == pytest.approx((up - down) / (2 * step), rel=1e-6, abs=1e-7)
