"""Plain 64-bit oracle of the output head's losses (NumPy only; shares no code
with the HIP path): cross entropy over a vocabulary and distillation from a
teacher's listed logits, with their gradients and elementwise bounds of what
a 16-bit gradient of the logits and 32-bit sums may be off by.

  z = h w^T;  cross entropy: loss = lse(z) - z[target];
  distillation: p = softmax over the listed teacher / tau,
                loss = tau^2 sum_k p_k (log p_k - z[index_k] / tau + lse(z / tau)).
"""

from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24                       # unit roundoff of fp32
U16 = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}   # of the 16-bit types: 8 and 11 significant bits
TINY16 = {"bfloat16": 0.0, "float16": 2.0 ** -25}      # half a step below their normal range


def _lse(x):
    top = x.max(axis=1, keepdims=True)
    return (top + np.log(np.exp(x - top).sum(axis=1, keepdims=True)))[:, 0]


def teacher_probabilities(index, teacher, tau):
    """(p, log p) [rows][top]; 0 where an entry is absent; rows without entries are all 0."""
    p = np.zeros(teacher.shape)
    logp = np.zeros(teacher.shape)
    for t in range(index.shape[0]):
        has = [k for k in range(index.shape[1]) if index[t, k] >= 0 and teacher[t, k] != -np.inf]
        if not has:
            continue
        x = teacher[t, has].astype(np.float64) / tau
        x = x - x.max()
        logp[t, has] = x - np.log(np.exp(x).sum())
        p[t, has] = np.exp(logp[t, has])
    return p, logp


def wanted_ce(target, n_vocab):
    """Dense wanted distribution [rows][n_vocab] and which rows take part."""
    want = np.zeros((len(target), n_vocab))
    for t, y in enumerate(target):
        if 0 <= y < n_vocab:
            want[t, y] = 1.0
    return want, np.asarray(target) >= 0


def wanted_kd(index, p, n_vocab):
    want = np.zeros((index.shape[0], n_vocab))
    for t in range(index.shape[0]):
        for k in range(index.shape[1]):
            if p[t, k] > 0 and index[t, k] < n_vocab:
                want[t, index[t, k]] += p[t, k]
    return want, p.sum(axis=1) > 0


def forward(h, w, want, row, entropy, tau=1.0):
    """(loss, lse, bound): bound of a 32-bit evaluation's error in both.
    A logit is a sum of k exact products in fp32: (k + 1) U32 sum|h w|, in any
    order.  Scaling, exponential, logarithm and the sums over the vocabulary
    add a few U32 of the largest term each, and less than 64 U32 in all of
    (1 + |lse| + largest |z|)."""
    h = np.where(row[:, None], h, 0.0).astype(np.float64)
    w = w.astype(np.float64)
    z = h @ w.T / tau
    lse = _lse(z)
    loss = tau * tau * (entropy - (want * z).sum(axis=1) + want.sum(axis=1) * lse)
    ez = ((h.shape[1] + 1) * U32 * (np.abs(h) @ np.abs(w).T) / tau).max(axis=1)
    bound = 2 * ez + 64 * U32 * (1.0 + np.abs(lse) + np.abs(z).max(axis=1))
    return np.where(row, loss, 0.0), np.where(row, lse, 0.0), bound


def entropy_of(p, logp):
    return (p * logp).sum(axis=1)


def backward(h, w, want, row, lse, dloss, dlse=None, tau=1.0, dtype="bfloat16"):
    """(dh, dw, dh_bound, dw_bound).  `lse` is taken as given.  The bounds:
    each logit gradient is rounded once to 16 bits (U16 of itself) after an
    evaluation in 32 bits whose error is that of the logit in the exponent
    (as in forward) and 64 U32 of its two parts; the products' sums are fp32 in
    any order; the output is rounded once more."""
    h = np.where(row[:, None], h, 0.0).astype(np.float64)
    w = w.astype(np.float64)
    n = row.astype(np.float64)
    dloss = np.where(row, dloss, 0.0).astype(np.float64)
    dlse = np.zeros_like(dloss) if dlse is None else np.where(row, dlse, 0.0).astype(np.float64)
    z = h @ w.T / tau
    lse = np.where(row, lse, 0.0).astype(np.float64)
    q = np.exp(np.where(row[:, None], z - lse[:, None], -np.inf))
    first = (tau * (dloss + dlse))[:, None] * q
    second = (tau * dloss)[:, None] * want * n[:, None]
    dz = first - second
    u, tiny = U16[dtype], TINY16[dtype]
    ez = (h.shape[1] + 1) * U32 * (np.abs(h) @ np.abs(w).T) / tau
    parts = np.abs(first) + np.abs(second)
    e = u * np.abs(dz) + np.abs(first) * (2 * ez + 64 * U32 * (1 + np.abs(lse)[:, None] + np.abs(z))) + 64 * U32 * parts
    scale = np.abs(tau * dloss).max(initial=0.0) + np.abs(tau * (dloss + dlse)).max(initial=0.0)
    e = e + 2.0 ** -38 * scale                      # below the scaled 16-bit type's normal range
    e = e * (1 + 2 * u)

    def product(a, ea, b):
        out = a @ b
        err = ea @ np.abs(b)
        err = err + (a.shape[1] + 8) * U32 * ((np.abs(a) + ea) @ np.abs(b))
        return out, (err + u * (np.abs(out) + err)) + tiny

    dh, eh = product(dz, e, w)
    dw, ew = product(dz.T, e.T, h)
    return dh, dw, eh, ew
