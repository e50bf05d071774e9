"""Plain oracle of what a training step needs around the layer and the head
(NumPy only; shares no code with the HIP path): the norm with the activation
quantizer's input, the embedding, and the AdamW update, with their gradients.

Where the result is a sequence of roundings (the norm's forward, AdamW) the
oracle takes the same fp32 steps and results must be equal bit for bit; sums
are compared within bounds that count their roundings."""

from __future__ import annotations

import numpy as np

F32 = np.float32
U32 = 2.0 ** -24                       # unit roundoff of fp32
# of the outputs' types: half a step relative to the value, and half a step of the subnormal range
HALF = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11, "float32": U32}
TINY = {"bfloat16": 2.0 ** -134, "float16": 2.0 ** -25, "float32": 2.0 ** -150}


# ---------------------------------------------------------------- norm

def norm_stats(x, eps, center=True):
    """mean, rstd in float64 of the rows of x."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1) if center else np.zeros(x.shape[0])
    var = ((x - mean[:, None]) ** 2).mean(axis=1)
    return mean, 1.0 / np.sqrt(var + eps)


def norm_forward(x, weight, bias, eps, center=True):
    """(y, mean, rstd) in fp32: statistics rounded once, then one rounding per step."""
    mean, rstd = norm_stats(x, eps, center)
    mean32, rstd32 = mean.astype(F32), rstd.astype(F32)
    return norm_apply(x, mean, rstd32, weight, bias), mean32, rstd32


def norm_apply(x, mean, rstd32, weight, bias):
    """y in fp32 from a mean in float64 and an fp32 rstd."""
    y = (np.asarray(x, dtype=np.float64) - mean[:, None]).astype(F32) * rstd32[:, None]
    if weight is not None:
        y = y * np.asarray(weight, F32)
    if bias is not None:
        y = y + np.asarray(bias, F32)
    return y


def norm_slack(x, eps, center=True):
    """How far two fp64 evaluations of the statistics may be apart: (mean, absolute; rstd, relative), per row.

    Sums of differences to the row's first value pass a term through at most 128 + 6 + 15 additions (a thread of
    a row of 131072 values, its wave, the waves), NumPy's pairwise sum through fewer than 40; with the
    division and the shift 200 roundings of 2^-53 of the sum of sizes cover both.  The variance is s2 / k - e^2,
    off by as much of the mean square of the differences; rstd by half its relative error, and 2^-50."""
    x = np.asarray(x, np.float64)
    mean, rstd = norm_stats(x, eps, center)
    shift = np.abs(x[:, 0]) if center else np.zeros(x.shape[0])
    u = 200 * 2.0 ** -53
    square = ((x - (x[:, :1] if center else 0.0)) ** 2).mean(axis=1)
    return u * (np.abs(x).mean(axis=1) + shift) * bool(center), u * 2 * square * rstd ** 2 + 2.0 ** -50


def norm_backward(dy, x, mean, rstd, weight, center=True):
    """(dx, dweight, dbias) in float64 and (bounds of an fp32 evaluation without its output's rounding).

    A sum of n terms through a tree passes each term through at most `depth` additions.  xh carries 2
    roundings, g one; a row's sums go through at most 16 additions in a thread (k / 1024 in rows of more
    than 16384 values), 6 in a wave and 15 between waves; a column's through the rows of one workgroup and
    then the workgroups.  The products of a sum are rounded or fused, one rounding at most."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    w = np.ones(x.shape[1]) if weight is None else np.asarray(weight, np.float64)
    rows, k = x.shape
    m = np.asarray(mean, np.float64)[:, None] if center else np.zeros((rows, 1))
    r = np.asarray(rstd, np.float64)[:, None]
    xh, g = (x - m) * r, dy * w
    c1 = g.mean(axis=1, keepdims=True) if center else np.zeros((rows, 1))
    c2 = (g * xh).mean(axis=1, keepdims=True)
    dx = r * (g - c1 - xh * c2)
    # depth + the terms' own roundings (g 1, g xh 4) + the division and its factor
    deep = 40 + k / 1024
    e1 = (deep + 4) * U32 * np.abs(g).mean(axis=1, keepdims=True) if center else np.zeros((rows, 1))
    e2 = (deep + 7) * U32 * np.abs(g * xh).mean(axis=1, keepdims=True)
    # g 1, xh c2 3 more roundings, two subtractions, the product with rstd
    ex = np.abs(r) * (e1 + np.abs(xh) * e2 + 8 * U32 * (np.abs(g) + np.abs(c1) + np.abs(xh * c2)))
    ew = (rows + 40) * U32 * np.abs(dy * xh).sum(axis=0)
    eb = (rows + 40) * U32 * np.abs(dy).sum(axis=0)
    return (dx, (dy * xh).sum(axis=0), dy.sum(axis=0)), (ex, ew, eb)


# ---------------------------------------------------------------- embedding

def embed(ids, table, scale):
    """fp32 rows scale * table[id]: zeros for a negative id, NaNs past the table."""
    ids, table = np.asarray(ids), np.asarray(table, F32)
    out = table[np.clip(ids, 0, table.shape[0] - 1)] * F32(scale)
    out[ids < 0] = 0.0
    out[ids >= table.shape[0]] = np.nan
    return out


def embed_backward(ids, dout, n_vocab, scale, old=None):
    """The table's gradient in float64, and the bound of an fp32 sum (without the output's rounding)."""
    ids, dout = np.asarray(ids), np.asarray(dout, np.float64)
    total = np.zeros((n_vocab, dout.shape[1]))
    size = np.zeros_like(total)
    many = np.zeros(n_vocab)
    for t, v in enumerate(ids):
        if 0 <= v < n_vocab:
            total[v] += dout[t]
            size[v] += np.abs(dout[t])
            many[v] += 1
    # at most as many additions as tokens, and the product with the scale
    bound = (many[:, None] + 1) * U32 * size * abs(scale)
    total = total * float(F32(scale))
    if old is not None:
        total = total + np.asarray(old, np.float64)
        bound = bound + U32 * (np.abs(total) + bound)
    return total, bound


# ---------------------------------------------------------------- e4m3

def e4m3_values():
    """The 128 non-negative codes' values (the last is NaN)."""
    c = np.arange(128)
    e, m = c >> 3, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (np.maximum(e, 1) - 10.0))
    v[127] = np.nan
    return v


def e4m3_decode(codes):
    codes = np.asarray(codes, np.uint8)
    return (e4m3_values()[codes & 127] * np.where(codes & 128, -1.0, 1.0)).astype(F32)


def e4m3_nearest(x):
    """Codes nearest to fp32 x (ties to an even code), |x| at most 448."""
    x = np.asarray(x, F32)
    mag = np.minimum(np.abs(x).astype(np.float64), 448.0)
    v = e4m3_values()[:127]
    hi = np.clip(np.searchsorted(v, mag, side="left"), 1, 126)
    lo = hi - 1
    below, above = mag - v[lo], v[hi] - mag
    pick = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def e4m3_cut(t, random, positive):
    """Codes of fp32 t >= 0: down to a code, or up where the 16 random bits reach; where `positive`, not zero.
    The steps of the rounding are those of include/sbl.h: below 2^-6 the value is first brought to
    [2^-6, 2^-5) by an fp32 addition."""
    t = np.asarray(t, F32)
    least = np.where(t < F32(2.0 ** -6), F32(2.0 ** -6), F32(0.0))
    at = (t + least).astype(F32)
    exponent = np.floor(np.log2(at.astype(np.float64)))
    step = 2.0 ** (exponent - 3)
    up = np.asarray(random, np.float64) * step / 65536.0
    cut = np.floor((at.astype(np.float64) + up) / step) * step - least
    cut = np.where(positive, np.clip(cut, 2.0 ** -9, 448.0), 0.0)
    return np.searchsorted(e4m3_values()[:127], cut).astype(np.uint8)


def dither(n, seed):
    """16 bits for each of n values: the halves of a 32-bit hash of the pair's number (the mixer of C. Wellons,
    "Prospecting for Hash Functions", 2018)."""
    h = np.arange((n + 1) // 2, dtype=np.uint64) * np.uint64(0x9E3779B9) + np.uint64(seed)
    mask = np.uint64(0xFFFFFFFF)
    h &= mask
    h ^= h >> np.uint64(16)
    h = (h * np.uint64(0x7FEB352D)) & mask
    h ^= h >> np.uint64(15)
    h = (h * np.uint64(0x846CA68B)) & mask
    h ^= h >> np.uint64(16)
    return np.stack((h & np.uint64(0xFFFF), h >> np.uint64(16)), axis=1).reshape(-1)[:n]


# ---------------------------------------------------------------- AdamW

def split_master(w):
    """(BF16 bits, low bits): nearest BF16, ties away from zero; one NaN for all."""
    w = np.asarray(w, F32)
    bits = np.where(np.isnan(w), np.int64(0x7FC00000), w.view(np.uint32).astype(np.int64))
    high = (bits + 0x8000) >> 16
    return high.astype(np.uint16), (bits - (high << 16)).astype(np.int16)


def join_master(high, low):
    bits = (np.asarray(high, np.uint16).astype(np.int64) << 16) + np.asarray(low, np.int16).astype(np.int64)
    return (bits & 0xFFFFFFFF).astype(np.uint32).view(F32)


def schedule(lr, beta1, beta2, step, factor=1.0):
    return dict(lr=F32(lr), bias1=F32(1.0 / (1.0 - beta1 ** step)), bias2=F32(1.0 / np.sqrt(1.0 - beta2 ** step)),
                factor=F32(factor), seed=step % (1 << 24))


def _scales(x):
    """fp32 scale of each 256 values, and the values over it."""
    n = x.size
    padded = np.zeros(-(-n // 256) * 256, F32)
    padded[:n] = np.abs(x)
    scale = np.maximum(padded.reshape(-1, 256).max(axis=1) * F32(1.0 / 448.0), F32(2.0 ** -126))
    inverse = F32(1.0) / scale
    return scale, x * np.repeat(inverse, 256)[:n]


def adamw(w, g, m, v, s, beta1, beta2, eps, lr_scale=1.0, weight_decay=0.0, m_scale=None, v_scale=None):
    """One step in fp32.  w, g fp32 values; m, v fp32, or uint8 codes with scales.  Returns (w, m, v) or
    (w, m, v, m_scale, v_scale), states in the form that they came in."""
    b1, a1, b2, a2 = F32(beta1), F32(1.0 - beta1), F32(beta2), F32(1.0 - beta2)
    small = m_scale is not None
    w, g = np.asarray(w, F32), np.asarray(g, F32)
    n = w.size
    if small:
        m = e4m3_decode(m) * np.repeat(m_scale, 256)[:n]
        v = e4m3_decode(v) * np.repeat(v_scale, 256)[:n]
        v = v * v
    g = g * s["factor"]
    m = m * b1 + g * a1
    v = v * b2 + (g * g) * a2
    root = np.sqrt(v)
    lr = s["lr"] * F32(lr_scale)
    decay = F32(1.0) - lr * F32(weight_decay)
    w = w * decay - (m / (root * s["bias2"] + F32(eps))) * (lr * s["bias1"])
    assert w.dtype == m.dtype == v.dtype == F32
    if not small:
        return w, m, v
    m_scale, mt = _scales(m)
    v_scale, vt = _scales(root)
    return w, e4m3_nearest(mt), e4m3_cut(vt, dither(n, s["seed"]), root > 0), m_scale, v_scale
