"""The norm, the embedding and AdamW on the GPU against the oracle: the norm's
codes and AdamW bit for bit, the norm's forward too but for fp64 sums next to
the border of a rounding, sums within the oracle's elementwise
bounds; over the variants' edges, every type, odd sizes, empty and single
rows, guard bands, dirty workspaces, streams and graphs."""

import numpy as np
import pytest

from gpu_util import say, to_np
from oracle import sbl_oracle as O
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu

PAIRS = [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float16", "float16"), ("float16", "float32"),
         ("float32", "float32"), ("float32", "bfloat16"), ("float32", "float16")]
GUARD = 0x5A


def _type(name):
    import torch
    return getattr(torch, name)


def _dev(x, dtype):
    """numpy -> GPU tensor of the type, and its values back in float64."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(_type(dtype))
    return t.cuda(), t.double().numpy()


def _f32(x):
    return _dev(x, "float32")[0]


def _i64(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int64)).cuda()


def _rounded(x, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(_type(dtype))


class Guarded:
    """Outputs inside larger buffers whose other bytes must stay as they are."""

    def __init__(self):
        self.all = []

    def new(self, shape, dtype, at=256, fill=None):
        import torch
        dt = _type(dtype) if isinstance(dtype, str) else dtype
        n = int(np.prod(shape, dtype=np.int64)) * torch.empty(0, dtype=dt).element_size()
        raw = torch.full((at + n + 512,), GUARD, dtype=torch.uint8, device="cuda")
        self.all.append((raw, at, n))
        t = raw[at:at + n].view(dt).view(shape)
        if fill is not None:
            t.copy_(fill)
        return t

    def check(self):
        for raw, at, n in self.all:
            r = to_np(raw)
            assert (r[:at] == GUARD).all() and (r[at + n:] == GUARD).all()


def _dirty(nbytes):
    import torch
    return torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")


def _same(got, want, name):
    """Equal bit for bit, a zero's sign aside."""
    import torch
    a, b = got.detach().cpu(), want
    assert a.dtype == b.dtype and a.shape == b.shape, (name, a.dtype, b.dtype, a.shape, b.shape)
    bad = ~((a == b) | (torch.isnan(a) & torch.isnan(b))) if a.is_floating_point() else a != b
    assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:4].tolist(), a[bad][:4].tolist(), b[bad][:4].tolist())


def _near(got, want, bound, dtype, name):
    """Within the bound and one rounding to the output's type."""
    g = to_np(got.double())
    allowed = bound + S.HALF[dtype] * (np.abs(want) + bound) + S.TINY[dtype]
    bad = ~(np.abs(g - want) <= allowed)
    assert not bad.any(), (name, int(bad.sum()), [tuple(int(i) for i in x) for x in np.argwhere(bad)[:4]],
                           g[bad][:4], want[bad][:4])


# ---------------------------------------------------------------- norm

# one slot per thread up to 4096 values, two, four up to 16384, rows in sweeps above; few and many rows
NORM = [(1, 1), (3, 2), (4, 3), (2, 5), (5, 63), (4, 64), (3, 65), (2, 250), (7, 1000), (3, 1541), (1, 3200), (2, 4095), (2, 4096),
        (2, 4097), (3, 8192), (2, 8200), (1, 16384), (2, 16385), (2, 28672), (1, 40000), (1, 131072),
        (1030, 64), (1025, 333), (1500, 512), (2100, 1541), (1100, 2048), (1030, 5120), (1024, 12000)]


def _norm_inputs(t, k, dtype, seed, offset=0.5):
    rng = np.random.default_rng(seed)
    x, xv = _dev(rng.standard_normal((t, k)) * 2 + offset, dtype)
    return rng, x, xv, rng.standard_normal(k).astype(np.float32), rng.standard_normal(k).astype(np.float32)


def _between(got, a, b, dtype, name):
    """got between a and b (fp32, almost always the same number), all rounded to the type."""
    a, b, g = to_np(_rounded(a, dtype).double()), to_np(_rounded(b, dtype).double()), to_np(got.double())
    bad = ~((np.minimum(a, b) <= g) & (g <= np.maximum(a, b)))
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4].tolist(), g[bad][:4], a[bad][:4], b[bad][:4])


def _check_norm(x, w, b, center, y, ty, mean, rstd):
    """mean, rstd and y: the oracle's, or its neighbour where fp64 sums in another order lead across the border
    of a rounding; every later step is the same fp32 operation (and grows or falls with the mean)."""
    rm, rr = S.norm_stats(x, 1e-5, center)
    dm, dr = S.norm_slack(x, 1e-5, center)
    _between(mean, (rm - dm).astype(np.float32), (rm + dm).astype(np.float32), "float32", "mean")
    _between(rstd, (rr * (1 - dr)).astype(np.float32), (rr * (1 + dr)).astype(np.float32), "float32", "rstd")
    _between(y, *(S.norm_apply(x, m, to_np(rstd), w, b) for m in (rm - dm, rm + dm)), ty, "y")


@pytest.mark.parametrize("tx,ty", PAIRS)
@pytest.mark.parametrize("t,k", NORM)
def test_norm_matches_oracle(t, k, tx, ty):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"norm t={t} k={k} {tx}->{ty}")
    rng, x, xv, w, b = _norm_inputs(t, k, tx, [80, t, k])
    for center, wt, bt in [(True, w, b), (False, w, None), (True, None, b)]:
        out = Guarded()
        y, mean, rstd = out.new((t, k), ty), out.new((t,), "float32"), out.new((t,), "float32")
        sbl.sbl_norm_forward(x, None if wt is None else _f32(wt), None if bt is None else _f32(bt), 1e-5, center, y=y,
                             mean=mean, rstd=rstd)
        torch.cuda.synchronize()
        _check_norm(xv, wt, bt, center, y, ty, mean, rstd)
        out.check()


@pytest.mark.parametrize("tx,ty", PAIRS)
@pytest.mark.parametrize("t,k", [(t, k) for t, k in NORM if k % 64 == 0])
def test_norm_with_quantizer_is_norm_and_quant_acts(t, k, tx, ty):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"norm_quant t={t} k={k} {tx}->{ty}")
    rng, x, xv, w, b = _norm_inputs(t, k, tx, [81, t, k])
    xv, row = xv.copy(), t // 2
    x[row] = 0.0                                        # a row of zeros: gamma from the bias alone
    xv[row] = 0.0
    y32, mean32, rstd32 = sbl.norm(x, _f32(w), _f32(b), dtype=torch.float32)
    _check_norm(xv, w, b, True, y32, "float32", mean32, rstd32)
    rq, rg = O.quant_acts(to_np(y32))
    out = Guarded()
    y, xq = out.new((t, k), ty), out.new((t, k), "int8")
    gamma, mean, rstd = (out.new((t,), "float32") for _ in range(3))
    for want_y in (y, None):
        sbl.sbl_norm_forward(x, _f32(w), _f32(b), 1e-5, True, y=want_y, xq=xq, gamma=gamma, mean=mean, rstd=rstd)
        torch.cuda.synchronize()
        _same(gamma, torch.from_numpy(rg), "gamma")
        _same(xq, torch.from_numpy(rq), "xq")
        xq.zero_()
        gamma.zero_()
    _same(y, y32.to(_type(ty)).cpu(), "y")
    _same(mean, mean32.cpu(), "mean")
    _same(rstd, rstd32.cpu(), "rstd")
    out.check()
    xq2, gamma2, y2, mean2, rstd2 = sbl.norm_quant(x, _f32(w), _f32(b), dtype=torch.float32)
    q, g = sbl.quant_acts(y2)
    assert torch.equal(q, xq2) and torch.equal(g, gamma2)


@pytest.mark.parametrize("center", [True, False])
def test_norm_far_from_zero(center):
    """A mean many times the spread, constant rows, one strong value, subnormal and huge rows."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    rng = np.random.default_rng(82)
    k = 1000
    x = rng.standard_normal((8, k)).astype(np.float32)
    x[1] += 1e4
    x[2] = 7.25
    x[3, 500] = 1e6
    x[4] *= 1e-40
    x[5] *= 1e18
    x[6, 0] = 1e5                                       # the value that the sums are shifted by is the odd one out
    x[7] = 0.0
    y, mean, rstd = sbl.norm(_f32(x), center=center)
    ry, rm, rr = S.norm_forward(x, None, None, 1e-5, center)
    # rows 1 and 6: the shifted sums cancel (a mean 10^4 times the spread, a shift 10^5 times it, in 64 bits: 10^-6 of
    # the sums' rounding of 2^-53 k at most), so a result may fall to the other side of a rounding; 2 units there
    _near(mean, rm, 2 * S.U32 * np.abs(rm), "float32", "mean")
    _near(rstd, rr, 2 * S.U32 * np.abs(rr), "float32", "rstd")
    _near(y, ry, 4 * S.U32 * np.abs(ry), "float32", "y")
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("tx,td", PAIRS)
@pytest.mark.parametrize("t,k", NORM)
def test_norm_backward_matches_oracle(t, k, tx, td):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"norm_backward t={t} k={k} {tx} {td}")
    rng, x, xv, w, _ = _norm_inputs(t, k, tx, [83, t, k])
    dy, dv = _dev(rng.standard_normal((t, k)), td)
    for center, wt in [(True, w), (False, None)]:
        mean, rstd = (s.astype(np.float32) for s in S.norm_stats(xv, 1e-5, center))
        (rx, rw, rb), (ex, ew, eb) = S.norm_backward(dv, xv, mean, rstd, wt, center)
        out = Guarded()
        dx, dw, db = out.new((t, k), tx), out.new((k,), "float32"), out.new((k,), "float32")
        args = (dy, x, _f32(mean) if center else None, _f32(rstd), None if wt is None else _f32(wt))
        ws = _dirty(sbl.sbl_norm_workspace_bytes(t, k))
        sbl.sbl_norm_backward(*args, dx, dw, db, ws, center=center)
        torch.cuda.synchronize()
        _near(dx, rx, ex, tx, "dx")
        _near(dw, rw, ew, "float32", "dw")
        _near(db, rb, eb, "float32", "db")
        out.check()
        # each output alone, the same bits
        first = [to_np(o.double()) for o in (dx, dw, db)]
        for i in range(3):
            one = [None] * 3
            one[i] = torch.full_like((dx, dw, db)[i], 3.0)
            sbl.sbl_norm_backward(*args, *one, ws, center=center)
            assert np.array_equal(to_np(one[i].double()), first[i])


# outputs past the caches, in rows that fill a workgroup's vectors and rows that do not, with the weights held in
# registers and read again, up to the widest rows of each kernel
@pytest.mark.parametrize("tx,ty", [("bfloat16", "float32"), ("float32", "float32"), ("float16", "float16")])
@pytest.mark.parametrize("t,k", [(1650, 5120), (1700, 5184), (1100, 8192), (1100, 8640), (1100, 13824), (1100, 17344),
                                 (1030, 28672), (1030, 32768)])
def test_norm_of_many_wide_rows(t, k, tx, ty):
    test_norm_matches_oracle(t, k, tx, ty)
    test_norm_with_quantizer_is_norm_and_quant_acts(t, k, tx, ty)
    test_norm_backward_matches_oracle(t, k, tx, ty)


def test_norm_backward_is_the_forwards_slope():
    """Central differences of the forward itself, in fp32 (a step of 2^-6 of the values' size: the difference of two
    sums of 64 products, each off by some 2^-24, over 2^-5)."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    rng = np.random.default_rng(84)
    x, w, b = rng.standard_normal((1, 64)), rng.standard_normal(64), rng.standard_normal(64)
    dy = rng.standard_normal((1, 64))
    y, mean, rstd = sbl.norm(_f32(x), _f32(w), _f32(b))
    dx, dw, db = sbl.norm_backward(_f32(dy), _f32(x), mean, rstd, _f32(w), want_bias=True)

    def loss(x, w, b):
        return float((to_np(sbl.norm(_f32(x), _f32(w), _f32(b))[0]).astype(np.float64) * dy).sum())

    h = 2.0 ** -6
    # truncation: h^2 / 6 times the third derivative (a few times rstd^3 |w dy|), rounding: 64 * 4 * 2^-24 * 4 / 2h
    for i, (at, grad) in enumerate(((x, to_np(dx)), (w, to_np(dw)), (b, to_np(db)))):
        for j in list(np.ndindex(at.shape))[::7]:
            args = [x.copy(), w.copy(), b.copy()]
            args[i][j] += h
            up = loss(*args)
            args[i][j] -= 2 * h
            assert abs((up - loss(*args)) / (2 * h) - float(grad[j])) < h * h * 10 + 64 * 4 * S.U32 * 4 / (2 * h)


def _at(values, off):
    """A tensor that begins `off` elements into a larger one of NaNs."""
    import torch
    raw = torch.full((values.numel() + off + 64,), float("nan"), dtype=values.dtype, device="cuda")
    view = raw[off:off + values.numel()].view(values.shape)
    view.copy_(values)
    return view


@pytest.mark.parametrize("tx,ty", [("bfloat16", "float32"), ("float32", "float32"), ("float16", "float16")])
@pytest.mark.parametrize("t,k", [(3, 2), (5, 63), (2, 4096), (1100, 5120), (1100, 8640), (2, 33000)])
def test_norm_of_tensors_anywhere_in_a_buffer(t, k, tx, ty):
    """Parameters and statistics at any 4 bytes, rows at any 16: the results of aligned ones (outputs that then are no
    whole lines are stored otherwise), and nothing beside them is read or written."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"norm anywhere t={t} k={k} {tx} {ty}")
    rng, x, _, w, b = _norm_inputs(t, k, tx, [88, t, k])
    dy = _dev(rng.standard_normal((t, k)), ty)[0]
    w, b, to = _f32(w), _f32(b), _type(ty)
    y, mean, rstd = sbl.norm(x, w, b, dtype=to)
    want = sbl.norm_backward(dy, x, mean, rstd, w, want_bias=True)
    rows = 16 // x.element_size(), 16 // y.element_size()
    x2, dy2, w2, b2 = _at(x, rows[0]), _at(dy, 3 * rows[1]), _at(w, 1), _at(b, 3)
    out = Guarded()
    y2, mean2, rstd2 = out.new((t, k), ty, at=272), out.new((t,), "float32", at=268), out.new((t,), "float32", at=260)
    sbl.sbl_norm_forward(x2, w2, b2, y=y2, mean=mean2, rstd=rstd2)
    for got, ref in ((y2, y), (mean2, mean), (rstd2, rstd)):
        assert torch.equal(got, ref)
    dx2, dw2, db2 = out.new((t, k), tx, at=304), out.new((k,), "float32", at=260), out.new((k,), "float32", at=268)
    sbl.sbl_norm_backward(dy2, x2, mean2, rstd2, w2, dx2, dw2, db2, sbl.new_norm_workspace(t, k))
    for got, ref in zip((dx2, dw2, db2), want):
        assert torch.equal(got, ref)
    out.check()


@pytest.mark.parametrize("t,k", [(5, 64), (1500, 512), (1100, 5120), (3, 40000 // 64 * 64)])
def test_norm_of_rows_that_are_not_finite(t, k):
    """They spoil nothing but themselves."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    rng, x, _, w, b = _norm_inputs(t, k, "bfloat16", [89, t, k])
    w, b = _f32(w), _f32(b)
    dy = _dev(rng.standard_normal((t, k)), "float32")[0]
    want = sbl.norm_quant(x, w, b, dtype=torch.float32)
    gx = sbl.norm_backward(dy, x, want[3], want[4], w)[0]
    bad = torch.tensor([1, t - 1], device="cuda")
    x[1, k // 2], x[t - 1, 0] = float("nan"), float("inf")
    got = sbl.norm_quant(x, w, b, dtype=torch.float32)
    keep = torch.ones(t, dtype=torch.bool, device="cuda")
    keep[bad] = False
    for a, r in zip(got, want):
        assert torch.equal(a[keep], r[keep])
    assert not torch.isfinite(got[2][bad]).any()
    assert torch.equal(sbl.norm_backward(dy, x, got[3], got[4], w)[0][keep], gx[keep])


def test_norm_of_no_rows():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    x = torch.empty((0, 72), dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = sbl.norm(x)
    assert y.shape == (0, 72) and mean.numel() == 0
    dx, dw, db = sbl.norm_backward(x, x, mean, rstd, want_bias=True)
    assert dx.shape == (0, 72) and not dw.any() and not db.any() and dw.shape == (72,)


# ---------------------------------------------------------------- embedding

EMBED = [(1, 1, 1), (5, 3, 2), (64, 10, 8), (9, 1000, 63), (37, 3200, 200), (300, 7, 1541), (513, 70001, 24), (64, 300, 4104),
         (2500, 50, 40), (4099, 900, 136), (3000, 2, 9), (20000, 5000, 16), (777, 257, 5000), (70000, 300, 8)]


def _ids(rng, t, v, skew):
    """Ids of which some come often; a few out of the table on both sides."""
    ids = (v * rng.random(t) ** skew).astype(np.int64)
    ids[rng.random(t) < 0.1] = -1
    if t > 8:
        ids[2], ids[3], ids[4], ids[5] = -100, v, v + 5, -(1 << 62)
        ids[6], ids[7] = (1 << 62), v - 1
    return ids


@pytest.mark.parametrize("tt,to", PAIRS)
@pytest.mark.parametrize("t,v,k", EMBED)
def test_embedding_matches_oracle(t, v, k, tt, to):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"embed t={t} v={v} k={k} {tt}->{to}")
    rng = np.random.default_rng([85, t, v, k])
    table, tv = _dev(rng.standard_normal((v, k)), tt)
    ids = _ids(rng, t, v, 2)
    for scale in (1.0, 3.7):
        out = Guarded()
        o = out.new((t, k), to)
        sbl.sbl_embed_forward(_i64(ids), table, o, scale)
        torch.cuda.synchronize()
        _same(o, _rounded(S.embed(ids, tv, scale), to), "out")
        out.check()


@pytest.mark.parametrize("skew", [1, 6])
@pytest.mark.parametrize("tt,to", PAIRS)
@pytest.mark.parametrize("t,v,k", EMBED)
def test_embedding_backward_matches_oracle(t, v, k, tt, to, skew):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"embed_backward t={t} v={v} k={k} {tt} {to} skew={skew}")
    rng = np.random.default_rng([86, t, v, k, skew])
    ids = _ids(rng, t, v, skew)
    dout, dv = _dev(rng.standard_normal((t, k)), to)
    old, ov = _dev(rng.standard_normal((v, k)), tt)
    gone = (ids < 0) | (ids >= v)
    dout[_i64(np.nonzero(gone)[0])] = float("nan")       # must reach nothing
    ws = _dirty(sbl.sbl_embed_workspace_bytes(t, v, k, _type(to)))
    for scale, add in ((1.0, False), (1.7, True), (0.3, False)):
        out = Guarded()
        d = out.new((v, k), tt, fill=old if add else None)
        sbl.sbl_embed_backward(_i64(ids), dout, d, ws, scale, add)
        torch.cuda.synchronize()
        want, bound = S.embed_backward(ids, dv, v, scale, ov if add else None)
        _near(d, want, bound, tt, "dtable")
        empty = np.bincount(ids[~gone], minlength=v) == 0
        if add:
            assert torch.equal(d[_i64(np.nonzero(empty)[0])], old[_i64(np.nonzero(empty)[0])])
        out.check()
        again = old.clone() if add else torch.full_like(d, 7.0)
        sbl.sbl_embed_backward(_i64(ids), dout, again, ws, scale, add)
        assert torch.equal(again, d)


# one id, two and 1024 of each sorting workgroup, one more than that; ids that a wave remembers and more
@pytest.mark.parametrize("tt,to", [("bfloat16", "bfloat16"), ("float32", "float16")])
@pytest.mark.parametrize("skew", [1, 9])
@pytest.mark.parametrize("t,v", [(5000, 255), (5000, 256), (20000, 257), (13000, 4097), (1024, 300), (1025, 300), (5000, 262143), (5000, 262144),
                                 (5000, 262145), (60000, 131072)])
def test_embedding_backward_around_the_sorts_ranges(t, v, skew, tt, to):
    test_embedding_backward_matches_oracle(t, v, 5, tt, to, skew)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("t", [1, 7, 8, 9, 16, 17, 63, 64, 65, 640, 1000, 4096])
def test_embedding_backward_of_one_id(t, add):
    """Every token has the same id: one run over every segment, and rows of ones, so that the sum is exact."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v, k = 40, 72
    for at in (0, 17, 39):
        ids = torch.full((t,), at, dtype=torch.int64, device="cuda")
        dout = torch.ones((t, k), dtype=torch.bfloat16, device="cuda")
        old = torch.full((v, k), 2.0, dtype=torch.bfloat16, device="cuda") if add else None
        d = sbl.embed_backward(ids, dout, v, scale=0.5, add_to=old)
        want = torch.full((v, k), 2.0 if add else 0.0)
        want[at] += 0.5 * t
        _same(d, want.to(torch.bfloat16), "dtable")


@pytest.mark.parametrize("tt,to", [("bfloat16", "bfloat16"), ("float32", "float16"), ("float16", "float32")])
@pytest.mark.parametrize("t,v,k", [(9, 20, 3), (4500, 700, 1024), (1200, 3000, 8640), (5000, 300, 1541)])
def test_embedding_of_tensors_anywhere_in_a_buffer(t, v, k, tt, to):
    """Rows at any 16 bytes: the results of aligned tensors, and nothing beside them is read or written."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"embed anywhere t={t} v={v} k={k} {tt} {to}")
    rng = np.random.default_rng([90, t, v, k])
    table, dout = _dev(rng.standard_normal((v, k)), tt)[0], _dev(rng.standard_normal((t, k)), to)[0]
    ids = _i64(_ids(rng, t, v, 3))
    table2, dout2 = _at(table, 16 // table.element_size()), _at(dout, 48 // dout.element_size())
    ids2 = torch.full((t + 3,), 1, dtype=torch.int64, device="cuda")[1:t + 1].copy_(ids)
    out = Guarded()
    rows = out.new((t, k), to, at=272)
    sbl.sbl_embed_forward(ids2, table2, rows, 1.5)
    _same(rows, sbl.embed(ids, table, 1.5, dtype=_type(to)).cpu(), "rows")
    ws = sbl.new_embed_workspace(t, v, k, _type(to))
    for add in (False, True):
        want = table.clone()
        sbl.sbl_embed_backward(ids, dout, want, ws, 0.7, add)
        grad = out.new((v, k), tt, at=304, fill=table)
        sbl.sbl_embed_backward(ids2, dout2, grad, ws, 0.7, add)
        assert torch.equal(grad, want)
    out.check()


def test_embedding_of_no_tokens_and_any_shape():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    table = torch.randn(50, 13, device="cuda")
    none = torch.empty((0,), dtype=torch.int64, device="cuda")
    assert sbl.embed(none, table).shape == (0, 13)
    d = sbl.embed_backward(none, torch.empty((0, 13), device="cuda"), 50)
    assert d.shape == (50, 13) and not d.any()
    kept = table.clone()
    assert sbl.embed_backward(none, torch.empty((0, 13), device="cuda"), 50, add_to=table) is table
    assert torch.equal(table, kept)
    ids = torch.arange(12, device="cuda").view(3, 4)
    assert torch.equal(sbl.embed(ids, table), table[ids])
    gone = torch.full((3, 4), -1, device="cuda")                  # a batch of padding alone
    d = sbl.embed_backward(gone, torch.full((3, 4, 13), float("nan"), device="cuda"), 50)
    assert not d.any() and not sbl.embed(gone, table).any()


def test_embedding_of_a_large_vocabulary():
    """More ids than 256 sorting workgroups hold, rows at both ends of the table."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v, k, t = 600001, 9, 5000
    rng = np.random.default_rng(87)
    ids = rng.integers(0, v, t)
    ids[:10], ids[10:20] = 0, v - 1
    dout, dv = _dev(rng.standard_normal((t, k)), "float16")
    d = sbl.embed_backward(_i64(ids), dout, v)
    want, bound = S.embed_backward(ids, dv, v, 1.0)
    _near(d, want, bound, "float16", "dtable")


# ---------------------------------------------------------------- AdamW

ADAM = dict(beta1=0.9, beta2=0.99, eps=1e-8)
WEIGHTS = [("bfloat16", True), ("bfloat16", False), ("float16", False), ("float32", False)]


def _tensor(rng, n, wt, low, gt, bits, shape=None, off=0, decay=0.1, lr_scale=1.0):
    """One tensor's inputs on both sides: the binding's dict and the oracle's arguments.  off: its place, in elements,
    in the larger buffers that it lies in."""
    import torch
    size = np.exp(2 * rng.standard_normal(n))
    w = rng.standard_normal(n).astype(np.float32)
    m = (0.3 * size * rng.standard_normal(n)).astype(np.float32)
    v = ((0.1 * size * rng.random(n)) ** 2).astype(np.float32)
    if n > 3:
        v[1] = m[1] = 0.0
        v[2] = 0.0
    g, gv = _dev(size * rng.standard_normal(n), gt)
    if n > 3:
        g[1] = 0.0
        gv[1] = 0.0
    here = Guarded()
    e = dict(weight_decay=decay, lr_scale=lr_scale, g=here.new((n,), gt, at=256 + off * g.element_size(), fill=g))
    o = dict(g=gv.astype(np.float32), weight_decay=decay, lr_scale=lr_scale)
    if low:
        high, lo = S.split_master(w)
        e["w"] = here.new((n,), "bfloat16", at=256 + 2 * off, fill=torch.from_numpy(high.view(np.int16)).view(torch.bfloat16))
        e["w_low"] = here.new((n,), "int16", at=256 + 2 * off, fill=torch.from_numpy(lo))
        o["w"] = w
    else:
        t, tv = _dev(w, wt)
        e["w"] = here.new((n,), wt, at=256 + off * t.element_size(), fill=t)
        o["w"] = tv.astype(np.float32)
    if bits == 32:
        e["m"], e["v"] = (here.new((n,), "float32", at=256 + 4 * off, fill=torch.from_numpy(x)) for x in (m, v))
        o["m"], o["v"] = m, v
    else:
        for name, x in (("m", m), ("v", np.sqrt(v))):
            scale, over = S._scales(x)
            codes = S.e4m3_nearest(over)
            e[name] = here.new((n,), "float8_e4m3fn", at=256 + 8 * off, fill=torch.from_numpy(codes).view(torch.float8_e4m3fn))
            e[name + "_scale"] = here.new(scale.shape, "float32", fill=torch.from_numpy(scale))
            o[name], o[name + "_scale"] = codes, scale
    if shape is not None:
        e["w"] = e["w"].view(shape)
    return e, o, here


def _check_tensor(e, o, wt, low, s):
    import torch
    args = {k: o[k] for k in ("m_scale", "v_scale") if k in o}
    got = S.adamw(o["w"], o["g"], o["m"], o["v"], s, ADAM["beta1"], ADAM["beta2"], ADAM["eps"], o["lr_scale"],
                  o["weight_decay"], **args)
    w = got[0]
    if low:
        high, lo = S.split_master(w)
        assert np.array_equal(to_np(e["w"].view(torch.int16)).reshape(-1).view(np.uint16), high)
        assert np.array_equal(to_np(e["w_low"]), lo)
        o["w"] = w
    else:
        want = _rounded(w, wt)
        _same(e["w"].reshape(-1), want, "w")
        o["w"] = want.float().numpy()
    for name, x in zip(("m", "v", "m_scale", "v_scale"), got[1:]):
        t = e[name]
        have = to_np(t.view(torch.uint8)) if x.dtype == np.uint8 else to_np(t)
        assert np.array_equal(have, x), (name, int((have != x).sum()), np.argwhere(have != x)[:4].tolist())
        o[name] = x


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gt", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("wt,low", WEIGHTS)
@pytest.mark.parametrize("n", [1, 3, 4, 255, 256, 257, 1000, 8191, 8192, 8193, 50001])
def test_adamw_matches_oracle(n, wt, low, gt, bits):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"adamw n={n} {wt} low={low} g={gt} bits={bits}")
    e, o, here = _tensor(np.random.default_rng([88, n, bits]), n, wt, low, gt, bits)
    items = sbl.AdamWItems([e])
    for step in (1, 2, 3):
        sbl.sbl_adamw_batch(items, 1e-2, **ADAM, step=step)
        torch.cuda.synchronize()
        _check_tensor(e, o, wt, low, S.schedule(1e-2, ADAM["beta1"], ADAM["beta2"], step))
    here.check()


@pytest.mark.parametrize("off", [1, 2, 3, 5])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_tensors_anywhere_in_a_buffer(off, bits):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    for wt, low, gt in (("bfloat16", True, "bfloat16"), ("float32", False, "float16"), ("float16", False, "float32")):
        e, o, here = _tensor(np.random.default_rng([89, off]), 9001, wt, low, gt, bits, off=off)
        sbl.sbl_adamw_batch([e], 1e-2, **ADAM, step=5)
        torch.cuda.synchronize()
        _check_tensor(e, o, wt, low, S.schedule(1e-2, ADAM["beta1"], ADAM["beta2"], 5))
        here.check()


def test_adamw_of_many_tensors():
    """More than one launch holds, every kind among them, some empty; a shared gradient; factors from the device."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    rng = np.random.default_rng(90)
    made = []
    for i in range(130):
        wt, low = WEIGHTS[i % 4]
        n = int([0, 1, 77, 300, 8192, 20000, 256][i % 7])
        made.append((wt, low, *_tensor(rng, n, wt, low, ("float32", "bfloat16", "float16")[i % 3], (32, 8)[i % 2],
                                       decay=0.1 * (i % 3), lr_scale=1.0 + 0.25 * (i % 2))))
    twin = _tensor(rng, 300, "float32", False, "float32", 32)
    twin[0]["g"] = made[3][2]["g"] if made[3][2]["g"].dtype == torch.float32 else twin[0]["g"]
    twin[1]["g"] = to_np(twin[0]["g"].float())
    made.append(("float32", False, *twin))
    s = sbl.adamw_schedule(3e-3, ADAM["beta1"], ADAM["beta2"], 11, 0.37)
    schedule = Guarded().new((5,), "float32", fill=s)
    items = sbl.AdamWItems([m[2] for m in made])
    sbl.sbl_adamw_batch(items, float("nan"), **ADAM, step=-3, schedule=schedule)
    torch.cuda.synchronize()
    for i, (wt, low, e, o, here) in enumerate(made):
        if e["w"].numel():
            _check_tensor(e, o, wt, low, S.schedule(3e-3, ADAM["beta1"], ADAM["beta2"], 11, 0.37))
        here.check()


def test_adamw_from_the_state_before_the_first_step():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    rng = np.random.default_rng(91)
    for bits in (32, 8):
        w, wv = _dev(rng.standard_normal((30, 41)), "float32")
        g, gv = _dev(rng.standard_normal((30, 41)) * 1e-3, "float32")
        e = dict(w=w, g=g, **sbl.adamw_state(w, bits))
        sbl.sbl_adamw_batch([e], 1e-2, 0.9, 0.99, 1e-8, 1)
        # the first step moves every weight by lr, whatever the gradient's size: m bias1 / (sqrt(v) bias2 + eps) is 1 but
        # for eps and some 20 roundings; the new weight is rounded once more
        moved = wv - to_np(w).astype(np.float64)
        allowed = 1e-2 * (1e-8 / np.abs(gv) + 20 * S.U32) + 2 * S.U32 * np.abs(wv)
        assert (np.abs(moved - 1e-2 * np.sign(gv)) <= allowed).all()


def test_adamw_spoils_only_what_is_not_finite():
    """A gradient that is not finite spoils its value, in 8 bits its block of 256."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    for bits, blast in ((32, 1), (8, 256)):
        rng = np.random.default_rng(92)
        e, o, _ = _tensor(rng, 5000, "float32", False, "float32", bits)
        for at, bad in ((700, float("nan")), (2000, float("inf")), (4000, float("-inf"))):
            e["g"][at] = bad
            o["g"][at] = 0.0
        sbl.sbl_adamw_batch([e], 1e-2, **ADAM, step=3)
        with np.errstate(all="ignore"):
            args = {k: o[k] for k in ("m_scale", "v_scale") if k in o}
            want = S.adamw(o["w"], o["g"], o["m"], o["v"], S.schedule(1e-2, ADAM["beta1"], ADAM["beta2"], 3), ADAM["beta1"],
                           ADAM["beta2"], ADAM["eps"], 1.0, o["weight_decay"], **args)
        fine = np.ones(5000, bool)
        for at in (700, 2000, 4000):
            fine[at // blast * blast:at // blast * blast + blast] = False
        assert np.array_equal(to_np(e["w"])[fine], want[0][fine])
        for name, x in zip(("m", "v"), want[1:]):
            have = to_np(e[name].view(torch.uint8)) if bits == 8 else to_np(e[name])
            assert np.array_equal(have[fine], x[fine])


# ---------------------------------------------------------------- streams, graphs, the binding

def test_binding_refuses_on_the_gpu():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    x = torch.zeros((4, 64), device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    stat = torch.zeros(4, device="cuda")
    bad = [lambda: sbl.norm(x, weight=torch.zeros(63, device="cuda")), lambda: sbl.norm(x.t()),
           lambda: sbl.norm(x, weight=torch.zeros(64, device="cuda", dtype=torch.bfloat16)),
           lambda: sbl.norm_quant(torch.zeros((4, 65), device="cuda")), lambda: sbl.norm(x, eps=0.0),
           lambda: sbl.norm_backward(x[:3], x, stat, stat), lambda: sbl.norm_backward(x, x, stat[:3], stat),
           lambda: sbl.norm_backward(x, x, stat, stat, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: sbl.embed(ids.int(), x), lambda: sbl.embed(ids, x[0]), lambda: sbl.embed(ids, x.double()),
           lambda: sbl.embed_backward(ids, x, 10, add_to=torch.zeros((9, 64), device="cuda")),
           lambda: sbl.embed_backward(ids, x, 10, dtype=torch.int32), lambda: sbl.embed_backward(ids[:3], x, 10),
           lambda: sbl.embed_backward(ids, x, 10, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: sbl.embed_backward(ids, x, 10, add_to=torch.zeros((10, 64), device="cuda").bfloat16().to(torch.int16)),
           lambda: sbl.sbl_embed_forward(ids, x, x), lambda: sbl.sbl_norm_forward(x, y=x),
           lambda: sbl.AdamWItems([dict(w=x, g=x[:3], m=x, v=x)]), lambda: sbl.AdamWItems([dict(w=x, g=x, m=x, v=x.bfloat16())]),
           lambda: sbl.sbl_adamw_batch([dict(w=x, g=x.clone(), m=x.clone(), v=x)], 1e-3, 0.9, 0.99, 1e-8, 1),
           lambda: sbl.AdamWItems([dict(w=x, g=x, **{**sbl.adamw_state(x, 8), "m_scale": None})]) and None or
           sbl.sbl_adamw_batch([dict(w=x, g=x.clone(), **{**sbl.adamw_state(x, 8), "m_scale": None})], 1e-3, 0.9, 0.99, 1e-8, 1)]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, sbl.SblError)):
            say(f"refusal {i}")
            call()


def test_calls_on_a_stream_of_the_callers():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    torch.manual_seed(0)
    s = torch.cuda.Stream()
    x, ids = torch.randn(300, 640, device="cuda"), torch.randint(0, 50, (300,), device="cuda")
    here = sbl.norm_quant(x, eps=1e-5)
    back = sbl.norm_backward(here[2], x, here[3], here[4])
    table = torch.randn(50, 640, device="cuda")
    rows, grad = sbl.embed(ids, table), sbl.embed_backward(ids, x, 50)
    torch.cuda.synchronize()
    there = sbl.norm_quant(x, eps=1e-5, stream=s)
    back2 = sbl.norm_backward(there[2], x, there[3], there[4], stream=s)
    rows2, grad2 = sbl.embed(ids, table, stream=s), sbl.embed_backward(ids, x, 50, stream=s.cuda_stream)
    s.synchronize()
    for a, b in zip((*here, *back[:2], rows, grad), (*there, *back2[:2], rows2, grad2)):
        assert torch.equal(a, b)


def test_a_step_replays_from_a_graph():
    """Lookup, norm with quantizer, both backwards and the update, captured: every replay, with eager work and
    synchronizations between, gives what eager steps give; the schedule is read when the step runs."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    torch.manual_seed(1)
    t, v, k = 200, 333, 320
    ids = torch.randint(0, v, (t,), device="cuda")
    dy = torch.randn(t, k, device="cuda")

    def fresh():
        torch.manual_seed(2)
        w = torch.randn(v, k, device="cuda")
        high, low = sbl.split_master(w)
        scale = torch.ones(k, device="cuda")
        return dict(table=dict(w=high, w_low=low, weight_decay=0.1, **sbl.adamw_state(w, 8)),
                    norm=dict(w=scale, **sbl.adamw_state(scale)))

    def buffers():
        return dict(x=torch.empty((t, k), device="cuda"), xq=torch.empty((t, k), dtype=torch.int8, device="cuda"),
                    gamma=torch.empty(t, device="cuda"), mean=torch.empty(t, device="cuda"), rstd=torch.empty(t, device="cuda"),
                    dx=torch.empty((t, k), device="cuda"), dw=torch.empty(k, device="cuda"),
                    dtable=torch.empty((v, k), device="cuda"), ws1=_dirty(sbl.sbl_norm_workspace_bytes(t, k)),
                    ws2=_dirty(sbl.sbl_embed_workspace_bytes(t, v, k, torch.float32)), schedule=torch.zeros(5, device="cuda"))

    def step(p, b, items):
        sbl.sbl_embed_forward(ids, p["table"]["w"], b["x"])
        sbl.sbl_norm_forward(b["x"], p["norm"]["w"], xq=b["xq"], gamma=b["gamma"], mean=b["mean"], rstd=b["rstd"])
        sbl.sbl_norm_backward(dy, b["x"], b["mean"], b["rstd"], p["norm"]["w"], b["dx"], b["dw"], None, b["ws1"])
        sbl.sbl_embed_backward(ids, b["dx"], b["dtable"], b["ws2"])
        sbl.sbl_adamw_batch(items, 0.0, 0.9, 0.99, 1e-8, 0, schedule=b["schedule"])

    def setup():
        p, b = fresh(), buffers()
        p["table"]["g"], p["norm"]["g"] = b["dtable"], b["dw"]
        return p, b, sbl.AdamWItems(list(p.values()))

    def values(p, b):
        torch.cuda.synchronize()
        return [x.clone().view(torch.uint8).cpu() for e in p.values() for n, x in sorted(e.items())
                if isinstance(x, torch.Tensor)] + [b["xq"].cpu().view(torch.uint8)]

    schedules = [sbl.adamw_schedule(1e-2 / n, 0.9, 0.99, n, 1.0 / n) for n in range(1, 6)]
    p, b, items = setup()
    want = []
    for s in schedules:
        b["schedule"].copy_(s)
        step(p, b, items)
        want.append(values(p, b))
    p, b, items = setup()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(p, b, items)
    assert torch.equal(p["norm"]["w"], torch.ones(k, device="cuda"))
    for s, w in zip(schedules, want):
        b["schedule"].copy_(s)
        graph.replay()
        got = values(p, b)
        assert len(got) == len(w) and all(torch.equal(x, y) for x, y in zip(got, w))
        torch.randn(1000, 1000, device="cuda").sum().item()          # other work between replays


def test_two_backwards_at_once():
    """Calls on two streams with workspaces of their own."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    torch.manual_seed(3)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    jobs = []
    for i in range(2):
        ids = torch.randint(0, 2000, (5000,), device="cuda")
        dout, x = torch.randn(5000, 512, device="cuda").bfloat16(), torch.randn(5000, 512, device="cuda")
        mean, rstd = sbl.norm(x)[1:]
        jobs.append((ids, dout, x, mean, rstd))
    alone = [(sbl.embed_backward(j[0], j[1], 2000), *sbl.norm_backward(j[2], j[2], j[3], j[4])[:2]) for j in jobs]
    torch.cuda.synchronize()
    for _ in range(3):
        both = []
        for j, s in zip(jobs, streams):
            both.append((sbl.embed_backward(j[0], j[1], 2000, stream=s),
                         *sbl.norm_backward(j[2], j[2], j[3], j[4], stream=s)[:2]))
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
