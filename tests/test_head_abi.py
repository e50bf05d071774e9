"""CPU checks of the output head's C ABI: workspace sizes and the refusals of
bad arguments on the host, before any HIP call."""

import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sparse_linear_layers_absmean_amd", "libsbl.so")

OK, NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 6
# fake device addresses, far apart, never dereferenced: every call below must be
# refused on the host.  Not run on a machine with a GPU, where a validation bug
# could reach a kernel.
needs_no_gpu = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="fake addresses: only where no GPU is")
GB = 1 << 30
H, W, T, X, L, S, D, E, DH, DW, WS = (GB * 16 * i for i in range(1, 12))
BIG = 1 << 33


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("libsbl.so is not built (run __graft_entry__.build())")
    import torch  # noqa: F401
    from sparse_linear_layers_absmean_amd import sbl
    return sbl.load()


def _ce_fwd(lib, **kw):
    a = dict(h=H, hs=64, w=W, dtype=0, target=T, m=8, v=100, k=64, loss=L, lse=S, ws=WS, wsb=BIG)
    a.update(kw)
    return lib.sbl_head_ce_forward(a["h"], a["hs"], a["w"], a["dtype"], a["target"], a["m"], a["v"], a["k"], a["loss"],
                                   a["lse"], a["ws"], a["wsb"], None)


def _ce_bwd(lib, **kw):
    a = dict(h=H, hs=64, w=W, dtype=0, target=T, lse=S, dloss=D, dlse=E, m=8, v=100, k=64, dh=DH, dw=DW, ws=WS, wsb=BIG)
    a.update(kw)
    return lib.sbl_head_ce_backward(a["h"], a["hs"], a["w"], a["dtype"], a["target"], a["lse"], a["dloss"], a["dlse"],
                                    a["m"], a["v"], a["k"], a["dh"], a["dw"], a["ws"], a["wsb"], None)


def _kd_fwd(lib, **kw):
    a = dict(h=H, hs=64, w=W, dtype=0, index=T, teacher=X, top=4, tau=2.0, m=8, v=100, k=64, loss=L, lse=S, ws=WS,
             wsb=BIG)
    a.update(kw)
    return lib.sbl_head_kd_forward(a["h"], a["hs"], a["w"], a["dtype"], a["index"], a["teacher"], a["top"], a["tau"],
                                   a["m"], a["v"], a["k"], a["loss"], a["lse"], a["ws"], a["wsb"], None)


def _kd_bwd(lib, **kw):
    a = dict(h=H, hs=64, w=W, dtype=0, index=T, teacher=X, top=4, tau=2.0, lse=S, dloss=D, m=8, v=100, k=64, dh=DH,
             dw=DW, ws=WS, wsb=BIG)
    a.update(kw)
    return lib.sbl_head_kd_backward(a["h"], a["hs"], a["w"], a["dtype"], a["index"], a["teacher"], a["top"], a["tau"],
                                    a["lse"], a["dloss"], a["m"], a["v"], a["k"], a["dh"], a["dw"], a["ws"], a["wsb"],
                                    None)


CALLS = {"ce_fwd": _ce_fwd, "ce_bwd": _ce_bwd, "kd_fwd": _kd_fwd, "kd_bwd": _kd_bwd}


@needs_no_gpu
@pytest.mark.parametrize("call", sorted(CALLS))
@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), SHAPE), (dict(m=(1 << 22) + 1), SHAPE), (dict(v=0), SHAPE), (dict(v=1 << 31), SHAPE),
    (dict(k=0, hs=0), SHAPE), (dict(k=60), SHAPE), (dict(k=131080, hs=131080), SHAPE),
    (dict(v=(1 << 34) // 64 + 1), SHAPE),                       # n_vocab * k
    (dict(m=1 << 18, k=4096, hs=4096), SHAPE),                  # (m_tok + 256) * k
    (dict(m=1 << 22, v=1 << 24), SHAPE),                        # m_tok * n_vocab
    (dict(hs=56), SHAPE), (dict(hs=68), SHAPE), (dict(m=9, hs=1 << 27), SHAPE),
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED),
    (dict(h=None), NULL), (dict(w=None), NULL), (dict(ws=None), WORKSPACE), (dict(wsb=0), WORKSPACE),
    (dict(h=H + 2), ALIGN), (dict(w=W + 8), ALIGN), (dict(ws=WS + 16), ALIGN),
    (dict(ws=W), SHAPE), (dict(ws=H), SHAPE),
])
def test_refusals_of_every_call(lib, call, kw, status):
    assert CALLS[call](lib, **kw) == status


@needs_no_gpu
@pytest.mark.parametrize("call", ["ce_fwd", "kd_fwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(loss=None), NULL), (dict(lse=None), NULL), (dict(loss=L + 2), ALIGN), (dict(lse=S + 1), ALIGN),
    (dict(loss=S), SHAPE), (dict(loss=H), SHAPE), (dict(lse=W + 64), SHAPE), (dict(loss=T), SHAPE), (dict(lse=WS), SHAPE),
    (dict(m=0, h=None, target=None, index=None, loss=None), OK),
])
def test_refusals_of_the_forward(lib, call, kw, status):
    assert CALLS[call](lib, **kw) == status


@needs_no_gpu
@pytest.mark.parametrize("call", ["ce_bwd", "kd_bwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(lse=None), NULL), (dict(dloss=None), NULL), (dict(lse=S + 2), ALIGN), (dict(dloss=D + 2), ALIGN),
    (dict(dh=DH + 8), ALIGN), (dict(dw=DW + 2), ALIGN), (dict(dh=H), SHAPE), (dict(dw=W), SHAPE), (dict(dh=DW), SHAPE),
    (dict(dw=S), SHAPE), (dict(dh=D), SHAPE), (dict(dw=WS), SHAPE), (dict(ws=S), SHAPE), (dict(dh=T), SHAPE),
    (dict(dh=None, dw=None), OK), (dict(m=0, dw=None), OK), (dict(m=0, dw=DW + 8), ALIGN),
])
def test_refusals_of_the_backward(lib, call, kw, status):
    assert CALLS[call](lib, **kw) == status


@needs_no_gpu
def test_refusals_of_the_lists(lib):
    assert _ce_fwd(lib, target=None) == NULL and _ce_bwd(lib, target=None) == NULL
    assert _ce_fwd(lib, target=T + 4) == ALIGN and _ce_bwd(lib, dlse=E + 2) == ALIGN
    assert _ce_bwd(lib, dh=E) == SHAPE
    for call in (_kd_fwd, _kd_bwd):
        assert call(lib, index=None) == NULL and call(lib, teacher=None) == NULL
        assert call(lib, index=T + 4) == ALIGN and call(lib, teacher=X + 2) == ALIGN
        assert call(lib, top=0) == SHAPE and call(lib, top=257) == SHAPE
        for tau in (0.0, -1.0, 1e-5, 1e5, float("inf"), float("nan")):
            assert call(lib, tau=tau) == SHAPE


def test_workspace_bytes(lib):
    f = lib.sbl_head_workspace_bytes
    assert f(8, 100, 60, 1, 0) == -1 and f(8, 100, 64, 0, 0) == -1 and f(8, 100, 64, 257, 1) == -1
    assert f(-1, 100, 64, 1, 0) == -1 and f(0, 100, 64, 1, 0) > 0 and f(0, 100, 64, 1, 1) > 0
    for t, v, k in [(1, 1, 8), (16, 1000, 256), (2048, 32000, 3200), (4096, 128256, 5120), (65536, 128256, 4096)]:
        fwd, bwd = f(t, v, k, 64, 0), f(t, v, k, 64, 1)
        assert 0 < fwd and f(t, v, k, 1, 0) <= fwd and 0 < bwd
        # never the logits: the forward keeps two words per 32 ids or more (and the
        # lists); the backward 2^28 gradients of 16 bits (256 ids at least) beside
        # copies and partial sums of h
        assert fwd <= t * (8 * (v // 32 + 1) + 4 * 64 + 12 + 2 * 64) + 8 * 4096
        assert f(t, v, k, 1, 1) <= 2 * max(1 << 28, 256 * t) + 2 * t * k * (1 + 2 * 1024) + 32 * t + 16 * 4096



@pytest.mark.parametrize("t,v,k", [(1, 40000000, 8), (7, 44000000, 24), (33, 1 << 26, 16), (64, 1 << 27, 8),
                                   (65, 1 << 27, 8), (1, (1 << 31) - 1025, 8)])
def test_gradients_held_at_a_time(lib, t, v, k):
    """2^28 logit gradients at most, counting the two rows of each of up to 64 tokens
    (64 or 128 rows in all): products read them within 32-bit offsets."""
    splits = 1024                                   # more shares of dh than any plan takes
    rows = t if t > 64 else 64 if t <= 32 else 128
    rest = rows * k * (2 + 4 * splits) + t * 64 + 16 * 4096
    assert lib.sbl_head_workspace_bytes(t, v, k, 1, 1) <= 2 * (1 << 28) + rest
