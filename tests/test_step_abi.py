"""CPU checks of the C ABI of the norm, the embedding and AdamW: workspace
sizes and the refusals of bad arguments on the host, before any HIP call, and
the binding's own refusals."""

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
A, B, C, D, E, F, G, H, I, WS = (GB * 64 * i for i in range(1, 11))
BIG = 1 << 35
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("libsbl.so is not built (run __graft_entry__.build())")
    import torch  # noqa: F401
    from sparse_linear_layers_absmean_amd import sbl
    return sbl.load()


def _norm(lib, **kw):
    a = dict(x=A, xt=0, w=B, b=C, m=8, k=64, eps=1e-5, center=1, y=D, yt=0, xq=E, gamma=F, mean=G, rstd=H)
    a.update(kw)
    return lib.sbl_norm_forward(a["x"], a["xt"], a["w"], a["b"], a["m"], a["k"], a["eps"], a["center"], a["y"], a["yt"],
                                a["xq"], a["gamma"], a["mean"], a["rstd"], None)


def _norm_bwd(lib, **kw):
    a = dict(dy=A, dt=0, x=B, xt=0, mean=C, rstd=D, w=E, m=8, k=64, center=1, dx=F, dw=G, db=H, ws=WS, wsb=BIG)
    a.update(kw)
    return lib.sbl_norm_backward(a["dy"], a["dt"], a["x"], a["xt"], a["mean"], a["rstd"], a["w"], a["m"], a["k"],
                                 a["center"], a["dx"], a["dw"], a["db"], a["ws"], a["wsb"], None)


@needs_no_gpu
@pytest.mark.parametrize("call", [_norm, _norm_bwd])
@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), SHAPE), (dict(m=(1 << 22) + 1), SHAPE), (dict(k=0), SHAPE), (dict(k=131073), SHAPE),
    (dict(m=1 << 20, k=16448), SHAPE), (dict(xt=3), UNSUPPORTED), (dict(xt=-1), UNSUPPORTED),
    (dict(x=None), NULL), (dict(x=A + 2), ALIGN), (dict(w=B + 2), ALIGN), (dict(rstd=H + 1), ALIGN),
    (dict(mean=G + 2), ALIGN),
])
def test_refusals_of_both_norm_calls(lib, call, kw, status):
    assert call(lib, **kw) == status


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(eps=0.0), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE), (dict(eps=INF), SHAPE), (dict(eps=1e-60), SHAPE),
    (dict(xt=0, yt=1), UNSUPPORTED), (dict(xt=1, yt=0), UNSUPPORTED), (dict(xt=1, yt=3), UNSUPPORTED),
    (dict(k=65), SHAPE), (dict(k=32), SHAPE), (dict(xq=None), NULL), (dict(gamma=None), NULL),
    (dict(y=D + 8), ALIGN), (dict(xq=E + 8), ALIGN), (dict(gamma=F + 2), ALIGN), (dict(b=C + 1), ALIGN),
    (dict(y=A), SHAPE), (dict(xq=A + 512), SHAPE), (dict(gamma=B), SHAPE), (dict(mean=C), SHAPE), (dict(rstd=D), SHAPE),
    (dict(xq=D), SHAPE), (dict(rstd=G), SHAPE), (dict(mean=F + 16), SHAPE),
    (dict(m=0, x=None, y=None), OK), (dict(y=None, xq=None, gamma=None, mean=None, rstd=None), OK),
    (dict(k=65, xq=None, gamma=None, y=None, mean=None, rstd=None), OK),
])
def test_refusals_of_the_norm(lib, kw, status):
    assert _norm(lib, **kw) == status


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(dt=1), UNSUPPORTED), (dict(xt=1, dt=0), UNSUPPORTED), (dict(dy=None), NULL), (dict(rstd=None), NULL),
    (dict(mean=None), NULL), (dict(ws=None), WORKSPACE), (dict(wsb=8 * 2 * 64 * 4 - 1), WORKSPACE),
    (dict(dy=A + 8), ALIGN), (dict(dx=F + 2), ALIGN), (dict(dw=G + 2), ALIGN), (dict(db=H + 1), ALIGN), (dict(ws=WS + 64), ALIGN),
    (dict(dx=A), SHAPE), (dict(dx=B + 16), SHAPE), (dict(dw=C), SHAPE), (dict(db=D), SHAPE), (dict(dw=E), SHAPE),
    (dict(db=G), SHAPE), (dict(dx=G), SHAPE), (dict(ws=F), SHAPE), (dict(ws=B), SHAPE),
    (dict(dx=None, dw=None, db=None), OK), (dict(m=0, dw=None, db=None, dx=None, ws=None, dy=None), OK),
    (dict(center=0, mean=None, dx=None, dw=None, db=None), OK),
])
def test_refusals_of_the_norms_backward(lib, kw, status):
    assert _norm_bwd(lib, **kw) == status


def _embed(lib, **kw):
    a = dict(ids=A, table=B, tt=0, m=8, v=100, k=64, scale=1.0, out=C, ot=0)
    a.update(kw)
    return lib.sbl_embed_forward(a["ids"], a["table"], a["tt"], a["m"], a["v"], a["k"], a["scale"], a["out"], a["ot"], None)


def _embed_bwd(lib, **kw):
    a = dict(ids=A, out=B, ot=0, m=8, v=100, k=64, scale=1.0, table=C, tt=0, add=0, ws=WS, wsb=BIG)
    a.update(kw)
    return lib.sbl_embed_backward(a["ids"], a["out"], a["ot"], a["m"], a["v"], a["k"], a["scale"], a["table"], a["tt"],
                                  a["add"], a["ws"], a["wsb"], None)


@needs_no_gpu
@pytest.mark.parametrize("call", [_embed, _embed_bwd])
@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), SHAPE), (dict(m=(1 << 22) + 1), SHAPE), (dict(k=0), SHAPE), (dict(k=131073), SHAPE), (dict(v=0), SHAPE),
    (dict(v=(1 << 24) + 1), SHAPE), (dict(v=1 << 24, k=1025), SHAPE), (dict(m=1 << 22, k=4097), SHAPE),
    (dict(tt=3), UNSUPPORTED), (dict(tt=1, ot=0), UNSUPPORTED), (dict(tt=0, ot=1), UNSUPPORTED), (dict(ot=-1), UNSUPPORTED),
    (dict(ids=None), NULL), (dict(table=None), NULL), (dict(out=None), NULL),
    (dict(ids=A + 4), ALIGN), (dict(table=C + 8), ALIGN), (dict(out=B + 2), ALIGN),
])
def test_refusals_of_both_embedding_calls(lib, call, kw, status):
    assert call(lib, **kw) == status


@needs_no_gpu
def test_refusals_of_the_embedding(lib):
    assert _embed(lib, out=B + 64) == SHAPE and _embed(lib, out=A) == SHAPE
    assert _embed(lib, m=0, ids=None, out=None) == OK
    assert _embed_bwd(lib, table=B) == SHAPE and _embed_bwd(lib, table=A) == SHAPE and _embed_bwd(lib, table=WS) == SHAPE
    assert _embed_bwd(lib, ws=B) == SHAPE and _embed_bwd(lib, ws=None) == WORKSPACE and _embed_bwd(lib, wsb=64) == WORKSPACE
    assert _embed_bwd(lib, ws=WS + 16) == ALIGN
    assert _embed_bwd(lib, m=0, add=1, ids=None, out=None, table=None, ws=None) == OK
    assert _embed_bwd(lib, m=0, table=None) == NULL


def _adam(lib, items=None, count=None, **kw):
    from sparse_linear_layers_absmean_amd import sbl
    a = dict(lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, step=1, schedule=None)
    top = {k: kw.pop(k) for k in list(kw) if k in a}
    a.update(top)
    if items is None:
        items = [kw]
    arr = (sbl.AdamWItem * len(items))()
    for i, it in enumerate(items):
        d = dict(w=A, w_low=B, g=C, m=D, v=E, m_scale=F, v_scale=G, n=1000, w_dtype=0, g_dtype=2, state_bits=32,
                 lr_scale=1.0, weight_decay=0.0)
        d.update(it)
        arr[i] = sbl.AdamWItem(**d)
    return lib.sbl_adamw_batch(arr, len(items) if count is None else count, a["lr"], a["b1"], a["b2"], a["eps"], a["step"],
                               a["schedule"], None)


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(b1=1.0), SHAPE), (dict(b1=-0.1), SHAPE), (dict(b2=1.0), SHAPE), (dict(b2=NAN), SHAPE), (dict(eps=0.0), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=1e-60), SHAPE), (dict(eps=INF), SHAPE), (dict(lr=NAN), SHAPE), (dict(lr=1e300), SHAPE),
    (dict(step=0), SHAPE), (dict(count=0), SHAPE), (dict(count=65537), SHAPE),
    (dict(n=-1), SHAPE), (dict(n=(1 << 34) + 1), SHAPE), (dict(lr_scale=NAN), SHAPE), (dict(weight_decay=INF), SHAPE),
    (dict(w_dtype=3), UNSUPPORTED), (dict(g_dtype=-1), UNSUPPORTED), (dict(state_bits=16), UNSUPPORTED),
    (dict(w_dtype=1), UNSUPPORTED), (dict(w_dtype=2), UNSUPPORTED),        # low bits are for BF16
    (dict(w=None), NULL), (dict(g=None), NULL), (dict(m=None), NULL), (dict(v=None), NULL),
    (dict(state_bits=8, m_scale=None), NULL), (dict(state_bits=8, v_scale=None), NULL),
    (dict(w=A + 1), ALIGN), (dict(w_low=B + 1), ALIGN), (dict(g=C + 2), ALIGN), (dict(m=D + 2), ALIGN), (dict(v=E + 2), ALIGN),
    (dict(state_bits=8, m=D + 4), ALIGN), (dict(state_bits=8, v=E + 4), ALIGN), (dict(state_bits=8, m_scale=F + 2), ALIGN),
    (dict(schedule=I + 2), ALIGN),
    (dict(w_low=A + 1998), SHAPE), (dict(m=E), SHAPE), (dict(v=D + 3996), SHAPE), (dict(g=A + 1996), SHAPE),
    (dict(g=D + 4), SHAPE), (dict(state_bits=8, m_scale=D), SHAPE), (dict(state_bits=8, v_scale=F + 12), SHAPE),
    (dict(schedule=D), SHAPE), (dict(schedule=A + 1984), SHAPE), (dict(n=0, w=None), OK),
])
def test_refusals_of_adamw(lib, kw, status):
    assert _adam(lib, **kw) == status


@needs_no_gpu
def test_refusals_across_the_tensors(lib):
    far = dict(w=A + GB, w_low=B + GB, g=C + GB, m=D + GB, v=E + GB, n=0)
    assert _adam(lib, items=[dict(n=0), far]) == OK
    assert _adam(lib, items=[{}, dict(far, n=10, w=None)]) == NULL
    assert _adam(lib, items=[{}, {}]) == SHAPE                             # the same tensor twice
    for name, at in [("w", A), ("w", D + 2000), ("m", E), ("g", E), ("w_low", A + 100), ("v", C)]:
        assert _adam(lib, items=[{}, dict(far, n=10, **{name: at})]) == SHAPE, (name, at)
    # a long buffer over several short ones, found whatever lies between
    many = [dict(n=4, **{k: at + 64 * i for k, at in dict(w=A, w_low=B, g=C, m=D, v=E).items()}) for i in range(100)]
    assert _adam(lib, items=many + [dict(far, n=2000, m=D - 4000)]) == SHAPE
    from sparse_linear_layers_absmean_amd import sbl
    assert sbl.load().sbl_adamw_batch(None, 1, 1e-3, 0.9, 0.999, 1e-8, 1, None, None) == NULL


def test_workspace_bytes(lib):
    norm, embed = lib.sbl_norm_workspace_bytes, lib.sbl_embed_workspace_bytes
    assert norm(-1, 64) == -1 and norm(8, 0) == -1 and norm(1 << 22, 8192) == -1 and norm(0, 64) == 0
    assert embed(8, 0, 64, 0) == -1 and embed(8, 100, 64, 3) == -1 and embed(8, 1 << 24, 2048, 0) == -1
    for m, k in [(1, 1), (777, 1541), (8192, 5120), (1 << 22, 4096), (4096, 28672), (300, 131072)]:
        # two column sums of at most 4096 shares of the rows; long rows: two means each
        assert 8 * k <= norm(m, k) <= 8 * k * min(m, 4096) + 8 * m + 256
    for m, v, k in [(1, 1, 1), (777, 50257, 1541), (65536, 32000, 3200), (1 << 22, 128256, 4096)]:
        # the order (ids, tokens, where each id begins) and two fp32 rows for each of at most 8192 segments
        assert 4 * (v + 1) + 8 * m <= embed(m, v, k, 0) <= 4 * (v + 1) + 8 * m + 8 * k * min(m, 8192) + 4 * 256


def test_the_binding_refuses(lib):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    x = torch.zeros(2, 64)
    for call in (lambda: sbl.norm(x), lambda: sbl.norm_quant(x), lambda: sbl.embed(torch.zeros(2, dtype=torch.int64), x),
                 lambda: sbl.AdamWItems([dict(w=x, g=x, m=x, v=x)])):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            call()
    with pytest.raises(TypeError):
        sbl.norm([1.0])
    with pytest.raises(TypeError):
        sbl.norm(x.bfloat16(), dtype=torch.float16)
    with pytest.raises(ValueError):
        sbl.norm(x[0])
    with pytest.raises(ValueError):
        sbl.AdamWItems([])
    with pytest.raises(ValueError):
        sbl.adamw_state(x, bits=16)
    with pytest.raises(ValueError):
        sbl.new_norm_workspace(-1, 64)
    with pytest.raises(ValueError):
        sbl.new_embed_workspace(1, 0, 64)


def test_masters_split_and_join():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    from oracle import step_oracle as S
    w = torch.randn(1000, generator=torch.Generator().manual_seed(1))
    high, low = sbl.split_master(w)
    want = S.split_master(w.numpy())
    assert (high.view(torch.int16).numpy().view("uint16") == want[0]).all() and (low.numpy() == want[1]).all()
    assert torch.equal(sbl.join_master(high, low), w)
    s = sbl.adamw_schedule(1e-3, 0.9, 0.999, 7, 0.5)
    want = S.schedule(1e-3, 0.9, 0.999, 7, 0.5)
    assert s.tolist() == [float(want[k]) for k in ("lr", "bias1", "bias2", "factor", "seed")]
