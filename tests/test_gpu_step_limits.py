"""The norm, the embedding and AdamW at sizes whose offsets pass 32 bits, and
outputs of more than one launch, against torch's own operations on the GPU
or the oracle at both ends."""

import numpy as np
import pytest

from gpu_util import say, to_np
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    import torch
    yield
    torch.cuda.empty_cache()


def _ends(n, count):
    return np.concatenate([np.arange(count), np.arange(n - count, n)])


def test_norm_of_more_than_2_32_values():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    t, k = 1100000, 4096
    say(f"norm t={t} k={k}")
    x = torch.empty((t, k), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    at = _ends(t, 3)
    rows = torch.from_numpy(at).cuda()
    xv = to_np(x[rows].double())
    xq, gamma, y, mean, rstd = sbl.norm_quant(x)
    ry, _, rr = S.norm_forward(xv, None, None, 1e-5)
    dm, dr = S.norm_slack(xv, 1e-5)
    assert np.abs(to_np(rstd[rows]) / rr - 1).max() <= 2 * S.U32
    # one rounding to BF16 of a value that fp64 sums in another order move by an fp32 step at most
    assert np.abs(to_np(y[rows].double()) - ry).max() <= (S.HALF["bfloat16"] + 4 * S.U32) * np.abs(ry).max()
    assert np.array_equal(to_np(gamma[rows]) > 0, np.ones(6, bool)) and int(xq[rows].abs().max()) == 127
    dx, dw, _ = sbl.norm_backward(y, x, mean, rstd)
    (rx, _, _), (ex, _, _) = S.norm_backward(to_np(y[rows].double()), xv, to_np(mean[rows]), to_np(rstd[rows]), None)
    got = to_np(dx[rows].double())
    assert (np.abs(got - rx) <= ex + S.HALF["bfloat16"] * (np.abs(rx) + ex)).all()
    # sum_t dy xh with dy = y = xh rounded: near t, each of its terms known to 2^-8
    assert np.abs(to_np(dw) / t - 1).max() < 2.0 ** -8 + 5 * np.sqrt(2.0 / t)


def test_embedding_past_32_bits():
    """A table and an output of more than 2^32 values: several launches of the lookup, rows at the table's end."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v, k, t = 1100000, 4097, 1060000
    say(f"embed v={v} k={k} t={t}")
    g = torch.Generator("cuda").manual_seed(2)
    table = torch.empty((v, k), dtype=torch.float16, device="cuda").normal_(generator=g)
    ids = torch.randint(0, v, (t,), generator=g, device="cuda")
    ids[-5:], ids[:5] = v - 1, -1
    out = sbl.embed(ids, table)
    assert not out[:5].any()
    for a in range(5, t, 100000):
        b = min(t, a + 100000)
        assert torch.equal(out[a:b], table[ids[a:b]])
    del out
    dout = torch.empty((t, k), dtype=torch.float16, device="cuda").normal_(generator=g)
    d = sbl.embed_backward(ids, dout, v, add_to=table.clone())
    count = torch.bincount(ids[ids >= 0], minlength=v)
    # an id of one token: the sum of two numbers, rounded once
    once = (count[ids] == 1).nonzero()[:, 0]
    once = once[(once > 5)]
    once = torch.cat([once[:2000], once[-2000:]])
    want = (table[ids[once]].float() + dout[once].float()).half()
    assert torch.equal(d[ids[once]], want)
    none = (count == 0).nonzero()[:, 0]
    none = torch.cat([none[:2000], none[-2000:]])
    assert torch.equal(d[none], table[none])
    last = table[v - 1].double() + dout[(ids == v - 1).nonzero()[:, 0]].double().sum(0)
    size = table[v - 1].double().abs() + dout[(ids == v - 1).nonzero()[:, 0]].double().abs().sum(0)
    assert ((d[v - 1].double() - last).abs() <= 2.0 ** -11 * last.abs() + 16 * 2.0 ** -24 * size + 2.0 ** -25).all()


def test_embedding_gradient_of_the_most_tokens():
    """2^22 tokens of few ids: long runs over many segments, ids read again while sorting."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    t, v, k = 1 << 22, 37, 8
    g = torch.Generator("cuda").manual_seed(3)
    ids = torch.randint(-1, v + 1, (t,), generator=g, device="cuda")
    dout = torch.randint(-2, 3, (t, k), generator=g, device="cuda").float()     # sums of whole numbers: exact
    want = torch.zeros(v, k, dtype=torch.float64, device="cuda")
    here = (ids >= 0) & (ids < v)
    want.index_add_(0, ids[here], dout[here].double())
    assert torch.equal(sbl.embed_backward(ids, dout, v).double(), want)
    with pytest.raises(sbl.SblError):
        sbl.embed(torch.cat([ids, ids[:1]]), torch.zeros(v, k, device="cuda"))


def test_embedding_of_the_most_ids():
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v, k, t = 1 << 24, 8, 3000
    g = torch.Generator("cuda").manual_seed(4)
    ids = torch.randint(0, v, (t,), generator=g, device="cuda")
    ids[:4] = torch.tensor([0, v - 1, v, v - 1], device="cuda")
    dout = torch.randint(-4, 5, (t, k), generator=g, device="cuda").bfloat16()
    d = sbl.embed_backward(ids, dout, v)
    want = torch.zeros(v, k, device="cuda")
    want.index_add_(0, ids[ids < v], dout[ids < v].float())
    assert torch.equal(d.float(), want)


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_of_more_than_2_32_values(bits):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    n = (1 << 32) + 1000
    say(f"adamw n={n} bits={bits}")
    at = _ends(n, 1000)
    rng = np.random.default_rng(5)
    values = rng.standard_normal(2000).astype(np.float32), (1e-3 * rng.standard_normal(2000)).astype(np.float32)
    w, grad = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    place = torch.from_numpy(at).cuda()
    for t, x in zip((w, grad), values):
        t[place] = torch.from_numpy(x).bfloat16().cuda()
    e = dict(w=w, g=grad, **sbl.adamw_state(w, bits))
    before = [to_np(t[place].float()) for t in (w, grad)]
    sbl.sbl_adamw_batch([e], 1e-2, 0.9, 0.99, 1e-8, 4)
    torch.cuda.synchronize()
    s = S.schedule(1e-2, 0.9, 0.99, 4)
    # the first 1000 values are whole blocks and a piece; the last begin 1000 before the end: blocks from 2^32 on
    for part in (slice(0, 768), slice(1000, 2000)):
        size = part.stop - part.start
        args = dict(m_scale=np.zeros(-(-size // 256), np.float32), v_scale=np.zeros(-(-size // 256), np.float32)) if bits == 8 else {}
        zero = np.zeros(size, np.uint8 if bits == 8 else np.float32)
        got = S.adamw(before[0][part], before[1][part], zero, zero, s, 0.9, 0.99, 1e-8, **args)
        assert np.array_equal(to_np(w[place[part]].float()), torch.from_numpy(got[0]).bfloat16().float().numpy())
        if bits == 32:
            assert np.array_equal(to_np(e["m"][place[part]]), got[1]) and np.array_equal(to_np(e["v"][place[part]]), got[2])
        else:
            first = int(at[part.start]) // 256
            assert np.array_equal(to_np(e["m_scale"][first:first + got[3].size]), got[3])
            assert np.array_equal(to_np(e["m"].view(torch.uint8)[place[part]]), got[1])
    assert not w[n // 2 - 10000:n // 2 + 10000].any()
