"""Corners of the norm and the embedding that lie between other tests' sizes: rows shorter than a vector in many rows, and
batches without a single id that counts."""

import numpy as np
import pytest

from gpu_util import say
from test_gpu_step import PAIRS, test_norm_backward_matches_oracle as backward, test_norm_matches_oracle as forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tx,ty", PAIRS)
@pytest.mark.parametrize("t,k", [(1500, 1), (5000, 2), (5000, 3), (70000, 3), (5000, 7)])
def test_norm_of_many_short_rows(t, k, tx, ty):
    forward(t, k, tx, ty)
    backward(t, k, tx, ty)


@pytest.mark.parametrize("t", [1, 1024, 1025, 5000])
def test_embedding_backward_without_an_id_that_counts(t):
    """Padding alone, ids past the table alone, both: zeros where written, nothing where added."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v = 3000
    for k in (5, 72, 520):
        say(f"embed_backward of no id t={t} k={k}")
        dout = torch.full((t, k), float("nan"), dtype=torch.bfloat16, device="cuda")
        for low, high in ((-5, 0), (v, v + 5), (1 << 40, (1 << 40) + v)):
            ids = torch.from_numpy(np.random.default_rng([105, t]).integers(low, high, t)).cuda()
            d = torch.full((v, k), float("nan"), dtype=torch.bfloat16, device="cuda")
            ws = torch.full((sbl.sbl_embed_workspace_bytes(t, v, k),), 255, dtype=torch.uint8, device="cuda")
            sbl.sbl_embed_backward(ids, dout, d, ws)
            assert not d.any() and not torch.isnan(d).any()
            old = torch.randn((v, k), device="cuda").bfloat16()
            kept = old.clone()
            sbl.sbl_embed_backward(ids, dout, old, ws, add=True)
            assert torch.equal(old, kept)
            rows = sbl.embed(ids, kept)
            assert torch.isnan(rows).all() if low > 0 else not rows.any()


def test_sorting_gradient_replays_from_a_graph():
    """More tokens than one launch takes, captured: every replay, with other ids and work between, is the eager result."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    t, v, k = 5000, 2000, 264
    g = torch.Generator("cuda").manual_seed(6)
    ids = torch.zeros(t, dtype=torch.int64, device="cuda")
    dout = torch.randn((t, k), device="cuda", generator=g).bfloat16()
    d, ws = torch.empty((v, k), dtype=torch.bfloat16, device="cuda"), sbl.new_embed_workspace(t, v, k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sbl.sbl_embed_backward(ids, dout, d, ws)
    for i in range(4):
        ids.copy_((torch.rand(t, device="cuda", generator=g) ** (1 + i) * (v + 50)).long() - 10)
        graph.replay()
        got = d.clone()
        torch.randn(500, 500, device="cuda").sum().item()
        assert torch.equal(got, sbl.embed_backward(ids, dout, v))
