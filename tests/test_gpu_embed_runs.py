"""The embedding's gradient of more tokens than one launch takes (1024): runs of
one id that end at, just before and just after the borders of the segments
that the sorted tokens are summed in (8 to 128 tokens, by the sizes)."""

import numpy as np
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

# (tokens at least, width): segments of 8, 16, 32 and 64 tokens; of 8 with one chunk of columns; of 64 and 128
SIZES = [(1025, 8192), (4500, 8192), (9000, 8192), (17000, 8192), (3000, 72), (2000, 5), (262100, 8), (270000, 8)]


def _check(counts, k, rng):
    """Whole numbers, so that every sum is exact in fp32 whatever its order."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    v, t = len(counts), int(np.sum(counts))
    ids = np.repeat(np.arange(v), counts)
    rng.shuffle(ids)
    ids = torch.from_numpy(ids).cuda()
    dout = torch.randint(-8, 9, (t, k), device="cuda", generator=torch.Generator("cuda").manual_seed(t)).bfloat16()
    total = torch.zeros((v, k), device="cuda").index_add_(0, ids, dout.float())
    d = sbl.embed_backward(ids, dout, v, scale=0.5, dtype=torch.float32)
    assert torch.equal(d, 0.5 * total)
    old = torch.randint(-8, 9, (v, k), device="cuda").float()
    assert torch.equal(sbl.embed_backward(ids, dout, v, scale=0.5, add_to=old.clone()), old + 0.5 * total)


@pytest.mark.parametrize("t,k", SIZES)
def test_runs_around_the_segments_borders(t, k):
    """Up to 256 ids the order is the ids' own, so the counts alone say where each run lies."""
    rng = np.random.default_rng([94, t, k])
    edges = [s * m + d for s in (8, 16, 32, 64, 128) for m in (1, 2, 3) for d in (-1, 0, 1)]
    for seed in range(3):
        counts = []
        while sum(counts) < t and len(counts) < 255:
            counts += [int(rng.choice(edges)), int(rng.integers(0, 10))]
        counts.append(max(0, t - sum(counts)))             # the last id: all that is left
        say(f"runs t={sum(counts)} k={k} seed={seed}")
        _check(counts, k, rng)


@pytest.mark.parametrize("before", [0, 1, 7, 8, 63, 64])
@pytest.mark.parametrize("run", [1025, 1032, 1087, 1088, 1089, 2048, 4096, 4097])
def test_one_long_run(run, before):
    """One id of nearly every token, from its segment's start, its end and between."""
    say(f"long run {run} after {before}")
    rng = np.random.default_rng([95, run, before])
    for k in (72, 5, 4104):
        _check([before, run, 0, 9], k, rng)
