"""CPU checks of the binding's own steps around the norm, the embedding and AdamW."""

import numpy as np
import pytest


def test_masters_that_are_nan_stay_nan():
    """Whatever bits a NaN has: both halves and the joined weight; infinities and the largest numbers join as they were."""
    import torch
    from oracle import step_oracle as S
    from sparse_linear_layers_absmean_amd import sbl
    bits = np.array([0x7FFFFFFF, 0xFFFFFFFF, 0x7FFFE000, 0xFFFFE000, 0x7FFF8000, 0x7FFF7FFF, 0x7FC00000, 0x7F800001, 0xFF800001,
                     0x7F800000, 0xFF800000, 0x7F7FFFFF, 0xFF7FFFFF, 0x7F7F8000, 0, 0x80000000, 1, 0x80000001], np.uint32)
    w = bits.view(np.float32)
    high, low = sbl.split_master(torch.from_numpy(w.copy()))
    assert high.dtype == torch.bfloat16 and low.dtype == torch.int16
    nan = np.isnan(w)
    assert torch.isnan(high).numpy()[nan].all() and not torch.isnan(high).numpy()[~nan].any()
    want = S.split_master(w)
    assert np.array_equal(high.view(torch.int16).numpy().view(np.uint16), want[0]) and np.array_equal(low.numpy(), want[1])
    back = sbl.join_master(high, low).numpy()
    assert np.isnan(back[nan]).all() and np.array_equal(back[~nan].view(np.uint32), bits[~nan])
    assert np.array_equal(S.join_master(*want)[~nan].view(np.uint32), bits[~nan])


def test_arguments_that_are_no_tensors_or_of_another_type():
    """Refused with the binding's own errors, before a GPU is asked for."""
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    x, ids = torch.zeros(2, 64), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: sbl.split_master(x.bfloat16()), lambda: sbl.split_master(x.double()), lambda: sbl.split_master([1.0]),
                 lambda: sbl.join_master(x, ids.to(torch.int16)), lambda: sbl.join_master(x.bfloat16(), x.to(torch.int32)),
                 lambda: sbl.join_master(None, x.to(torch.int16)),
                 lambda: sbl.embed([0, 1], x), lambda: sbl.embed(ids, [[0.0]]), lambda: sbl.embed_backward([0, 1], x, 4),
                 lambda: sbl.embed_backward(ids, [[0.0]], 4), lambda: sbl.embed_backward(ids, x, 4, add_to=[[0.0]]),
                 lambda: sbl.new_embed_workspace(2, 4, 64, torch.float64), lambda: sbl.sbl_embed_workspace_bytes(2, 4, 64, "bf16"),
                 lambda: sbl.norm_backward(x, [[0.0]], x, x), lambda: sbl.adamw_state([1.0]),
                 lambda: sbl.AdamWItems([dict(w=[1.0], g=x, m=x, v=x)]), lambda: sbl.AdamWItems([dict(w=x, g=x, m=None, v=x)])):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        sbl.join_master(x.bfloat16(), torch.zeros(2, 63, dtype=torch.int16))
    for missing in ("w", "g", "m", "v"):
        with pytest.raises(ValueError, match=missing):
            sbl.AdamWItems([{n: x for n in ("w", "g", "m", "v") if n != missing}])
    for step in (0, -1):
        with pytest.raises(ValueError):
            sbl.adamw_schedule(1e-3, 0.9, 0.999, step)
