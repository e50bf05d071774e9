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
