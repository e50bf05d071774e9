"""AdamW: a gradient that is not finite shows in the weight's own BF16 half, whatever bits its NaN has."""

import numpy as np
import pytest

from gpu_util import say, to_np
from oracle import step_oracle as S
from test_gpu_step import ADAM, _tensor

pytestmark = pytest.mark.gpu

# NaNs whose bits past the BF16 half would carry into exponent and sign, and ordinary ones; infinities
BAD = {"float32": ("int32", (0x7FFFFFFF, -1, 0x7FC00000, 0x7FFF8000, -0x8000, 0x7F800000, -0x800000)),
       "bfloat16": ("int16", (0x7FFF, -1, 0x7FC0, 0x7F80, -0x80)),
       "float16": ("int16", (0x7FFF, -1, 0x7E00, 0x7C00, -0x400))}


@pytest.mark.parametrize("low", [True, False])
@pytest.mark.parametrize("gt", list(BAD))
@pytest.mark.parametrize("bits", [32, 8])
def test_weights_spoiled_by_their_gradient_are_nan(bits, gt, low):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    say(f"adamw not finite g={gt} bits={bits} low={low}")
    n = 5000
    e, o, here = _tensor(np.random.default_rng([96, bits]), n, "bfloat16", low, gt, bits)
    view, codes = BAD[gt]
    raw = e["g"].view(getattr(torch, view))
    at = [300 + 512 * i + 7 * i for i in range(len(codes))]      # in blocks of their own
    for i, c in zip(at, codes):
        raw[i] = c
        o["g"][i] = 0.0
    sbl.sbl_adamw_batch([e], 1e-2, **ADAM, step=3)
    torch.cuda.synchronize()
    w = e["w"]
    assert torch.isnan(w[at]).all()
    if low:
        assert torch.isnan(sbl.join_master(w, e["w_low"])[at]).all()
    args = {k: o[k] for k in ("m_scale", "v_scale") if k in o}
    want = S.adamw(o["w"], o["g"], o["m"], o["v"], S.schedule(1e-2, ADAM["beta1"], ADAM["beta2"], 3), ADAM["beta1"],
                   ADAM["beta2"], ADAM["eps"], 1.0, o["weight_decay"], **args)
    # the weight alone is spoiled by this step, in 8 bits too (its block's states are)
    fine = np.ones(n, bool)
    fine[at] = False
    if low:
        high, lo = S.split_master(want[0])
        assert np.array_equal(to_np(w.view(torch.int16)).view(np.uint16)[fine], high[fine])
        assert np.array_equal(to_np(e["w_low"])[fine], lo[fine])
    else:
        nearest = torch.from_numpy(want[0]).bfloat16()
        assert torch.equal(w.cpu()[fine], nearest[fine])
    here.check()
    # from the next step on as well: a NaN stays one
    sbl.sbl_adamw_batch([e], 1e-2, **ADAM, step=4)
    assert torch.isnan(e["w"][at]).all()
