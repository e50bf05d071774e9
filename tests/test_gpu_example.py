"""The example that trains a Sparse-BitLinear layer under the head's losses."""

import importlib.util
import math
import os

import pytest

from conftest import ROOT
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [40, 512])
def test_training_example_learns(tokens):
    say(f"examples/train_head tokens={tokens}")
    spec = importlib.util.spec_from_file_location("train_head", os.path.join(ROOT, "examples", "train_head.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=40, tokens=tokens)
    assert len(losses) == 40 and all(math.isfinite(x) for pair in losses for x in pair)
    first, last = losses[0], losses[-1]
    # random weights start near the uniform guess, log 1000 = 6.9; 256 features fit 512 tokens
    assert 6.0 < first[0] < 8.0
    assert last[0] < 0.5 * first[0] and last[1] < 0.5 * first[1]
    assert losses == example.train(steps=40, tokens=tokens)          # step for step the same numbers
