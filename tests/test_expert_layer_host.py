"""The example's judgement of its own distances from plain torch, which smoke() goes by."""
from __future__ import annotations

import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

GOOD = {"one token": 1e-3, "batch": 0.0, "dropped": 2.0 ** -9, "dx": 1e-7, "dweight": 1e-6}


def test_good_distances_pass():
    import expert_layer
    assert expert_layer.close(GOOD)


@pytest.mark.parametrize("which", GOOD)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 0.1])
def test_a_distance_that_is_no_small_number_does_not(which, value):
    import expert_layer
    assert not expert_layer.close({**GOOD, which: value})
