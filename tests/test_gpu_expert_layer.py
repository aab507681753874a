"""The expert layer's calls as a program uses them together: examples/expert_layer.py against the
same layer in plain torch.

The layer rounds to bf16 where plain torch does, so the two differ where a binary32 sum falls on
the other side of a rounding: by at most one bf16 step (2^-8) of single values of the two
intermediate results and the output, well under 2^-8 of the whole.  The training step is binary32
throughout: sums of at most topk * hidden products."""
from __future__ import annotations

import os
import sys

import pytest

from gpu_util import say

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [dict(), dict(tokens=700, experts=5, topk=2, hidden=320, inner=128,
                                                group=32),
                                   dict(tokens=300, experts=3, topk=3, hidden=512, inner=256,
                                        group=128)])
def test_expert_layer(shape):
    import expert_layer
    say(f"expert layer {shape}")
    errors = expert_layer.run(**shape)
    for name in ("one token", "batch", "dropped"):
        assert errors[name] < 2.0 ** -8, errors
    for name in ("dx", "dweight"):
        assert errors[name] < 4 * 1024 * 2.0 ** -24, errors
