"""Attention over the 4-bit cache at the limits of its other arguments: scales and rows of q that are
very small together, and sequences with more rows than the call computes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import DEV, say, sync
from test_gpu_attn import ATTN, Case

import block_quantized_wire_amd as bq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("new", [None, (4, 2), (70, 3)])
def test_scales_and_rows_of_q_that_are_very_small(kind, new):
    """Scores that are about 0 whatever their factors: every row is the mean of the values it sees."""
    for scale, size in ((2.0 ** -70, -95), (-2.0 ** -90, -110), (2.0 ** -126, 0), (2.0 ** -140, -60), (2.0 ** -149, 4)):
        say(f"attn small scale {kind} new={new} {scale} 2^{size}")
        c = Case([3], (150, 40), new, 4, 2, 128, 64, 16, kind)
        if kind == "f16":
            size = max(size, -20)
        c.q = (c.q.double() * 2.0 ** size).to(c.q.dtype)
        c.check(scale=scale)
        c.check(scale=scale, window=33)
