"""The cache's calls as a server uses them together: examples/cached_attention.py, prompts in chunks
and decode steps, eager and replayed, against plain torch on what the cache holds.

A row is rounded to bf16 once, by at most 2^-8 of a value; binary32 sums and weights held to 2^-12
add less than a tenth of that to the whole."""
from __future__ import annotations

import os
import sys

import pytest

from gpu_util import say

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [dict(), dict(seqs=1, prompt=40, heads=4, kv_heads=4, dim=64, group=32, page=8,
                                                hidden=256),
                                   dict(seqs=3, prompt=700, heads=8, kv_heads=1, dim=256, group=128, page=24,
                                        hidden=384, steps=5)])
def test_cached_attention(shape):
    import cached_attention
    say(f"cached attention {shape}")
    errors = cached_attention.run(**shape)
    assert set(errors) == {"first chunk", "second chunk", "steps", "graph"}
    assert cached_attention.close(errors), errors
