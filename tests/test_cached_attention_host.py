"""examples/cached_attention.py without a GPU: what it takes as near enough, how its cache hands out
slots, and how it reads the cache's bytes."""
from __future__ import annotations

import os
import sys

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import kv_ref  # noqa: E402


def test_what_is_near_enough():
    import cached_attention
    assert cached_attention.close({"steps": 1e-3, "graph": 2e-3})
    for bad in (float("nan"), float("inf"), 0.1):
        assert not cached_attention.close({"steps": 1e-3, "graph": bad})


def test_slots_go_on_in_a_sequence_and_take_pages_when_needed():
    import cached_attention
    cache = cached_attention.Cache(4, 2, 1, 8, 64, 32, torch.bfloat16, "cpu")
    assert cache.slots([3, 8]) == [0, 1, 2, 8, 9, 10, 11, 12, 13, 14, 15]
    assert cache.slots([6, 1]) == [3, 4, 5, 6, 7, 16, 24]
    assert cache.table == [[0, 2], [1, 3]] and cache.lens == [9, 9]
