"""The closer bounds notice what they are there for: weights times scales, and values, that are rounded once
to binary16."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attn_tight
import kv_ref as ref


class HostCase:
    def __init__(self, seed, lens, new, heads, kv_heads, dim, group, page, kind, q_size):
        rng = np.random.default_rng(seed)
        self.pool = ref.Pool(-(-lens[0] // page), kv_heads, page, dim, group, kind).random(rng)
        self.table = rng.permutation(self.pool.pages)[None]
        self.lens = lens
        rows = 1 if new is None else new[0]
        self.q = torch.from_numpy(rng.normal(0, q_size, (rows, heads, dim)).astype(np.float32)).half()


@pytest.mark.parametrize("dim,group,n", [(64, 32, 200), (128, 64, 200), (256, 128, 200), (128, 128, 33)])
def test_a_planted_rounding_is_noticed(dim, group, n):
    c = attn_tight.case(HostCase, dim, group, n)
    good, e = attn_tight.attend(c.pool, c.q, c.table, c.lens, dim ** -0.5)
    rounded = attn_tight.binary16(good)
    assert (np.abs(rounded - good) <= e).all()
    bad, _ = attn_tight.attend(c.pool, c.q, c.table, c.lens, dim ** -0.5, held=attn_tight.binary16)
    assert (np.abs(attn_tight.binary16(bad) - good) > e).any()
    # the wider bound of the many-row kernel does not
    y, _, ey, _ = ref.attend(c.pool, c.q, c.table, c.lens, None, True, 0, dim ** -0.5, "f16")
    assert np.abs(y - good).max() < 1e-12 and (np.abs(bad - y) <= ey).all()


@pytest.mark.parametrize("dim,group,n", [(64, 32, 200), (128, 64, 33), (256, 128, 200)])
def test_a_planted_rounding_of_values_is_noticed(dim, group, n):
    c = attn_tight.case_rows(HostCase, dim, group, n)
    good, e = attn_tight.attend_rows(c.pool, c.q, c.table[0], n, dim ** -0.5)
    y = ref.attend(c.pool, c.q, c.table, c.lens, np.array([0, 40]), False, 0, dim ** -0.5, "f16")[0]
    assert np.abs(y - good).max() < 1e-12
    assert (np.abs(attn_tight.binary16(good) - good) <= e).all()
    bad, _ = attn_tight.attend_rows(c.pool, c.q, c.table[0], n, dim ** -0.5, held=attn_tight.binary16)
    assert (np.abs(attn_tight.binary16(bad) - good) > e).any()
