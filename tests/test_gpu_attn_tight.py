"""Over a binary16 cache weights to 2^-21 and values to 2^-22 or as they are, for few rows and many; long sums
of bf16 without a bias."""
from __future__ import annotations

import numpy as np
import pytest

import attn_tight
from gpu_util import say, sync
from test_gpu_attn import Case
from test_gpu_kv import WIDTHS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,group", WIDTHS)
@pytest.mark.parametrize("n", [1, 33, 200, 3000])
def test_weights_and_values_of_few_rows_are_not_cut(dim, group, n):
    say(f"attn tight D={dim} G={group} n={n}")
    c = attn_tight.case(Case, dim, group, n)
    got, _ = c.run()
    sync()
    y, e = attn_tight.attend(c.pool, c.q.cpu(), c.table, c.lens, dim ** -0.5)
    far = np.abs(got.cpu().double().numpy() - y)
    assert (far <= e).all(), float((far / e).max())


@pytest.mark.parametrize("dim,group", WIDTHS)
@pytest.mark.parametrize("n", [1, 33, 200, 1500])
def test_weights_and_values_of_many_rows_are_not_cut(dim, group, n):
    say(f"attn tight many rows D={dim} G={group} n={n}")
    c = attn_tight.case_rows(Case, dim, group, n)
    got, _ = c.run(causal=False)
    sync()
    y, e = attn_tight.attend_rows(c.pool, c.q.cpu(), c.table[0], n, dim ** -0.5)
    far = np.abs(got.cpu().double().numpy() - y)
    assert (far <= e).all(), float((far / e).max())


def test_long_bf16_sums_are_not_biased():
    """Many tokens of about the same weight.  A rounding to bf16 is off by at most 2^-8 of a result, to either
    side, so the mean of n of them has a deviation of at most 2^-8 of their size by sqrt(3 n)."""
    for dim, group in ((128, 128), (64, 32)):
        say(f"attn long bf16 sums dim={dim}")
        c = Case([dim], (60000,), None, 16, 1, dim, group, 64, "bf16", q_size=0.1)
        got, _ = c.check()
        y = c.want()[0]
        off = got.cpu().double().numpy() - y
        assert abs(off.mean()) <= 5 * 2.0 ** -8 * np.sqrt((y * y).mean()) / np.sqrt(3 * y.size)
