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


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,max_q", [(2, 1, 3), (16, 1, 7), (2, 2, 90)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 20), (False, 0), (False, 9)])
def test_rows_beyond_max_q_keep_the_others_places(kind, heads, kv_heads, max_q, causal, window):
    """A sequence has more rows than max_q: those that are computed stand where they stand."""
    new = (2 * max_q + 5, max_q, 1)
    # the first: short, or long enough that its turns are dealt out
    c = Case([max_q], (300 if heads == kv_heads else 4000, 130, 40), new, heads, kv_heads, 64, 64, 16, kind)
    say(f"attn max_q={max_q} {kind} causal={causal} window={window}")
    whole, whole_lse = c.check(causal=causal, window=window)
    c.max_q = max_q
    got, lse = c.run(causal=causal, window=window)
    sync()
    # the other rows are not written
    assert (got[max_q:new[0]] == 123.0).all() and (lse[max_q:new[0]] == 123.0).all()
    y, l, ey, el = c.want(causal=causal, window=window)
    on = np.r_[0:max_q, new[0]:sum(new)]
    far = np.abs(got.cpu().double().numpy() - y)[on]
    assert (far <= ey[on]).all()
    assert (np.abs(lse.cpu().double().numpy() - l)[on] <= el[on]).all()


def test_many_rows_beyond_max_q_and_the_sequence():
    """Rows in front of a short sequence see nothing, as far in front as they may stand."""
    rows = 3 << 20
    q = torch.ones((rows, 1, 64), dtype=torch.bfloat16, device=DEV)
    c = Case([5], (20,), None, 1, 1, 64, 64, 8, "bf16")
    table, lens, _ = c.arrays()
    starts = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    for window in (0, 10 ** 12):
        out, lse = torch.full_like(q, 9.0), torch.full((rows, 1), 9.0, device=DEV)
        bq.bq_attn_i4(q, c.cache, table, lens, out, starts=starts, max_q=4, max_len=20, window=window, lse=lse)
        sync()
        assert (out[:4] == 0).all() and (lse[:4] == -float("inf")).all() and (out[4:] == 9.0).all()
