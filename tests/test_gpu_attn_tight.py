"""Few rows over a binary16 cache: weights to 2^-21 and values as they are, on the GPU."""
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
