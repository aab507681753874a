"""The expert products on orders that no sort wrote, for every kernel that reads one: what the
arrays name out of range is left out, and nothing outside the arrays is touched."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import i4_moe_ref as ref
from gpu_util import DEV, say, sync

from block_quantized_wire_amd import build as _build

if _build.stale():
    _build.build()
import block_quantized_wire_amd as bq  # noqa: E402

pytestmark = pytest.mark.gpu

MOE = {"bf16": bq.bq_moe_mm_i4, "f16": bq.bq_moe_mm_i4_f16}
MIN, MAX = -(1 << 31), (1 << 31) - 1

# rows of y, rows of W: few rows an expert; tiles of 64 x 128, 64 x 256 and 128 x 256
SIZES = [(40, 96), (300, 96), (300, 12000), (700, 12000)]


def product(x, mats, off, src, topk, y, kind, zeros=True):
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    c, s, z = (torch.stack([m[i] for m in mats]) if mats[0][i] is not None else None for i in range(3))
    MOE[kind](d(x), d(torch.tensor(off, dtype=torch.int32)), d(c), d(s), y, zero=d(z), group=64,
              src=d(src), topk=topk)
    sync()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("rows,n", SIZES)
def test_offsets_out_of_range(rows, n, kind):
    """Neighbouring offsets whose difference wraps to a positive count, and ends past the rows.
    One expert of the four has rows that are there: its products are right, the rest of y is
    as it was."""
    say(f"moe_mm_i4 offsets out of range: rows={rows} n={n} {kind}")
    rng = np.random.default_rng([rows, n])
    mats = [ref.matrix(rng, n, 128, 64, kind, True, exact=True)] * 4
    x = torch.from_numpy(rng.integers(-3, 4, (rows, 128))).to(ref.TORCH[kind])
    want = ref.rne(ref.product(x, *mats[0], 128, 64, kind)[0], kind)
    for off, lo, hi in (([0x60000000, -0x60000000, 17, MIN, -1], 0, 17),
                        ([1 << 30, MIN, 1 << 30, MIN, rows - 3], 0, rows),
                        ([MAX, MIN, MIN, -1, MIN], 0, 0),
                        ([9, rows - 5, 9, MIN, -64], 9, rows - 5),
                        ([MAX, MAX, MAX, rows - 2, MAX], rows - 2, rows)):
        y = torch.full((rows, n), 5.0, dtype=ref.TORCH[kind], device=DEV)
        product(x, mats, off, None, 1, y, kind)
        got = y.cpu()
        assert torch.equal(got[lo:hi], want[lo:hi]), off
        assert bool((got[:lo] == 5.0).all()) and bool((got[hi:] == 5.0).all()), off


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("rows,n", SIZES)
def test_sources_out_of_range(rows, n, kind):
    """Sources that name no row of x give rows of zeros: those just below 0, which a division
    by topk would bring to row 0, among them."""
    say(f"moe_mm_i4 sources out of range: rows={rows} n={n} {kind}")
    rng = np.random.default_rng([rows, n, 1])
    topk, x_rows = 3, rows // 2
    mats = [ref.matrix(rng, n, 128, 64, kind, True, exact=True)] * 4
    x = torch.from_numpy(rng.integers(1, 4, (x_rows, 128))).to(ref.TORCH[kind])
    src = rng.integers(0, x_rows * topk, rows)
    bad = rng.random(rows) < 0.4
    bad[:6] = True
    src[bad] = rng.choice([-1, -2, -3, -4, MIN, x_rows * topk, MAX], int(bad.sum()))
    src[:5] = [-1, -2, -3, MIN, x_rows * topk]
    cut = rows // 4
    off = [0, cut, 2 * cut, 3 * cut, rows]
    y = torch.full((rows, n), 5.0, dtype=ref.TORCH[kind], device=DEV)
    product(x, mats, off, torch.from_numpy(src.astype(np.int32)), topk, y, kind)
    want = ref.rne(ref.product(x, *mats[0], 128, 64, kind)[0], kind)[np.where(bad, 0, src // topk)]
    want[torch.from_numpy(bad)] = 0
    assert torch.equal(y.cpu(), want)
