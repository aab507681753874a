"""NaN and infinities through the 4-bit codec: a group that holds one is never read back as
ordinary numbers, and the groups beside it are as they are without it."""
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

QUANT = {"bf16": bq.bq_quant_i4, "f16": bq.bq_quant_i4_f16}
DEQUANT = {"bf16": bq.bq_dequant_i4, "f16": bq.bq_dequant_i4_f16}
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_nonfinite_groups(group, kind):
    """Group 1 of every row holds what the row's case names, at every place in turn."""
    say(f"quant_i4 non-finite group={group} {kind}")
    rng = np.random.default_rng([group, 5])
    cases = [[NAN], [-NAN], [INF], [-INF], [INF, -INF], [NAN, INF], [-INF, NAN], [INF, INF]]
    rows, cols = len(cases) * group, 3 * group
    clean = torch.from_numpy(rng.standard_normal((rows, cols))).to(ref.TORCH[kind])
    clean[::7, group:2 * group] = 0.0
    x = clean.clone()
    for r in range(rows):
        for i, v in enumerate(cases[r % len(cases)]):
            x[r, group + (r // len(cases) + 5 * i) % group] = v
    ldc, lds = -(-(cols // 2) // 16) * 16, 4
    c = torch.zeros((rows, ldc), dtype=torch.uint8, device=DEV)
    s = torch.zeros((rows, lds), dtype=ref.TORCH[kind], device=DEV)
    y = torch.empty((rows, cols), dtype=ref.TORCH[kind], device=DEV)
    QUANT[kind](x.to(DEV), c, s, group=group)
    DEQUANT[kind](c, s, y, group=group)
    sync()
    wc, ws = ref.quant(clean, group, kind)
    c, s, y = c.cpu().numpy(), s.cpu(), y.cpu()
    half = group // 2
    for g in (0, 2):                                # the groups beside it
        assert np.array_equal(c[:, g * half:(g + 1) * half], wc[:, g * half:(g + 1) * half])
        assert torch.equal(s[:, g], ws[:, g])
    mid, back = x[:, group:2 * group], y[:, group:2 * group]
    nan = torch.isnan(mid).any(1)
    assert bool(torch.isnan(s[nan, 1]).all()) and bool(torch.isnan(back[nan]).all())
    assert bool((s[~nan, 1] == INF).all())
    held = torch.isinf(mid[~nan])
    assert torch.equal(back[~nan][held], mid[~nan][held])
    assert bool(torch.isnan(back[~nan][~held]).all())
    codes = np.stack((c & 15, c >> 4), -1).reshape(rows, -1)[:, group:2 * group]
    want = np.where(mid.float().numpy() == INF, 15, np.where(mid.float().numpy() == -INF, 1, 8))
    want[nan.numpy()] = 8
    assert np.array_equal(codes, want)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_every_nan_pattern(kind):
    """All NaN bit patterns of the type, one in each group."""
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    x = torch.from_numpy(bits.view(np.int16).copy()).view(ref.TORCH[kind])
    nans = x[torch.isnan(x)]
    v = torch.ones((nans.numel(), 32), dtype=ref.TORCH[kind])
    v.view(torch.int16)[:, 9] = nans.view(torch.int16)
    c = torch.zeros((nans.numel(), 16), dtype=torch.uint8, device=DEV)
    s = torch.zeros((nans.numel(), 4), dtype=ref.TORCH[kind], device=DEV)
    QUANT[kind](v.to(DEV), c, s, group=32)
    sync()
    assert nans.numel() > 200 and bool(torch.isnan(s[:, 0]).all()) and bool((c == 0x88).all())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(4, 40, 384), (16, 4100, 256), (24, 40, 640), (40, 70, 256),
                                   (300, 700, 352), (300, 7000, 128), (4100, 3000, 256)])
def test_products_keep_them_in_their_row_and_column(m, n, k, kind):
    """Non-finite rows of x and non-finite scales: nothing ordinary in their rows and columns, the
    same bits everywhere else."""
    say(f"mm_i4 non-finite m={m} n={n} k={k} {kind}")
    rng = np.random.default_rng([m, n, k])
    codes, scale, zero = ref.matrix(rng, n, k, 32, kind, True)
    x = torch.from_numpy(rng.standard_normal((m, k))).to(ref.TORCH[kind])
    mm = bq.bq_mm_i4 if kind == "bf16" else bq.bq_mm_i4_f16

    def product():
        y = torch.empty((m, n), dtype=ref.TORCH[kind], device=DEV)
        mm(x.to(DEV), codes.to(DEV), scale.to(DEV), y, zero=zero.to(DEV), group=32)
        sync()
        return y.cpu()

    want = product()
    assert bool(torch.isfinite(want).all())
    rows, cols = [0, 2, m - 1], [1, n // 2, n - 1]
    for i, v in enumerate((NAN, INF, -INF)):
        x[rows[i], [3, k // 2, k - 1][i]] = v
        scale[cols[i], [0, k // 64, k // 32 - 1][i]] = v
    got = product()
    assert not bool(torch.isfinite(got[rows]).any()) and not bool(torch.isfinite(got[:, cols]).any())
    keep = np.ix_([r for r in range(m) if r not in rows], [c for c in range(n) if c not in cols])
    assert torch.equal(got[keep], want[keep])
