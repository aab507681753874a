"""Every form of the 4-bit product kernels, dense and by expert, at depths where its loops run
for a while and end inside a stage or a unit, with sums that are exact: the results have to be
the rounded sums bit for bit.  Which form a size takes follows from the launch rules: up to 16
rows of x by 4, 8 or 16 and by the rows of W; more while workgroups of 32 rows of W fit few
rounds; then tiles of 64 x 128, 64 x 256 and 128 x 256.  And strides of every operand of the
expert products, and rows as far apart as the 32-bit offsets of the staged kernel reach."""
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

MM = {"bf16": bq.bq_mm_i4, "f16": bq.bq_mm_i4_f16}
MOE = {"bf16": bq.bq_moe_mm_i4, "f16": bq.bq_moe_mm_i4_f16}
FORMS = pytest.mark.parametrize("group,zeros,kind", [(g, z, k) for g in (32, 64, 128)
                                                     for z in (False, True) for k in ("bf16", "f16")])


def dev(t):
    return None if t is None else t.to(DEV)


def rounded(x, codes, scale, zero, k, group, kind):
    """The rounded products: 64-bit sums on the device, rounded on the way through binary32,
    which holds them (every term is a multiple of 2^-2 below 2^24)."""
    w = torch.from_numpy(ref.dense(codes, scale, zero, k, group)[0]).to(DEV)
    y = x.to(DEV).double() @ w.t()
    assert float(y.abs().max()) < 2 ** 22
    return y.float().to(ref.TORCH[kind])


def whole(rng, m, k, kind):
    return torch.from_numpy(rng.integers(-3, 4, (m, k))).to(ref.TORCH[kind])


def check(m, n, k, group, zeros, kind):
    say(f"mm_i4 m={m} n={n} k={k} group={group} {kind} zeros={zeros}")
    rng = np.random.default_rng([m, n, k, group, zeros])
    codes, scale, zero = ref.matrix(rng, n, k, group, kind, zeros, exact=True)
    x = whole(rng, m, k, kind)
    y = torch.full((m, n), 7.0, dtype=ref.TORCH[kind], device=DEV)
    MM[kind](dev(x), dev(codes), dev(scale), y, zero=dev(zero), group=group)
    sync()
    assert torch.equal(y, rounded(x, codes, scale, zero, k, group, kind))


@FORMS
@pytest.mark.parametrize("n", [40, 4100])
@pytest.mark.parametrize("m", [1, 3, 4, 6, 8, 12, 16])
def test_staged_rows(m, n, group, zeros, kind):
    check(m, n, 2816, group, zeros, kind)                   # eleven whole units
    check(m, n, 2304 + group, group, zeros, kind)           # one group of a tenth


@FORMS
@pytest.mark.parametrize("m,n", [(20, 4000), (32, 8000), (20, 8200), (31, 16400), (48, 4000), (64, 4090),
                                 (50, 8100), (64, 8192)])
def test_rows_through_registers(m, n, group, zeros, kind):
    check(m, n, 2048, group, zeros, kind)
    check(m, n, 2304 + group, group, zeros, kind)


@FORMS
@pytest.mark.parametrize("m,n", [(256, 700), (300, 7000), (4100, 3000)])
def test_tiles_at_depth(m, n, group, zeros, kind):
    check(m, n, 2304 + group, group, zeros, kind)
    check(m, n, 2816 - group, group, zeros, kind)


# ---- by expert -----------------------------------------------------------------------------

EACH = {"few, 64 rows of W": (lambda rng: rng.integers(0, 27, 64), 520),
        "few, 32 rows of W": (lambda rng: rng.integers(0, 20, 8), 520),
        "64 x 128": (lambda rng: np.array([17, 0, 200, 64, 65]), 300),
        "64 x 256": (lambda rng: rng.integers(0, 120, 30), 1300),
        "128 x 256": (lambda rng: rng.integers(0, 400, 20), 1300)}


def experts(name, k, group, zeros, kind, gathered, pad):
    """One call over strided operands: every row of every operand is followed by `pad` units of its
    alignment, every expert's matrix by rows of its own, all of it NaN and 255."""
    say(f"moe_mm_i4 {name} k={k} group={group} {kind} zeros={zeros} gathered={gathered} pad={pad}")
    make, n = EACH[name]
    rng = np.random.default_rng([n, k, group, zeros, gathered, pad])
    each = make(rng)
    e, groups = len(each), k // group
    mats = [ref.matrix(rng, n, k, group, kind, zeros, exact=True) for _ in each]
    off = np.concatenate([[0], np.cumsum(each)]).astype(np.int32)
    rows, topk = int(off[-1]), 3
    x_rows = rows // topk + 1 if gathered else rows
    src = torch.from_numpy(rng.integers(0, x_rows * topk, rows).astype(np.int32)) if gathered else None

    def strided(shape, ld, between, fill, dtype):
        """A tensor of `fill` and a view of `shape` in it, rows ld apart, experts `between` rows more."""
        lead = shape[0] if len(shape) == 3 else 1
        step = (shape[-2] + between) * ld
        buf = torch.full((lead * step,), fill).to(dtype)
        strides = (step, ld, 1) if len(shape) == 3 else (ld, 1)
        return buf.as_strided(shape, strides)

    c = strided((e, n, k // 2), -(-k // 32) * 16 + 16 * pad, 2 * pad, 255, torch.uint8)
    s = strided((e, n, groups), -(-groups // 4) * 4 + 4 * pad, 3 * pad, float("nan"), ref.TORCH[kind])
    z = None
    if zeros:
        z = strided((e, n, groups), -(-groups // 4) * 4 + 8 * pad, pad, 255, torch.uint8)
    for i, (ci, si, zi) in enumerate(mats):
        c[i].copy_(ci[:, : k // 2])
        s[i].copy_(si[:, :groups])
        if zeros:
            z[i].copy_(zi[:, :groups])
    x = strided((x_rows, k), k + 8 * pad, 0, float("nan"), ref.TORCH[kind])
    x.copy_(whole(rng, x_rows, k, kind))

    def on_device(t):
        """The view's whole storage on the device, and the same view of it."""
        if t is None:
            return None
        base = torch.empty(0, dtype=t.dtype).set_(t.untyped_storage())
        return base.to(DEV).as_strided(t.shape, t.stride())

    ybuf = torch.full((rows, n + 5 * pad), 7.0, dtype=ref.TORCH[kind], device=DEV)
    MOE[kind](on_device(x), dev(torch.from_numpy(off)), on_device(c), on_device(s), ybuf[:, :n],
              zero=on_device(z), group=group, src=dev(src), topk=topk)
    sync()
    pick = src.long() // topk if gathered else torch.arange(rows)
    for i in range(e):
        lo, hi = int(off[i]), int(off[i + 1])
        if hi > lo:
            want = rounded(x[pick[lo:hi]], *mats[i], k, group, kind)
            assert torch.equal(ybuf[lo:hi, :n], want), i
    assert bool((ybuf[:, n:] == 7.0).all())


@FORMS
@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("name", EACH)
def test_experts_at_depth(name, gathered, group, zeros, kind):
    experts(name, 2304 + group, group, zeros, kind, gathered, 0)


@FORMS
@pytest.mark.parametrize("name", EACH)
def test_experts_with_strides(name, group, zeros, kind):
    experts(name, 640 + group, group, zeros, kind, True, 1)
    experts(name, 768, group, zeros, kind, False, 3)


# ---- rows far apart --------------------------------------------------------------------------

@pytest.mark.parametrize("m,n", [(4, 40), (8, 4100), (16, 40), (16, 4100)])
@pytest.mark.parametrize("ld", [(1 << 27) - 8, 1 << 27])
def test_rows_of_x_at_the_reach_of_32_bits(m, n, ld):
    """Rows of x up to 2^27 values apart take the staged kernel, whose last row of 16 starts just
    below 2^31 values; the next stride takes the kernel with 64-bit addresses."""
    rng = np.random.default_rng([m, n])
    k = 640
    say(f"mm_i4 m={m} n={n} ldx={ld}")
    codes, scale, zero = ref.matrix(rng, n, k, 64, "bf16", True, exact=True)
    x = whole(rng, m, k, "bf16")
    far = torch.empty((m - 1) * ld + k, dtype=torch.bfloat16, device=DEV).as_strided((m, k), (ld, 1))
    far.copy_(x)
    y = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    bq.bq_mm_i4(far, dev(codes), dev(scale), y, zero=dev(zero), group=64)
    sync()
    assert torch.equal(y, rounded(x, codes, scale, zero, k, 64, "bf16"))


@pytest.mark.parametrize("m,n", [(1, 40), (16, 40), (100, 40)])
@pytest.mark.parametrize("which", ["codes", "scales", "zeros"])
@pytest.mark.parametrize("ld", [(1 << 26) - 16, 1 << 26])
def test_rows_of_weights_at_the_reach_of_32_bits(m, n, which, ld):
    """The same for the three arrays of W, whose rows are addressed 32 at a time."""
    rng = np.random.default_rng([m, n, 1])
    k = 640
    say(f"mm_i4 m={m} n={n} {which} {ld} apart")
    arrays = dict(zip(("codes", "scales", "zeros"), ref.matrix(rng, n, k, 64, "bf16", True, exact=True)))
    x = whole(rng, m, k, "bf16")
    on = {name: dev(t) for name, t in arrays.items()}
    t = arrays[which]
    far = torch.empty((n - 1) * ld + t.shape[1], dtype=t.dtype, device=DEV).as_strided(t.shape, (ld, 1))
    far.copy_(t)
    on[which] = far
    y = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    bq.bq_mm_i4(dev(x), on["codes"], on["scales"], y, zero=on["zeros"], group=64)
    sync()
    assert torch.equal(y, rounded(x, *arrays.values(), k, 64, "bf16"))
