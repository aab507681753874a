"""Products with 4-bit weights at the ends of the types' range: finite rows of x up to the
largest, whose sums over a group leave binary32 when nothing scales them, and rows of the
smallest subnormals, whose products with the codes do.  Every kernel, dense and by expert."""
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

# rows of x and of W, columns: each kernel for few rows, then the tiles of 64 x 128, 64 x 256 and
# 128 x 256
DENSE = [(1, 40, 384), (6, 40, 256), (16, 4100, 256), (24, 40, 640), (40, 70, 256), (300, 700, 384),
         (300, 7000, 128), (4100, 3000, 256)]


def dev(t):
    return None if t is None else t.to(DEV)


def mm(x, codes, scale, zero, group, kind):
    y = torch.empty((x.shape[0], codes.shape[0]), dtype=ref.TORCH[kind], device=DEV)
    MM[kind](dev(x), dev(codes), dev(scale), y, zero=dev(zero), group=group)
    sync()
    return y.cpu()


def largest(rng, m, k, kind):
    """Rows of the type's largest values: all of one sign, all of the other, mixed signs."""
    top = float(torch.finfo(ref.TORCH[kind]).max)
    x = rng.choice([1.0, 0.996], (m, k)) * top
    x[1::3] *= -1
    x[2::3] *= rng.choice([-1.0, 1.0], x[2::3].shape)
    return torch.from_numpy(x).to(ref.TORCH[kind])


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k", DENSE)
def test_largest_rows(m, n, k, group, zeros, kind):
    """Scales small enough for finite results: k * 15 * scale < 1."""
    say(f"mm_i4 largest rows m={m} n={n} k={k} group={group} {kind} zeros={zeros}")
    rng = np.random.default_rng([m, n, k, group, zeros])
    codes, scale, zero = ref.matrix(rng, n, k, group, kind, zeros)
    scale = (scale.float() * 2.0 ** -11).to(ref.TORCH[kind])      # below 2^-14
    codes[::5] = 0x00
    codes[1::5] = 0xFF
    x = largest(rng, m, k, kind)
    got = mm(x, codes, scale, zero, group, kind)
    want, bound = ref.product(x, codes, scale, zero, k, group, kind)
    off = np.abs(got.double().numpy() - want)
    assert (off <= bound).all(), (np.isfinite(got.float().numpy()).all(), (off / bound).max())


@pytest.mark.parametrize("m,n,k", DENSE)
def test_weights_of_zero_times_large_rows(m, n, k):
    """Every code at its zero point: the weights are 0, whatever x holds; what the sums may leave
    is the bound's."""
    rng = np.random.default_rng([m, n])
    for z in (None, 15):
        codes = torch.full((n, k // 2), 0x88 if z is None else 0xFF, dtype=torch.uint8)
        scale = torch.full((n, -(-k // 128) * 4), 0.5).to(torch.bfloat16)
        zero = None if z is None else torch.full(scale.shape, z, dtype=torch.uint8)
        x = torch.full((m, k), 1e36).to(torch.bfloat16)
        x[0] = largest(rng, 1, k, "bf16")
        got = mm(x, codes, scale, zero, 128, "bf16")
        _, bound = ref.product(x, codes, scale, zero, k, 128, "bf16")
        assert (np.abs(got.double().numpy()) <= bound).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k", DENSE)
def test_smallest_rows(m, n, k, group, zeros):
    """Multiples of the smallest subnormal, brought back to ordinary size by the scales: every
    sum is exact."""
    for kind, small, big in (("bf16", 2.0 ** -133, 2.0 ** 120), ("f16", 2.0 ** -24, 2.0 ** 10)):
        say(f"mm_i4 smallest rows m={m} n={n} k={k} group={group} {kind} zeros={zeros}")
        rng = np.random.default_rng([m, n, k, group, zeros])
        codes, scale, zero = ref.matrix(rng, n, k, group, kind, zeros, exact=True)
        scale = (scale.float() * big).to(ref.TORCH[kind])
        x = torch.from_numpy(rng.integers(-3, 4, (m, k)) * small).to(ref.TORCH[kind])
        got = mm(x, codes, scale, zero, group, kind)
        want, _ = ref.product(x, codes, scale, zero, k, group, kind)
        assert torch.equal(got, ref.rne(want, kind)), kind


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("each,n", [([3, 0, 9], 40), ([12] * 8, 4100), ([40, 0, 90], 300),
                                    ([60, 31, 200], 17000), ([400, 131], 17000)])
def test_largest_rows_by_expert(each, n, kind):
    say(f"moe_mm_i4 largest rows each={each} n={n} {kind}")
    rng = np.random.default_rng([n, len(each)])
    k, group, rows = 256, 64, sum(each)
    mats = [ref.matrix(rng, n, k, group, kind, True) for _ in each]
    mats = [(c, (s.float() * 2.0 ** -11).to(s.dtype), z) for c, s, z in mats]
    off = np.concatenate([[0], np.cumsum(each)]).astype(np.int32)
    x = largest(rng, rows, k, kind)
    y = torch.empty((rows, n), dtype=ref.TORCH[kind], device=DEV)
    stack = [dev(torch.stack([m[i] for m in mats])) for i in range(3)]
    MOE[kind](dev(x), dev(torch.from_numpy(off)), stack[0], stack[1], y, zero=stack[2], group=group)
    sync()
    got = y.cpu().double().numpy()
    for e, (c, s, z) in enumerate(mats):
        want, bound = ref.product(x[off[e]:off[e + 1]], c, s, z, k, group, kind)
        assert (np.abs(got[off[e]:off[e + 1]] - want) <= bound).all(), e
