"""The I4 codec and the products with I4 weights on the GPU, against plain forms on the host:
the codec bit for bit, products bit for bit where every sum is exact, and within the bound
that binary32 sums and one rounding allow otherwise."""
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
QUANT = {"bf16": bq.bq_quant_i4, "f16": bq.bq_quant_i4_f16}
DEQUANT = {"bf16": bq.bq_dequant_i4, "f16": bq.bq_dequant_i4_f16}


def dev(t):
    return None if t is None else t.to(DEV)


def rows_of_x(rng, m, k, kind, exact, pad=0):
    """x (m, k) in a buffer whose columns past k hold NaN."""
    x = np.full((m, k + pad), np.nan)
    x[:, :k] = rng.integers(-3, 4, (m, k)) if exact else rng.standard_normal((m, k))
    return torch.from_numpy(x).to(ref.TORCH[kind])


def check_mm(m, n, k, group, kind, zeros, exact=False, pad=False, seed=0):
    say(f"mm_i4 m={m} n={n} k={k} group={group} {kind} zeros={zeros} exact={exact} pad={pad}")
    rng = np.random.default_rng([m, n, k, group, zeros, seed])
    codes, scale, zero = ref.matrix(rng, n, k, group, kind, zeros, 32 * pad, 4 * pad, exact)
    x = rows_of_x(rng, m, k, kind, exact, 8 * pad)
    y = torch.full((m, n + 3 * pad), 7.0, dtype=ref.TORCH[kind], device=DEV)
    MM[kind](dev(x), dev(codes), dev(scale), y, zero=dev(zero), group=group, N=n, K=k)
    sync()
    got = y.cpu()
    want, bound = ref.product(x, codes, scale, zero, k, group, kind)
    if exact:
        assert torch.equal(got[:, :n], ref.rne(want, kind))
    else:
        off = np.abs(got[:, :n].double().numpy() - want)
        assert (off <= bound).all(), (off / bound).max()
    assert bool((got[:, n:] == 7.0).all())      # nothing beyond the row's N columns


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 7, 8, 9, 13, 16, 17, 31, 48, 63, 64, 65, 130])
def test_rows(m, group, kind, zeros):
    check_mm(m, 33, 384, group, kind, zeros, exact=True, pad=True)
    check_mm(m, 40, 1024, group, kind, zeros)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 257, 1001])
@pytest.mark.parametrize("m", [1, 6, 20, 200])
def test_weight_rows(m, n):
    check_mm(m, n, 256, 64, "bf16", True, exact=True)


@pytest.mark.parametrize("group,k", [(32, 32), (32, 64), (32, 96), (32, 128), (32, 160), (32, 992),
                                     (64, 64), (64, 128), (64, 192), (64, 1088), (128, 128),
                                     (128, 256), (128, 1152), (128, 7168), (64, 43008)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1, 10, 70])
def test_depths(m, group, k, kind):
    check_mm(m, 19, k, group, kind, True, exact=k <= 1152, pad=True)
    check_mm(m, 19, k, group, kind, False)


@pytest.mark.parametrize("m,n,k", [(300, 500, 1024), (517, 1001, 640), (129, 300, 4096)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_many_rows(m, n, k, group, kind):
    check_mm(m, n, k, group, kind, True, exact=k <= 1024)
    check_mm(m, n, k, group, kind, False, pad=True)


@pytest.mark.parametrize("m,n", [(4100, 401), (24583, 300), (65, 12300), (20, 49170), (3000, 70),
                                 (20, 4000)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_many_workgroups(m, n, group, kind):
    """Long on one side, with depths that end inside a stage or a unit of scales."""
    check_mm(m, n, {32: 160, 64: 192, 128: 384}[group], group, kind, True, exact=True)
    check_mm(m, n, {32: 32, 64: 320, 128: 128}[group], group, kind, False, exact=True, pad=True)


@pytest.mark.parametrize("m,n", [(1100, 700), (333, 2000), (40, 10001)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_rows_for_one_round_of_workgroups(m, n, group, kind):
    """Two parts of the columns: one or none for the second, an odd unit, ends inside one."""
    for cols in (128, 256, 384, 640, 1152):
        check_mm(m, n, cols, group, kind, cols != 640, exact=True, pad=cols == 384)
    check_mm(m, n, {32: 1056, 64: 1088, 128: 2176}[group], group, kind, True)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("each,n", [([21, 0, 17, 40] * 15, 600), ([201, 0, 260, 129] * 10, 900)])
def test_many_rows_by_expert(each, n, group, kind):
    check_experts(each, n, 384, group, kind, True, False)
    check_experts(each, n, 128, group, kind, False, True)


def test_extremes_of_codes_and_zero_points():
    """Codes 0 and 15 against zero points 0 and 15, scales of 0 and of the type's largest and
    smallest normal numbers, rows of x that are all zero."""
    for kind, big, small in (("bf16", 2.0 ** 120, 2.0 ** -126), ("f16", 1024.0, 2.0 ** -14)):
        n, k, group = 32, 256, 128
        codes = torch.zeros((n, k // 2), dtype=torch.uint8)
        codes[1::2] = 0xFF
        scale = torch.ones((n, 4), dtype=ref.TORCH[kind])
        scale[4:8] = 0.0
        scale[8:12] = big
        scale[12:16] = small
        zero = torch.zeros((n, 4), dtype=torch.uint8)
        zero[2::4] = 15
        zero[3::4] = 15
        x = torch.zeros((3, k), dtype=ref.TORCH[kind])
        x[0, :2] = 1.0
        x[2] = 0.125
        y = torch.empty((3, n), dtype=ref.TORCH[kind], device=DEV)
        MM[kind](dev(x), dev(codes), dev(scale), y, zero=dev(zero), group=group)
        want, _ = ref.product(x, codes, scale, zero, k, group, kind)
        sync()
        assert torch.equal(y.cpu(), ref.rne(want, kind)), kind


def test_a_token_with_nan_leaves_the_others():
    rng = np.random.default_rng(3)
    for m in (4, 16, 100):
        codes, scale, zero = ref.matrix(rng, 48, 512, 32, "bf16", True)
        x = rows_of_x(rng, m, 512, "bf16", False)
        y = torch.empty((m, 48), dtype=torch.bfloat16, device=DEV)
        bq.bq_mm_i4(dev(x), dev(codes), dev(scale), y, zero=dev(zero), group=32)
        want = y.cpu()
        x[1, 77] = float("nan")
        x[m - 1, 5] = float("inf")
        bq.bq_mm_i4(dev(x), dev(codes), dev(scale), y, zero=dev(zero), group=32)
        sync()
        got = y.cpu()
        assert torch.equal(got[2: m - 1], want[2: m - 1]) and torch.equal(got[0], want[0])
        assert bool(torch.isnan(got[1].float()).all())


def test_same_bits_again_and_on_another_stream():
    rng = np.random.default_rng(4)
    codes, scale, zero = (dev(t) for t in ref.matrix(rng, 600, 1024, 64, "bf16", True))
    for m in (1, 16, 150):
        x = dev(rows_of_x(rng, m, 1024, "bf16", False))
        y = [torch.empty((m, 600), dtype=torch.bfloat16, device=DEV) for _ in range(3)]
        bq.bq_mm_i4(x, codes, scale, y[0], zero=zero, group=64)
        bq.bq_mm_i4(x, codes, scale, y[1], zero=zero, group=64)
        sync()
        st = torch.cuda.Stream()
        bq.bq_mm_i4(x, codes, scale, y[2], zero=zero, group=64, stream=st)
        st.synchronize()
        assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])


def test_weights_past_32_bit_offsets():
    """A matrix of more than 2^31 code bytes: its last rows are the right ones."""
    n, k = 16400, 2 * 131072 + 128
    say(f"mm_i4 n={n} k={k}: {n * (k // 2) / 2**31:.2f} x 2^31 bytes of codes")
    codes = torch.zeros((n, -(-(k // 2) // 16) * 16), dtype=torch.uint8, device=DEV)
    assert codes.numel() > 2 ** 31
    groups = k // 128
    scale = torch.ones((n, -(-groups // 4) * 4), dtype=torch.bfloat16, device=DEV)
    codes[:, : k // 2] = 0x88                       # every value 0
    codes[n - 1, k // 2 - 1] = 0xA9                 # columns k-2: +1, k-1: +2
    codes[n - 2, 0] = 0x78                          # column 1: -1
    for m in (1, 70):
        x = torch.ones((m, k), dtype=torch.bfloat16, device=DEV)
        y = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
        bq.bq_mm_i4(x, codes, scale, y, group=128)
        sync()
        assert y[m - 1, n - 1].item() == 3.0 and y[0, n - 2].item() == -1.0
        assert bool((y[:, : n - 2] == 0).all())


@pytest.mark.parametrize("m,n", [(4, 40), (16, 40), (17, 40), (17, 20000), (70, 6100)])
def test_rows_of_x_far_apart(m, n):
    """Rows of x more than 2^31 bytes apart in all, for every kernel."""
    rng = np.random.default_rng([m, n])
    k, ld = 640, 8 * ((1 << 28) // m + 1)
    say(f"mm_i4 m={m} n={n} ldx={ld}")
    codes, scale, zero = ref.matrix(rng, n, k, 64, "bf16", True, exact=True)
    x = rows_of_x(rng, m, k, "bf16", True)
    base = torch.empty((m - 1) * ld + k, dtype=torch.bfloat16, device=DEV)
    far = base.as_strided((m, k), (ld, 1))
    far.copy_(x)
    y = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    bq.bq_mm_i4(far, dev(codes), dev(scale), y, zero=dev(zero), group=64)
    sync()
    want, _ = ref.product(x, codes, scale, zero, k, 64, "bf16")
    assert torch.equal(y.cpu(), ref.rne(want, "bf16"))


# ---- expert products -----------------------------------------------------------------------

def check_experts(counts, n, k, group, kind, zeros, gathered, exact=True, tail=0, seed=0):
    say(f"moe_mm_i4 counts={counts[:8]} n={n} k={k} group={group} {kind} gathered={gathered}")
    rng = np.random.default_rng([n, k, group, zeros, gathered, seed, *counts])
    mats = [ref.matrix(rng, n, k, group, kind, zeros, exact=exact) for _ in counts]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    kept, topk = int(off[-1]), 2
    rows = kept + tail
    x_rows = max(1, rows // 2 + 1) if gathered else max(rows, 1)
    x = rows_of_x(rng, x_rows, k, kind, exact)
    src = rng.integers(0, x_rows * topk, rows).astype(np.int32) if gathered else None
    pick = src // topk if gathered else np.arange(rows)
    y = torch.full((max(rows, 1), n), 5.0, dtype=ref.TORCH[kind], device=DEV)
    MOE[kind](dev(x), dev(torch.from_numpy(off)), dev(torch.stack([a[0] for a in mats])),
              dev(torch.stack([a[1] for a in mats])), y,
              zero=dev(torch.stack([a[2] for a in mats])) if zeros else None, group=group,
              src=None if src is None else dev(torch.from_numpy(src)), topk=topk)
    sync()
    got = y.cpu()
    for e, (c, s, z) in enumerate(mats):
        lo, hi = off[e], off[e + 1]
        want, bound = ref.product(x[pick[lo:hi]], c, s, z, k, group, kind)
        if exact:
            assert torch.equal(got[lo:hi], ref.rne(want, kind)), e
        else:
            assert (np.abs(got[lo:hi].double().numpy() - want) <= bound).all(), e
    assert bool((got[kept:] == 5.0).all())      # rows of no expert are not written


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [3, 0, 0, 17, 1], [0, 0], [5] * 9,
                                    [130, 0, 1, 64, 65], [300, 2, 0, 257]])
def test_experts(counts, gathered, kind):
    check_experts(counts, 33, 256, 64, kind, True, gathered, tail=3)
    check_experts(counts, 48, 512, 128, kind, False, gathered, exact=False)
    check_experts(counts, 20, 160, 32, kind, True, gathered)


def test_many_experts():
    rng = np.random.default_rng(9)
    check_experts(rng.integers(0, 4, 1024).tolist(), 17, 64, 32, "bf16", True, True)
    check_experts(rng.integers(0, 40, 300).tolist(), 140, 256, 128, "f16", False, True)


def test_expert_offsets_out_of_range_stay_inside():
    """Offsets and sources that no sort wrote: rows past the arrays are never touched."""
    rng = np.random.default_rng(11)
    c, s, _ = ref.matrix(rng, 32, 128, 128, "bf16", False)
    x = rows_of_x(rng, 6, 128, "bf16", True)
    y = torch.full((40, 32), 5.0, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([-7, 4, 1 << 29, 3], dtype=torch.int32, device=DEV)
    src = torch.full((8,), 1 << 29, dtype=torch.int32, device=DEV)
    src[0] = 3
    three = lambda t: dev(torch.stack([t] * 3))  # noqa: E731
    bq.bq_moe_mm_i4(dev(x), off, three(c), three(s), y[:8], group=128, src=src, topk=1)
    sync()
    want, _ = ref.product(x[3:4], c, s, None, 128, 128, "bf16")
    assert torch.equal(y[:1].cpu(), ref.rne(want, "bf16"))
    assert bool((y[1:8] == 0).all()) and bool((y[8:] == 5.0).all())


# ---- the codec -----------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,groups", [(1, 1), (3, 1), (7, 5), (65, 9), (1001, 8), (2, 337)])
def test_codec(rows, groups, group, kind):
    say(f"quant_i4 rows={rows} cols={groups * group} group={group} {kind}")
    rng = np.random.default_rng([rows, groups, group])
    cols = groups * group
    v = rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-8, 8, (rows, 1)))
    v[rng.random((rows, cols)) < 0.01] *= 50
    v[rng.random(rows) < 0.1] = 0.0
    if rows > 2:       # subnormals of the type, ties and the largest values
        v[0] = rng.integers(-20, 21, cols) * (2.0 ** -133 if kind == "bf16" else 2.0 ** -24)
        v[1] = rng.integers(-14, 15, cols) * 0.5
        v[1, ::group] = 7.0
        v[2] = rng.choice([-1.0, 1.0], cols) * (3.3e38 if kind == "bf16" else 65504.0)
    if kind == "f16":
        v = np.clip(v, -65504, 65504)
    x = torch.full((rows, cols + 8), float("nan")).to(ref.TORCH[kind])
    x[:, :cols] = torch.from_numpy(v).to(ref.TORCH[kind])
    ldc, lds = -(-(cols // 2) // 16) * 16 + 16, -(-groups // 4) * 4 + 4
    c = torch.full((rows, ldc), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((rows, lds), 3.0, dtype=ref.TORCH[kind], device=DEV)
    QUANT[kind](dev(x), c, s, group=group, cols=cols)
    y = torch.full((rows, cols + 8), 3.0, dtype=ref.TORCH[kind], device=DEV)
    DEQUANT[kind](c, s, y, group=group, cols=cols)
    zero = torch.from_numpy(rng.integers(0, 16, (rows, lds)).astype(np.uint8))
    yz = torch.full((rows, cols + 8), 3.0, dtype=ref.TORCH[kind], device=DEV)
    DEQUANT[kind](c, s, yz, zero=dev(zero), group=group, cols=cols)
    sync()
    wc, ws = ref.quant(x[:, :cols], group, kind)
    assert np.array_equal(c.cpu().numpy()[:, : cols // 2], wc)
    assert torch.equal(s.cpu()[:, :groups].view(torch.int16), ws.view(torch.int16))
    assert bool((c[:, cols // 2:] == 0xA5).all()) and bool((s[:, groups:] == 3.0).all())
    for got, z in ((y, None), (yz, zero)):
        w, _, _, _ = ref.dense(torch.from_numpy(wc), ws, z, cols, group)
        with np.errstate(over="ignore"):
            want = torch.from_numpy(w.astype(np.float32)).to(ref.TORCH[kind])
        assert torch.equal(got.cpu()[:, :cols], want)
        assert bool((got[:, cols:] == 3.0).all())
