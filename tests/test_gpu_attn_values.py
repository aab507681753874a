"""Attention over the 4-bit cache where sizes of values differ: blocks of zeros, very small and very
unequal values, values beyond binary16's range.  Against kv_ref's 64-bit form."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_ref as ref
from gpu_util import DEV, say, sync
from test_gpu_attn import Case
from test_gpu_kv import WIDTHS

import block_quantized_wire_amd as bq

pytestmark = pytest.mark.gpu


def places(c, tokens, b=0):
    """(page, place) of tokens of a sequence."""
    return [(int(c.table[b, t // c.pool.page]), t % c.pool.page) for t in tokens]


def scale_values(c, tokens, by):
    """The values of these tokens times a power of two (exact, as long as it stays in range)."""
    for page, place in places(c, tokens):
        s = c.pool.scales[1][page, :, :, place]
        c.pool.scales[1][page, :, :, place] = (s.double() * by).to(s.dtype)


def near(c, **how):
    """Like Case.check, with what the header grants small values beside large ones.

    A weight times 2^(6 + k - b) (many rows; b, k: the power of two of a block of 8 tokens, and of the
    sequence) or times a scale and 2^k (few rows) is a binary16 number, whose steps below 2^-14 are 2^-24, so
    it is off by 2^-25 at most.  The block's values times 2^b are below 2^15 and the sequence's largest,
    top, times 2^k is 2^14 or more: that is 2^-25 * 2^15 / 2^6 * top / 2^14 = 2^-30 top a token.  Few rows:
    codes are up to 8 from the middle and the largest scale times 2^k is 2^6 or more where the weight of the
    reference is 1: 2^-25 * 8 / 2^6 = 2^-28 of the largest scale a token.  Weights sum to 1 or more then.
    2^-27 top covers both."""
    got, lse = c.run(**how)
    sync()
    y, l, ey, el = c.want(**how)
    n = max(c.lens)
    pairs = c.pool.scales[1].double().numpy()
    used = np.concatenate([c.table[b, : -(-m // c.pool.page)] for b, m in enumerate(c.lens)])
    s, m = pairs[used, ..., 0], pairs[used, ..., 1]
    top = (8 * np.abs(s) + np.abs(m + 8 * s)).max()
    far = np.abs(got.cpu().double().numpy() - y)
    assert np.isfinite(far).all()
    assert (far <= ey + n * 2.0 ** -27 * top).all()
    seen = np.isfinite(l)
    found = lse.cpu().double().numpy()
    assert (found[~seen] == -np.inf).all()
    assert (np.abs(found - np.where(seen, l, 0))[seen] <= el[seen]).all()
    return got, lse


@pytest.mark.parametrize("dim,group,size", [(d, g, -30) for d, g in WIDTHS] +
                         [(64, 32, -60), (128, 64, -110), (256, 128, -110)])
def test_values_that_are_all_small(dim, group, size):
    """Tokens behind a sequence's end and before a window, and a block of zeros, have no size of their
    own: the small values beside them keep their bits."""
    for lens, new, window in (((150,), (120,), 0), ((150,), (120,), 61), ((150, 41), (66, 1), 0), ((150,), (17,), 0),
                              ((150, 41), None, 0)):
        say(f"attn small values D={dim} G={group} 2^{size} new={new} window={window}")
        c = Case([dim, group, 1], lens, new, 4, 1, dim, group, 16, "bf16")
        c.pool.scales[1] = (c.pool.scales[1].double() * 2.0 ** size).to(torch.bfloat16)
        c.check(window=window)
        for page, place in places(c, range(40, 48)):
            c.pool.scales[1][page, :, :, place] = 0
        c.cache = None
        c.check(window=window)


@pytest.mark.parametrize("dim,group", WIDTHS)
@pytest.mark.parametrize("new", [(120,), (100, 3)])
def test_many_rows_of_very_unequal_values(dim, group, new):
    """Blocks near 2^-90 beside others near 2^60, either first: small values go, weights and
    log-sum-exps stay."""
    lens = (150,) if len(new) == 1 else (150, 30)
    for first, then in ((60, -90), (-90, 60), (0, -80), (-85, 90)):
        say(f"attn unequal D={dim} G={group} new={new} 2^{first} then 2^{then}")
        c = Case([dim, group, 2], lens, new, 4, 2, dim, group, 16, "bf16", q_size=1.0)
        scale_values(c, range(64), 2.0 ** first)
        scale_values(c, range(64, 150), 2.0 ** then)
        near(c)
        near(c, window=70)


@pytest.mark.parametrize("dim,group", WIDTHS)
@pytest.mark.parametrize("new", [None, (4,), (3, 8)])
def test_few_rows_of_very_unequal_values(dim, group, new):
    lens = (150, 30) if new is not None and len(new) > 1 else (150,)
    for first, then in ((60, -90), (-90, 60), (0, -80), (-85, 90)):
        say(f"attn unequal D={dim} G={group} new={new} 2^{first} then 2^{then}")
        c = Case([dim, group, 3], lens, new, 4, 2, dim, group, 16, "bf16", q_size=1.0)
        scale_values(c, range(128), 2.0 ** first)       # a turn of the four waves, each of which has both
        scale_values(c, range(128, 150), 2.0 ** then)
        near(c)
    # long enough that turns are dealt out and joined
    c = Case([dim, group, 4], (3000,), new and (4,), 8, 1, dim, group, 64, "bf16", q_size=1.0)
    scale_values(c, range(500, 1700), 2.0 ** -85)
    scale_values(c, range(1700, 3000), 2.0 ** 80)
    near(c)


def test_scales_that_are_far_below_their_least_values():
    """Groups of nearly equal numbers, some exactly equal: sums of least values stay in range whatever the
    power of two of the scales."""
    for kind in ("bf16", "f16"):
        for new in (None, (4,), (90,)):
            say(f"attn tiny scales {kind} new={new}")
            c = Case([5], (300,), new, 4, 2, 128, 64, 16, kind, q_size=1.0)
            by = 2.0 ** -95 if kind == "bf16" else 0.0
            v = c.pool.scales[1]
            v[..., 0] = (v[..., 0].double() * by).to(v.dtype)
            if kind == "bf16":
                v[..., 1] = (v[..., 1].double() * 2.0 ** 40).to(v.dtype)
            near(c)


@pytest.mark.parametrize("dim,group", WIDTHS)
@pytest.mark.parametrize("new", [(120,), (66, 3), (4,)])
def test_binary16_values_beyond_the_range(dim, group, new):
    """Finite scales and least values whose 15 s + m is 65536, which binary16 does not hold: rows that do
    not see the token lose nothing by it, the others have the value itself."""
    lens = (150,) if len(new) == 1 else (150, 20)
    first = 149 - new[0] + 1            # place of the sequence's first row
    for token in (149, first + 2):
        c = Case([dim, group, 6], lens, new, 4, 2, dim, group, 16, "f16", q_size=0.1)
        page, place = places(c, [token])[0]
        codes = np.full((2, dim), 15, np.uint8)
        codes[:, ::2] = 0
        c.pool.put(1, page * 16 + place, codes, torch.full((2, dim // group), 8736.0).half(),
                   torch.full((2, dim // group), -65504.0).half())
        say(f"attn beyond binary16 D={dim} G={group} new={new} token={token}")
        near(c)


@pytest.mark.parametrize("low", [0.0, -65504.0])
def test_binary16_rows_of_the_largest_range_are_written_and_attended(low):
    """What bq_kv_write_i4_f16 makes of rows up to 65504: a scale whose 15 steps pass the type's range."""
    c = Case([8], (150,), (120,), 4, 2, 128, 64, 16, "f16", q_size=0.1)
    c.arrays()
    page, place = places(c, [149])[0]
    x = torch.full((1, 2, 128), low, dtype=torch.float16, device=DEV)
    x[..., ::2] = 65504.0
    k = torch.zeros_like(x)
    bq.bq_kv_write_i4_f16(k, x, torch.tensor([page * 16 + place], dtype=torch.int32, device=DEV), c.cache)
    for which, rows in enumerate((k, x)):
        codes, s, m = ref.quantise(rows.cpu(), 64, "f16")
        assert which == 0 or float((15 * s.double() + m.double()).max()) > 65504
        c.pool.put(which, page * 16 + place, codes[0], s[0], m[0])
    near(c)


def test_a_weight_of_zero_beside_a_value_beyond_binary16():
    """Rows see the token, but its score is so low that its weight is 0."""
    c = Case([9], (150,), (120,), 4, 2, 64, 32, 16, "f16")
    page, place = places(c, [10])[0]
    slot = page * 16 + place
    # the keys of the token are 0; every other key has a score of some 200 and more
    c.q = torch.full_like(c.q, 4.0)
    for which in (0, 1):
        c.pool.put(which, slot, np.full((2, 64), 15, np.uint8), torch.full((2, 2), 8736.0 if which else 0.0).half(),
                   torch.full((2, 2), -65504.0 if which else 0.0).half())
    k = c.pool.scales[0]
    k[..., 1] = (k[..., 1].float() + 20.0).half()
    c.pool.scales[0][page, :, :, place] = 0
    got, _ = near(c)
    assert float(got.abs().max()) < 100.0


@pytest.mark.parametrize("dim,group", WIDTHS)
@pytest.mark.parametrize("new", [(120,), (4,)])
def test_unseen_values_as_large_as_bf16_holds(dim, group, new):
    """The last token's scales and least values are finite, its values are not: rows that do not see it are
    finite, and their log-sum-exps are right."""
    for scale, least in ((1.5 * 2.0 ** 127, -2.0 ** 127), (2.0 ** 124, 1.5 * 2.0 ** 127), (2.0 ** 110, 0.0)):
        say(f"attn largest unseen values D={dim} G={group} new={new} {scale}")
        c = Case([dim, group, 10], (150,), new, 4, 2, dim, group, 16, "bf16", q_size=1.0)
        page, place = places(c, [149])[0]
        c.pool.scales[1][page, :, :, place, 0] = scale
        c.pool.scales[1][page, :, :, place, 1] = least
        got, lse = c.run()
        sync()
        _, l, _, el = c.want()
        assert torch.isfinite(got[:-1]).all()
        assert (np.abs(lse.cpu().double().numpy() - l)[:-1] <= el[:-1]).all()


@pytest.mark.parametrize("n", [3000, 1 << 22])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 64), (256, 128)])
def test_long_sums_of_the_largest_values_stay_in_range(dim, group, n):
    """Scores of 0 and values of 2^100.  Sums of n equal terms in binary32, 32 tokens or more to a step, are off
    by 2^-24 a step: 2^-7 for 2^22 tokens, as is the sum of the weights."""
    pages, size = 4, 256
    codes = torch.zeros((pages, 1, size, dim // 2), dtype=torch.uint8, device=DEV)
    scales = [torch.zeros((pages, 1, dim // group, size, 2), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    scales[1][..., 1] = 2.0 ** 100
    cache = bq.KvI4(codes, codes.clone(), *scales, group=group)
    cols = -(-n // size)
    table = (torch.arange(cols, dtype=torch.int32, device=DEV) % pages)[None].contiguous()
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    for rows in (1, 80):
        say(f"attn largest values D={dim} n={n} rows={rows}")
        q = torch.ones((rows, 1, dim), dtype=torch.bfloat16, device=DEV)
        out, lse = torch.empty_like(q), torch.empty((rows, 1), device=DEV)
        starts = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
        need = bq.bq_attn_i4_ws_bytes(1, rows, rows, n, 1, 1, dim)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        bq.bq_attn_i4(q, cache, table, lens, out, starts=starts, max_q=rows, max_len=n, causal=False, lse=lse, ws=ws)
        sync()
        assert ((out.float() * 2.0 ** -100 - 1).abs() < 2.0 ** -5).all()
        assert ((lse.double() - float(np.log(n))).abs() < 2.0 ** -6).all()
