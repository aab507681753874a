"""Attention over the 4-bit cache on the GPU, against the 64-bit form of kv_ref within its bound."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_ref as ref
from gpu_util import DEV, say, sync
from test_gpu_kv import WIDTHS, on_gpu

import block_quantized_wire_amd as bq

pytestmark = pytest.mark.gpu

ATTN = {"bf16": bq.bq_attn_i4, "f16": bq.bq_attn_i4_f16}


class Case:
    """A filled pool, sequences on pages in any order, and rows of q out of a wider projection."""

    def __init__(self, seed, lens, new, heads, kv_heads, dim, group, page, kind, gap=0, outer=False,
                 spare=2, q_size=2.0):
        rng = np.random.default_rng(seed)
        self.kind, self.dim, self.heads, self.lens = kind, dim, heads, list(lens)
        need = [-(-n // page) for n in lens]
        self.pool = ref.Pool(sum(need) + spare, kv_heads, page, dim, group, kind).random(rng)
        order = rng.permutation(self.pool.pages)
        cols = max(1, max(need))
        # what a table holds behind a sequence's pages is anything
        self.table = rng.choice([-1, -(1 << 31), (1 << 31) - 1, 0], (len(lens), cols)).astype(np.int32)
        used = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[used:used + n]
            used += n
        self.starts = None
        rows = len(lens)
        if new is not None:
            self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
            rows = int(self.starts[-1])
        self.max_q = 1 if new is None else max(1, max(new))
        x = torch.from_numpy(rng.normal(0, q_size, (rows, heads + 1, dim)).astype(np.float32))
        self.q = x.to(ref.TORCH[kind]).to(DEV)[:, :heads]
        self.gap, self.outer = gap, outer
        self.cache = None

    def arrays(self):
        if self.cache is None:
            self.cache = on_gpu(self.pool, self.outer, self.gap)
        t = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).to(DEV)  # noqa: E731
        return t(self.table), t(self.lens), t(self.starts)

    def run(self, causal=True, window=0, scale=None, max_len=None, extra=0, stream=None, lse=True, ws=None):
        table, lens, starts = self.arrays()
        rows = self.q.shape[0]
        q = self.q
        if extra:       # rows behind the last sequence
            q = torch.cat([q, q[:1].expand(extra, -1, -1)])
        out = torch.full((rows + extra, self.heads, self.dim), 123.0, dtype=q.dtype, device=DEV)
        l = torch.full((rows + extra, self.heads), 123.0, device=DEV)
        most = max(self.lens) if max_len is None else max_len
        need = bq.bq_attn_i4_ws_bytes(len(self.lens), rows + extra, self.max_q, most, self.heads,
                                      self.pool.heads, self.dim)
        assert 0 <= need <= 64 << 20
        if ws is None and need:
            ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)       # NaN
        ATTN[self.kind](q, self.cache, table, lens, out, starts=starts, max_q=self.max_q, max_len=most,
                        causal=causal, window=window, scale=scale, lse=l if lse else None, ws=ws, stream=stream)
        return out, l

    def want(self, causal=True, window=0, scale=None):
        return ref.attend(self.pool, self.q.cpu(), self.table, self.lens, self.starts, causal, window,
                          self.dim ** -0.5 if scale is None else scale, self.kind)

    def check(self, **how):
        got, lse = self.run(**how)
        sync()
        keep = {k: how[k] for k in ("causal", "window", "scale") if k in how}
        y, l, ey, el = self.want(**keep)
        n = self.q.shape[0]
        far = np.abs(got[:n].cpu().double().numpy() - y)
        assert np.isfinite(got[:n].float().cpu().numpy()).all()
        assert (far <= ey).all(), float((far / np.maximum(ey, 1e-300)).max())
        seen = np.isfinite(l)
        found = lse[:n].cpu().double().numpy()
        assert (found[~seen] == -np.inf).all() and (got[:n].cpu()[torch.from_numpy(~seen)] == 0).all()
        assert (np.abs(found - np.where(seen, l, 0))[seen] <= el[seen]).all()
        assert (got[n:] == 123.0).all() and (lse[n:] == 123.0).all()
        return got, lse


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim,group", WIDTHS)
def test_one_token(dim, group, kind):
    for lens, heads, kv_heads, page in (((1,), 1, 1, 8), ((7, 8, 9), 4, 2, 8), ((31, 0, 32, 33, 1), 6, 2, 24),
                                        ((127, 128, 129, 300), 16, 1, 16), ((1001,), 32, 2, 64),
                                        ((5, 2100, 640), 3, 3, 200)):
        say(f"attn one token dim={dim} group={group} {kind} lens={lens} heads={heads}/{kv_heads} page={page}")
        Case([dim, group, len(lens)], lens, None, heads, kv_heads, dim, group, page, kind).check()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim,group", WIDTHS)
def test_some_and_many_tokens(dim, group, kind):
    for lens, new, heads, kv_heads, page, window in (
            ((40, 300), (2, 5), 8, 2, 16, 0), ((5, 64, 3), (5, 17, 9), 12, 3, 8, 0),
            ((400, 33), (70, 33), 4, 2, 24, 0), ((150,), (150,), 6, 2, 64, 40),
            ((700, 90, 260), (65, 1, 129), 2, 1, 40, 100)):
        say(f"attn dim={dim} group={group} {kind} lens={lens} new={new} heads={heads}/{kv_heads} window={window}")
        Case([dim, group, len(lens)], lens, new, heads, kv_heads, dim, group, page, kind).check(window=window)


@pytest.mark.parametrize("dim,group,kind", [(64, 32, "f16"), (128, 64, "bf16"), (256, 128, "f16")])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 2, 31, 32, 33, 10 ** 12])
def test_masks(dim, group, kind, causal, window):
    for lens, new in (((97, 40, 8), None), ((97, 40, 8), (9, 40, 1)), ((260, 5), (200, 20))):
        say(f"attn mask dim={dim} {kind} causal={causal} window={window} lens={lens} new={new}")
        c = Case([dim, window % 97], lens, new, 6, 2, dim, group, 16, kind)
        c.check(causal=causal, window=window)


def test_rows_that_see_nothing():
    """More new rows than tokens: the first rows stand before the sequence.  Empty sequences, and
    sequences without rows."""
    for lens, new in (((3, 0, 40), (10, 4, 0)), ((0, 0), (1, 1)), ((0, 17, 5), (0, 100, 70))):
        for kind in ("bf16", "f16"):
            say(f"attn empty rows lens={lens} new={new} {kind}")
            c = Case([len(lens)], lens, new, 8, 2, 128, 64, 16, kind)
            c.check()
            c.check(causal=False, window=3)


@pytest.mark.parametrize("new", [None, (3, 1), (70, 2)])
def test_tables_without_a_page(new):
    """Rows of sequences that have no page: nothing is read of a table that has no column."""
    say(f"attn no pages new={new}")
    c = Case([1], (0, 0), new, 4, 2, 64, 32, 16, "bf16")
    c.table = c.table[:, :0]
    out, lse = c.run(max_len=0)
    sync()
    assert (out == 0).all() and (lse == float("-inf")).all()


@pytest.mark.parametrize("share", [1, 2, 3, 5, 7, 8, 16, 17, 32, 64])
def test_shared_heads(share):
    for new in (None, (3, 1), (9, 2)):
        say(f"attn share={share} new={new}")
        Case([share], (200, 77), new, 2 * share, 2, 64, 64, 16, "bf16").check()


@pytest.mark.parametrize("lens,new,heads,kv_heads", [((20000,), None, 8, 1), ((9001, 3), (2, 1), 8, 1),
                                                     ((5003,), (40,), 4, 2), ((4100, 4000), (130, 3), 2, 1),
                                                     ((5000, 3000, 10, 0, 700), (1, 8, 5, 0, 2), 8, 1),
                                                     ((0, 900, 4000, 0), (3, 0, 1, 16), 8, 2)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_split_over_the_tokens(lens, new, heads, kv_heads, kind):
    """Few rows and many tokens: workgroups share a sequence and their results are joined."""
    say(f"attn split lens={lens} new={new} {kind}")
    c = Case([sum(lens)], lens, new, heads, kv_heads, 128, 128, 64, kind)
    need = bq.bq_attn_i4_ws_bytes(len(lens), c.q.shape[0], c.max_q, max(lens), heads, kv_heads, 128)
    assert need > 0
    a = c.check(extra=3)
    b = c.run(extra=3)
    sync()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])      # the same call, the same bits
    c.check(window=700)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim,group", WIDTHS)
@pytest.mark.parametrize("new,window", [(None, 0), ((3, 0, 9, 1, 2), 0), ((2, 5, 16, 0, 1), 1000)])
def test_turns_dealt_out(dim, group, kind, new, window):
    """Few rows of a ragged batch with one long sequence: its turns go to many workgroups, those of short
    ones to some of them as well."""
    say(f"attn dealt D={dim} G={group} {kind} new={new} window={window}")
    lens = (2805, 0, 33, 1400, 7)
    c = Case([dim, group], lens, new, 8, 2, dim, group, 24, kind)
    assert bq.bq_attn_i4_ws_bytes(len(lens), c.q.shape[0], c.max_q, max(lens), 8, 2, dim) > 0
    c.check(window=window)


def test_long_sums_are_not_biased():
    """Many tokens of about the same weight: a result is far smaller than its values, and what the sums
    lose on the way must not add up.  A rounding to binary16 is off by at most 2^-11 of a result, to either
    side, so the mean of n of them has a deviation of at most 2^-11 of their size by sqrt(3 n)."""
    for dim, group in ((128, 32), (64, 64), (256, 128)):
        say(f"attn long sums dim={dim}")
        c = Case([dim], (21071,), None, 8, 2, dim, group, 64, "f16", q_size=0.1)
        got, _ = c.check()
        y = c.want()[0]
        off = got.cpu().double().numpy() - y
        assert abs(off.mean()) <= 5 * 2.0 ** -11 * np.sqrt((y * y).mean()) / np.sqrt(3 * y.size)


def test_rows_behind_the_last_sequence_are_left():
    for new, extra in ((None, 5), ((3, 8), 7), ((80, 2), 1)):
        c = Case([extra], (50, 90), new, 4, 2, 128, 32, 8, "bf16")
        c.check(extra=extra)


def test_scales_given_and_large_scores():
    for scale, q_size in ((1.0, 2.0), (-0.3, 1.0), (0.0, 1.0), (1e-6, 1.0), (0.5, 60.0)):
        for new in (None, (5, 70)):
            say(f"attn scale={scale} q={q_size} new={new}")
            Case([7], (300, 90), new, 4, 2, 128, 64, 16, "bf16", q_size=q_size).check(scale=scale)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_sizes_of_q(kind):
    """Rows of q of very different sizes, up to what the score's own rounding allows."""
    c = Case([9], (200,), (48,), 2, 1, 128, 128, 16, kind)
    rng = np.random.default_rng(9)
    lo, hi = (-100, 4) if kind == "bf16" else (-20, 4)
    by = torch.from_numpy(2.0 ** rng.integers(lo, hi, (48, 1, 1))).to(DEV)
    c.q = (c.q.double() * by).to(c.q.dtype)
    c.q[3] = 0
    c.check(scale=0.5)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_sizes_of_values_and_rising_scores(kind):
    """Scales of values that grow and shrink along a sequence, and scores that rise by more than
    the reference's slack again and again."""
    for new in (None, (20, ), (90,)):
        c = Case([11], (900,), new, 4, 1, 128, 32, 16, kind)
        n = c.pool.pages * c.pool.page
        size = 2.0 ** np.interp(np.arange(n), [0, n // 2, n], [-8, 6, -8]).round()
        by = torch.from_numpy(size).view(c.pool.pages, 1, 1, c.pool.page, 1)
        # along the sequence: its pages in their order
        where = np.argsort(np.concatenate([c.table[0], np.setdiff1d(np.arange(c.pool.pages), c.table[0])]))
        c.pool.scales[1] = (c.pool.scales[1].double() * by[where]).to(c.pool.scales[1].dtype)
        ramp = torch.from_numpy(np.linspace(0.02, 1.0, n)).view(c.pool.pages, 1, 1, c.pool.page, 1)
        c.pool.scales[0] = (c.pool.scales[0].double() * ramp[where]).to(c.pool.scales[0].dtype)
        say(f"attn rising {kind} new={new}")
        c.check(scale=0.6)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("new", [None, (4,), (120,)])
def test_unseen_tokens_hold_anything(kind, new):
    """NaN and infinities in the scales of tokens that no row, or not every row, sees, and of pages
    that no sequence has; pages outside the pool are seen by no row."""
    clean = Case([13], (150,), new, 4, 2, 128, 64, 16, kind, spare=3)
    table, lens, starts = clean.arrays()
    dirty = Case([13], (150,), new, 4, 2, 128, 64, 16, kind, spare=3)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")])
    used = set(clean.table[0].tolist())
    for which in (0, 1):
        s = dirty.pool.scales[which]
        for page in range(dirty.pool.pages):
            if page not in used:
                s[page] = bad[page % 3]
        s[int(clean.table[0, 150 // 16]), :, :, 150 % 16:] = float("nan")       # behind the last token
    a, b = clean.check(), dirty.run()
    sync()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    if new is not None:
        # the last token is NaN: under a causal mask only the last row sees it
        for which in (0, 1):
            page, place = int(clean.table[0, 149 // 16]), 149 % 16
            dirty.pool.scales[which][page, :, :, place] = float("nan")
            dirty.cache = None
            c = dirty.run()
            sync()
            assert torch.equal(a[0][:-1], c[0][:-1]) and torch.equal(a[1][:-1], c[1][:-1])
            assert torch.isnan(c[0][-1]).any()
    # a page that is not there
    for page in (-1, clean.pool.pages, (1 << 31) - 1, -(1 << 31)):
        gone = Case([13], (150,), new, 4, 2, 128, 64, 16, kind, spare=3)
        gone.table[0, 4] = page
        gone.check()


def test_numbers_that_are_not_finite_in_q():
    for kind in ("bf16", "f16"):
        for new in (None, (6, 80)):
            c = Case([17], (90, 200), new, 4, 2, 64, 32, 16, kind)
            clean, _ = c.run()
            c.q = c.q.clone()
            c.q[0, 1, 5] = float("nan")
            c.q[1, 2, 63] = float("inf")
            c.q[1, 3, 0] = -float("inf")
            out, lse = c.run()
            sync()
            for row, head in ((0, 1), (1, 2), (1, 3)):
                assert torch.isnan(out[row, head]).all() and torch.isnan(lse[row, head])
                out[row, head] = clean[row, head]
            assert torch.equal(out, clean)


@pytest.mark.parametrize("outer,gap", [(False, 0), (True, 0), (False, 2), (True, 3)])
def test_layouts_of_the_pool(outer, gap):
    for new in (None, (3, 90)):
        Case([19], (300, 140), new, 6, 3, 128, 64, 24, "f16", gap=gap, outer=outer).check()


def test_lengths_beyond_what_is_given_are_brought_inside():
    """lens larger than the table has room for or than max_len, or negative; starts that fall, pass
    the rows or leave more rows than max_q."""
    c = Case([23], (64, 40), None, 2, 1, 64, 64, 16, "bf16")
    good, _ = c.check()
    table, lens, _ = c.arrays()
    lens.copy_(torch.tensor([1 << 30, -5], dtype=torch.int32))
    out, lse = torch.full_like(good, 9.0), torch.zeros((2, 2), device=DEV)
    bq.bq_attn_i4(c.q, c.cache, table, lens, out, lse=lse, max_len=64)
    sync()
    assert torch.equal(out[0], good[0]) and (out[1] == 0).all() and (lse[1] == -float("inf")).all()
    c = Case([29], (64, 40), (3, 4), 2, 1, 64, 64, 16, "bf16")
    good, _ = c.check()
    table, lens, starts = c.arrays()
    out = torch.full_like(good, 9.0)
    starts.copy_(torch.tensor([3, 7, 2], dtype=torch.int32))
    bq.bq_attn_i4(c.q, c.cache, table, lens.flip(0).contiguous(), out, starts=starts, max_q=4, max_len=64)
    sync()
    assert (out[:3] == 9.0).all()
    starts.copy_(torch.tensor([0, 3, 1 << 30], dtype=torch.int32))
    bq.bq_attn_i4(c.q, c.cache, table, lens, out, starts=starts, max_q=4, max_len=64)
    sync()
    assert torch.equal(out, good)
    out.fill_(9.0)
    starts.copy_(torch.tensor([-7, 3, 7], dtype=torch.int32))
    bq.bq_attn_i4(c.q, c.cache, table, lens, out, starts=starts, max_q=2, max_len=64)
    sync()
    assert (out[[2, 5, 6]] == 9.0).all() and torch.isfinite(out).all()


def test_two_calls_at_once_and_a_side_stream():
    a = Case([31], (5000,), None, 8, 1, 128, 128, 64, "bf16")
    b = Case([37], (4000,), None, 8, 1, 128, 32, 64, "f16")
    wa, wb = a.check(), b.check()
    sides = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        got = []
        for c, s in ((a, sides[0]), (b, sides[1])):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(c.run())
        sync()
        assert torch.equal(got[0][0], wa[0]) and torch.equal(got[1][0], wb[0])
        assert torch.equal(got[0][1], wa[1]) and torch.equal(got[1][1], wb[1])


def test_captured_and_replayed():
    """A decode step in a graph: lengths and tables change between the replays."""
    c = Case([41], (3000, 900), None, 8, 2, 128, 64, 16, "bf16")
    table, lens, _ = c.arrays()
    out, lse = torch.zeros_like(c.q), torch.zeros((2, 8), device=DEV)
    need = bq.bq_attn_i4_ws_bytes(2, 2, 1, 3000, 8, 2, 128)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    q = c.q.clone()
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bq.bq_attn_i4(q, c.cache, table, lens, out, max_len=3000, lse=lse, ws=ws)
    for turn, now in enumerate(((3000, 900), (1, 900), (2999, 0), (128, 129))):
        c.lens = list(now)
        c.q = (c.q.float() * 0.9).to(c.q.dtype)
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        q.copy_(c.q)
        graph.replay()
        sync()
        eager = c.run(max_len=3000)
        sync()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        c.check()


def test_long_cache_beyond_32_bit_offsets():
    """Pages and rows of q more than 2^32 bytes apart."""
    c = Case([43], (40, 24), None, 4, 2, 64, 64, 8, "bf16", spare=0)
    c.arrays()
    pool, far = c.pool, 3 << 28          # 8 pages: 6 GiB
    parts = []
    say("attn pool of 8 pages 768 MiB apart")
    for which in (0, 1):
        codes = torch.empty(pool.pages * far, dtype=torch.uint8, device=DEV)
        scale = torch.empty(pool.pages * far // 2, dtype=torch.bfloat16, device=DEV)
        ck = codes.as_strided((8, 2, 8, 32), (far, 256, 32, 1))
        sk = scale.as_strided((8, 2, 1, 8, 2), (far // 2, 16, 16, 2, 1))
        ck.copy_(torch.from_numpy(pool.codes[which]).view(8, 2, 8, 32).to(DEV))
        sk.copy_(pool.scales[which].to(DEV))
        parts += [ck, sk]
    near = c.check()
    c.cache = bq.KvI4(parts[0], parts[2], parts[1], parts[3], group=64)
    got = c.run()
    sync()
    assert torch.equal(near[0], got[0]) and torch.equal(near[1], got[1])


def test_without_lse_and_defaults():
    c = Case([47], (48, 16), None, 4, 2, 128, 128, 16, "f16")
    want, _ = c.check()
    table, lens, _ = c.arrays()
    out = torch.zeros_like(want)
    bq.bq_attn_i4_f16(c.q, c.cache, table, lens, out)
    sync()
    assert torch.equal(out, want)
