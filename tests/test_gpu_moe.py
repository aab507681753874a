"""The expert layer's sort, gather, combine and gradients on the GPU against plain forms on
the host: the order and copies exactly, the weighted sums bit for bit (their order is part
of the definition), the weights' gradient within the bound of binary32 sums."""
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

COMBINE = {"bf16": bq.bq_moe_combine, "f16": bq.bq_moe_combine_f16, "f32": bq.bq_moe_combine_f32}
BWD = {"bf16": bq.bq_moe_combine_bwd, "f16": bq.bq_moe_combine_bwd_f16,
       "f32": bq.bq_moe_combine_bwd_f32}


def choices(rng, tokens, topk, experts, drop):
    ids = rng.integers(0, experts, (tokens, topk)).astype(np.int32)
    gone = rng.random(ids.shape) < drop
    ids[gone] = rng.choice([-1, -(1 << 31), experts, (1 << 31) - 1], int(gone.sum()))
    return ids


def sort_on_gpu(ids, experts, stream=None):
    tokens, topk = ids.shape
    n = tokens * topk
    off = torch.full((experts + 1,), -9, dtype=torch.int32, device=DEV)
    src = torch.full((n,), -9, dtype=torch.int32, device=DEV)
    pos = torch.full((n,), -9, dtype=torch.int32, device=DEV)
    need = bq.bq_moe_sort_ws_bytes(tokens, topk, experts)
    ws = torch.full((need,), 0x5A, dtype=torch.uint8, device=DEV) if need else None
    bq.bq_moe_sort(torch.from_numpy(ids).to(DEV), experts, off, src, pos, ws, stream=stream)
    return off, src, pos


@pytest.mark.parametrize("tokens,topk,experts,drop", [
    (1, 1, 1, 0.0), (1, 1, 1, 1.0), (1, 8, 256, 0.0), (3, 2, 5, 0.3), (63, 1, 4, 0.0),
    (64, 1, 4, 0.1), (65, 1, 1024, 0.0), (511, 1, 2, 0.5), (512, 1, 1, 0.0), (513, 3, 511, 0.1),
    (512, 8, 512, 0.0), (4097, 1, 7, 0.2), (1024, 8, 512, 0.0), (8193, 1, 7, 0.2), (1025, 8, 64, 0.0), (4097, 6, 48, 0.125),
    (20000, 8, 256, 0.0), (20000, 8, 1024, 0.5), (70000, 64, 3, 0.1), (300, 64, 513, 0.0),
])
def test_sort(tokens, topk, experts, drop):
    say(f"moe_sort tokens={tokens} topk={topk} experts={experts} drop={drop}")
    rng = np.random.default_rng([tokens, topk, experts])
    ids = choices(rng, tokens, topk, experts, drop)
    got = sort_on_gpu(ids, experts)
    sync()
    for g, w in zip(got, ref.sort(ids, experts)):
        assert np.array_equal(g.cpu().numpy(), w)


def test_sort_one_expert_takes_all_and_none():
    for fill in (0, 6, -1):
        ids = np.full((9000, 2), fill, np.int32)
        got = sort_on_gpu(ids, 7)
        sync()
        for g, w in zip(got, ref.sort(ids, 7)):
            assert np.array_equal(g.cpu().numpy(), w)


def test_sort_of_no_tokens():
    got = sort_on_gpu(np.empty((0, 4), np.int32), 5)
    sync()
    assert got[0].tolist() == [0] * 6


def order(rng, tokens, topk, experts, drop):
    off, src, pos = ref.sort(choices(rng, tokens, topk, experts, drop), experts)
    t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    return off, src, pos, t(off), t(pos)


def strided(values, pad, kind, shift):
    """A device matrix with row stride cols + pad, starting `shift` values into its buffer; what
    lies around the rows holds NaN."""
    rows, cols = values.shape
    ld = cols + pad
    buf = torch.full((rows * ld + shift + 8,), float("nan")).to(ref.TORCH[kind])
    view = torch.as_strided(buf, (rows, cols), (ld, 1), shift)
    view.copy_(values)
    buf = buf.to(DEV)
    return buf, torch.as_strided(buf, (rows, cols), (ld, 1), shift)


def untouched(buf, view):
    """Nothing around the rows was written."""
    keep = torch.ones(buf.shape, dtype=torch.bool, device=buf.device)
    torch.as_strided(keep, view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool(torch.isnan(buf.float()[keep]).all())


SHAPES = [(1, 1, 1, 0.0, 1), (1, 8, 16, 0.0, 8), (2, 3, 4, 0.5, 7), (5, 8, 16, 0.3, 9),
          (33, 6, 48, 0.125, 2055), (64, 4, 8, 0.0, 2048), (17, 9, 12, 0.4, 4100),
          (7, 64, 128, 0.1, 513), (40, 2, 4, 1.0, 100), (300, 8, 64, 0.0, 264)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (1, 1), (3, 5)])
@pytest.mark.parametrize("tokens,topk,experts,drop,cols", SHAPES)
def test_gather(tokens, topk, experts, drop, cols, pad, shift, kind):
    say(f"moe_gather tokens={tokens} topk={topk} cols={cols} {kind} pad={pad} shift={shift}")
    rng = np.random.default_rng([tokens, topk, cols])
    off, src, pos, off_d, pos_d = order(rng, tokens, topk, experts, drop)
    x = torch.from_numpy(rng.standard_normal((tokens, cols))).to(ref.TORCH[kind])
    x[0, 0] = float("nan")
    _, xd = strided(x, pad, kind, shift)
    buf, out = strided(torch.full((len(src), cols), float("nan")).to(ref.TORCH[kind]), pad, kind,
                       shift)
    bq.bq_moe_gather(xd, pos_d, off_d, out, topk=topk)
    sync()
    want = x[torch.from_numpy(src).long() // topk]
    want[off[-1]:] = 0
    i = torch.int32 if kind == "f32" else torch.int16
    assert torch.equal(out.cpu().contiguous().view(i), want.view(i))
    assert untouched(buf, out)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (1, 1), (3, 5)])
@pytest.mark.parametrize("tokens,topk,experts,drop,cols", SHAPES)
def test_combine_and_its_gradient(tokens, topk, experts, drop, cols, pad, shift, kind):
    say(f"moe_combine tokens={tokens} topk={topk} cols={cols} {kind} pad={pad} shift={shift}")
    rng = np.random.default_rng([tokens, topk, cols, 1])
    off, src, pos, off_d, pos_d = order(rng, tokens, topk, experts, drop)
    kept = int(off[-1])
    rows = torch.from_numpy(rng.standard_normal((len(src), cols))).to(ref.TORCH[kind])
    rows[kept:] = float("nan")                    # nothing of a dropped row is used
    weight = rng.standard_normal((tokens, topk)).astype(np.float32)
    weight[(pos >= kept).reshape(tokens, topk)] = np.inf
    wd = torch.from_numpy(weight).to(DEV)
    _, rd = strided(rows, pad, kind, shift)
    blank = torch.full((tokens, cols), float("nan")).to(ref.TORCH[kind])
    for w, w_dev in ((weight, wd), (None, None)):
        buf, y = strided(blank, pad, kind, shift)
        COMBINE[kind](rd, pos_d, off_d, y, weight=w_dev, topk=topk)
        sync()
        want = ref.combine32(rows, pos, kept, w, topk)
        assert torch.equal(y.cpu(), ref.rne(want, kind)), w is None
        assert untouched(buf, y)

    dy = torch.from_numpy(rng.standard_normal((tokens, cols))).to(ref.TORCH[kind])
    _, dyd = strided(dy, pad, kind, shift)
    buf, drows = strided(torch.full((len(src), cols), float("nan")).to(ref.TORCH[kind]), pad, kind,
                         shift)
    dw = torch.full((tokens, topk), float("nan"), device=DEV)
    BWD[kind](dyd, rd, pos_d, off_d, wd, drows, dw)
    sync()
    token = src // topk
    live = np.arange(len(src)) < kept
    want = np.zeros((len(src), cols), np.float32)
    want[live] = weight.reshape(-1)[src[live], None] * dy.float().numpy()[token[live]]
    assert torch.equal(drows.cpu(), ref.rne(want, kind))
    assert untouched(buf, drows)
    r, g = rows.double().numpy()[pos], dy.double().numpy()[np.arange(len(src)) // topk]
    on = pos < kept
    full = np.where(on[:, None], r * g, 0.0)
    off_by = np.abs(dw.cpu().double().numpy().reshape(-1) - full.sum(1))
    assert (off_by <= (cols + 8) * 2.0 ** -24 * np.abs(full).sum(1)).all()
    assert not dw.cpu().numpy().reshape(-1)[~on].any()


def test_gradients_against_differences():
    """The loss sum(dy * combine(rows, weight)) is linear in every row value and every weight,
    so a difference quotient with any step is the derivative, up to binary32 rounding."""
    rng = np.random.default_rng(21)
    tokens, topk, experts, cols = 6, 3, 5, 40
    off, src, pos, off_d, pos_d = order(rng, tokens, topk, experts, 0.2)
    kept = int(off[-1])
    rows = rng.standard_normal((len(src), cols)).astype(np.float32)
    weight = rng.standard_normal((tokens, topk)).astype(np.float32)
    x = rng.standard_normal((tokens, cols)).astype(np.float32)
    dy = rng.standard_normal((tokens, cols)).astype(np.float32)
    t = lambda a: torch.from_numpy(np.array(a)).to(DEV)  # noqa: E731

    def combine(r, w):
        y = torch.empty((tokens, cols), device=DEV)
        bq.bq_moe_combine_f32(t(r), pos_d, off_d, y, weight=t(w), topk=topk)
        return y.double().cpu().numpy()

    drows, dw = torch.empty((len(src), cols), device=DEV), torch.empty((tokens, topk), device=DEV)
    bq.bq_moe_combine_bwd_f32(t(dy), t(rows), pos_d, off_d, t(weight), drows, dw)
    sync()
    # |sums| stay below 2^5 here, so a quotient is off by at most 2 * 2^5 * 2^-24 per output
    # column times |dy| < 8 and cols columns, over the step of 1
    tol = 2 * 2 ** 5 * 2.0 ** -24 * 8 * cols
    for p in range(len(src)):
        c = int(rng.integers(cols))
        hi, lo = rows.copy(), rows.copy()
        hi[p, c] += 0.5
        lo[p, c] -= 0.5
        step = float(hi[p, c]) - float(lo[p, c])
        num = ((combine(hi, weight) - combine(lo, weight)) * dy).sum() / step
        assert abs(num - drows[p, c].item()) <= tol, p
        if p >= kept:
            assert num == 0.0
    for a in range(tokens):
        for b in range(topk):
            hi, lo = weight.copy(), weight.copy()
            hi[a, b] += 0.5
            lo[a, b] -= 0.5
            step = float(hi[a, b]) - float(lo[a, b])
            num = ((combine(rows, hi) - combine(rows, lo)) * dy).sum() / step
            assert abs(num - dw[a, b].item()) <= tol, (a, b)

    # gather's gradient is the combine without weights
    g = rng.standard_normal((len(src), cols)).astype(np.float32)
    dx = torch.empty((tokens, cols), device=DEV)
    bq.bq_moe_combine_f32(t(g), pos_d, off_d, dx, topk=topk)

    def gather(v):
        out = torch.empty((len(src), cols), device=DEV)
        bq.bq_moe_gather(t(v), pos_d, off_d, out, topk=topk)
        return out.double().cpu().numpy()

    for a in range(tokens):
        c = int(rng.integers(cols))
        hi, lo = x.copy(), x.copy()
        hi[a, c] += 0.5
        lo[a, c] -= 0.5
        step = float(hi[a, c]) - float(lo[a, c])
        num = ((gather(hi) - gather(lo)) * g).sum() / step
        assert abs(num - dx[a, c].item()) <= tol, a


def test_positions_out_of_range_are_skipped():
    """Rows past the arrays' ends are neither read nor written."""
    x = torch.ones((2, 16), device=DEV)
    off = torch.tensor([0, 1 << 30], dtype=torch.int32, device=DEV)
    pos = torch.tensor([1 << 29, 0, -5, 2], dtype=torch.int32, device=DEV)
    out = torch.full((6, 16), 9.0, device=DEV)
    bq.bq_moe_gather(x, pos, off, out[:4], topk=2)
    y = torch.full((2, 16), 9.0, device=DEV)
    bq.bq_moe_combine_f32(out[:4], pos, off, y, topk=2)
    dw = torch.full((2, 2), 9.0, device=DEV)
    dr = torch.full((6, 16), 9.0, device=DEV)
    bq.bq_moe_combine_bwd_f32(x, out[:4], pos, off, torch.ones((2, 2), device=DEV), dr[:4], dw)
    sync()
    assert out[:, 0].tolist() == [1.0, 9.0, 1.0, 9.0, 9.0, 9.0]
    assert y[:, 0].tolist() == [1.0, 1.0]
    assert dw.tolist() == [[0.0, 16.0], [0.0, 16.0]]
    assert dr[:, 0].tolist() == [1.0, 9.0, 1.0, 9.0, 9.0, 9.0]


def test_rows_past_32_bit_offsets():
    """Sorted rows of more than 2^31 values: out and back."""
    tokens, topk, cols = 9000, 4, 65536 + 8
    assert tokens * topk * cols > 2 ** 31
    say(f"moe_gather {tokens * topk} rows of {cols}")
    ids = np.tile(np.arange(topk, dtype=np.int32)[::-1], (tokens, 1))
    off, src, pos = sort_on_gpu(np.ascontiguousarray(ids), topk)
    x = torch.arange(tokens, device=DEV, dtype=torch.float32)[:, None].remainder(97).to(
        torch.float16).expand(tokens, cols).contiguous()
    out = torch.empty((tokens * topk, cols), dtype=torch.float16, device=DEV)
    bq.bq_moe_gather(x, pos, off, out, topk=topk)
    y = torch.empty_like(x)
    bq.bq_moe_combine_f16(out, pos, off, y, topk=topk)
    sync()
    assert torch.equal(out[-tokens:], x) and torch.equal(y, x * 4)
    del y
    dw = torch.empty((tokens, topk), device=DEV)
    drows = torch.empty_like(out)
    w = torch.full((tokens, topk), 0.5, device=DEV)
    bq.bq_moe_combine_bwd_f16(torch.ones_like(x), out, pos, off, w, drows, dw)
    sync()
    assert bool((drows == 0.5).all())
    assert torch.equal(dw[:97], (torch.arange(97, device=DEV).float() * cols)[:, None].expand(97, 4))


def test_the_layer_in_a_captured_graph_and_on_another_stream():
    """sort, gather, combine and its gradient captured once and replayed: every replay equals
    the eager calls, with new choices copied in between."""
    rng = np.random.default_rng(31)
    tokens, topk, experts, cols = 2100, 4, 16, 320     # two sort blocks
    x = torch.from_numpy(rng.standard_normal((tokens, cols))).to(torch.bfloat16).to(DEV)
    w = torch.rand((tokens, topk), device=DEV)
    ids = torch.zeros((tokens, topk), dtype=torch.int32, device=DEV)
    n = tokens * topk
    ws = torch.empty(bq.bq_moe_sort_ws_bytes(tokens, topk, experts), dtype=torch.uint8, device=DEV)

    def buffers():
        i = lambda k: torch.zeros(k, dtype=torch.int32, device=DEV)  # noqa: E731
        r = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        return (i(experts + 1), i(n), i(n), r(n, cols), r(tokens, cols), r(n, cols),
                torch.zeros((tokens, topk), device=DEV))

    def layer(b):
        off, src, pos, out, y, drows, dw = b
        bq.bq_moe_sort(ids, experts, off, src, pos, ws)
        bq.bq_moe_gather(x, pos, off, out, topk=topk)
        bq.bq_moe_combine(out, pos, off, y, weight=w, topk=topk)
        bq.bq_moe_combine_bwd(y, out, pos, off, w, drows, dw)

    eager, held = buffers(), buffers()
    layer(held)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(held)
    for k in range(4):
        ids.copy_(torch.from_numpy(choices(rng, tokens, topk, experts, 0.1)))
        graph.replay()
        sync()
        layer(eager)
        sync()
        assert all(torch.equal(a, b) for a, b in zip(eager, held)), k
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        layer(held)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, held))
