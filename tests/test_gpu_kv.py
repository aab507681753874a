"""Rows into the 4-bit cache and back on the GPU, against the plain forms of kv_ref: codes, scales
and rows bit for bit, and nothing else of the cache changed."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_ref as ref
from gpu_util import DEV, say, sync

from block_quantized_wire_amd import build as _build

if _build.stale():
    _build.build()
import block_quantized_wire_amd as bq  # noqa: E402

pytestmark = pytest.mark.gpu

WRITE = {"bf16": bq.bq_kv_write_i4, "f16": bq.bq_kv_write_i4_f16}
READ = {"bf16": bq.bq_kv_read_i4, "f16": bq.bq_kv_read_i4_f16}
WIDTHS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


def on_gpu(pool, heads_outer=False, gap=0):
    """The pool's arrays on the GPU; gap: entries of another use between the pages."""
    p, h, s, d, g = pool.pages, pool.heads, pool.page, pool.dim, pool.group
    parts = []
    for which in (0, 1):
        codes = torch.from_numpy(pool.codes[which]).view(p, h, s, d // 2)
        scales = pool.scales[which]
        for t in (codes, scales):
            order = (1, 0) if heads_outer else (0, 1)
            size = [t.shape[i] for i in order] + list(t.shape[2:])
            size[1] += gap
            room = torch.full(size, 77, dtype=t.dtype, device=DEV)
            view = room[:, :size[1] - gap]
            view = view.transpose(0, 1) if heads_outer else view
            view.copy_(t.to(DEV))
            parts.append(view)
    return bq.KvI4(parts[0], parts[2], parts[1], parts[3], group=g)


def same_bits(a, b):
    """Equal bit for bit, but for which NaN a NaN is."""
    a, b = a.cpu(), b.cpu()
    assert a.shape == b.shape and a.dtype == b.dtype
    nan = torch.isnan(a) & torch.isnan(b)
    return bool(((a.view(torch.int16) == b.view(torch.int16)) | nan).all())


def check_pool(cache, pool):
    for which, (codes, scales) in enumerate(((cache.k, cache.ks), (cache.v, cache.vs))):
        got = codes.cpu().reshape(pool.codes[which].shape).numpy()
        assert np.array_equal(got, pool.codes[which])
        assert same_bits(scales, pool.scales[which])


def rows(rng, tokens, heads, dim, kind, extra=0):
    """Rows out of a wider projection: heads and tokens apart from each other."""
    x = torch.from_numpy(rng.normal(0, 1, (tokens, heads, dim + extra)).astype(np.float32))
    x[:, :, :: 17] *= 6
    return x.to(ref.TORCH[kind]).to(DEV)[:, :, :dim]


def store(rng, pool, cache, slots, kind, extra=8):
    k, v = (rows(rng, len(slots), pool.heads, pool.dim, kind, extra) for _ in "kv")
    WRITE[kind](k, v, torch.tensor(slots, dtype=torch.int32, device=DEV), cache)
    for which, x in enumerate((k, v)):
        codes, scale, least = ref.quantise(x.cpu(), pool.group, kind)
        for t, slot in enumerate(slots):
            if 0 <= slot < pool.pages * pool.page:
                pool.put(which, slot, codes[t], scale[t], least[t])


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim,group", WIDTHS)
def test_write_and_read(dim, group, kind):
    rng = np.random.default_rng([dim, group])
    for tokens, heads, page, gap, outer in ((1, 1, 8, 0, False), (7, 3, 24, 0, False), (8, 2, 8, 1, True),
                                            (9, 5, 16, 2, False), (131, 2, 64, 1, True), (1000, 3, 200, 0, False)):
        say(f"kv dim={dim} group={group} {kind} tokens={tokens} heads={heads} page={page} gap={gap} {outer}")
        pool = ref.Pool(-(-tokens // page) + 3, heads, page, dim, group, kind)
        cache = on_gpu(pool, outer, gap)
        slots = rng.permutation(pool.pages * page)[:tokens]
        if tokens > 100:        # as a prefill writes them: runs of tokens, pages in any order
            order = rng.permutation(pool.pages)
            at = np.arange(tokens) + 5
            slots = order[at // page] * page + at % page
        slots = slots.astype(np.int64)
        slots[rng.random(tokens) < 0.1] = rng.choice([-1, -(1 << 31), pool.pages * page, (1 << 31) - 1])
        store(rng, pool, cache, slots.tolist(), kind)
        sync()
        check_pool(cache, pool)
        want = [ref.read(pool, w, slots) for w in (0, 1)]
        wide = torch.full((tokens, 2 * heads, dim), 5.0, dtype=ref.TORCH[kind], device=DEV)
        READ[kind](cache, torch.from_numpy(slots).to(torch.int32).to(DEV), wide[:, :heads], wide[:, heads:])
        sync()
        assert same_bits(wide[:, :heads], want[0]) and same_bits(wide[:, heads:], want[1])


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_read_names_a_slot_many_times(kind):
    rng = np.random.default_rng(3)
    pool = ref.Pool(4, 2, 16, 128, 64, kind).random(rng)
    cache = on_gpu(pool)
    slots = np.array([5] * 9 + [63, 0, 64, -1, 5], np.int32)
    k, v = (torch.empty((len(slots), 2, 128), dtype=ref.TORCH[kind], device=DEV) for _ in "kv")
    READ[kind](cache, torch.from_numpy(slots).to(DEV), k, v)
    sync()
    assert same_bits(k, ref.read(pool, 0, slots)) and same_bits(v, ref.read(pool, 1, slots))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_groups_that_are_special(kind):
    """Constants, zeros of both signs, subnormal and the largest ranges, NaN and infinities."""
    dim, group, t = 128, 32, ref.TORCH[kind]
    info = torch.finfo(t)
    x = torch.zeros((8, 1, dim), dtype=torch.float64)
    x[0] = 3.25
    x[1, 0, 1::2] = -0.0
    x[2] = torch.arange(dim) * (info.smallest_normal / 64)
    x[3, 0, ::2], x[3, 0, 1::2] = info.max, -info.max
    x[4] = torch.arange(dim) % 15
    x[4, 0, 3], x[4, 0, 40], x[4, 0, 70] = float("nan"), float("inf"), -float("inf")
    x[5] = -1000.0
    x[5, 0, 7] = -1000.0 - info.eps * 1024
    x[6] = torch.arange(dim).repeat_interleave(1) / 2 % 15     # ties: codes of k + 1/2
    x[7, 0, 5] = info.tiny / 2
    pool = ref.Pool(1, 1, 8, dim, group, kind)
    cache = on_gpu(pool)
    k = x.to(t).to(DEV)
    v = k.flip(0).contiguous()
    slots = torch.arange(8, dtype=torch.int32, device=DEV)
    WRITE[kind](k, v, slots, cache)
    for which, y in enumerate((k, v)):
        codes, scale, least = ref.quantise(y.cpu(), group, kind)
        for i in range(8):
            pool.put(which, i, codes[i], scale[i], least[i])
    sync()
    check_pool(cache, pool)
    back = [torch.empty_like(k) for _ in "kv"]
    READ[kind](cache, slots, *back)
    sync()
    for which in (0, 1):
        want = ref.read(pool, which, range(8))
        assert same_bits(back[which], want)
    assert torch.equal(back[0][0], k[0])                    # constants come back as they are
    nan = torch.isnan(back[0][4, 0]).view(4, 32).all(1).tolist()
    assert nan == [True, True, True, False]                # the groups with them, and no other
    assert not torch.isnan(back[0][[0, 1, 2, 5, 6, 7]]).any()


@pytest.mark.parametrize("dim,group,kind", [(64, 64, "f16"), (128, 32, "bf16"), (256, 128, "bf16")])
def test_distance_of_what_comes_back(dim, group, kind):
    """Half a step of the codes, and the roundings of the scale and of the result."""
    rng = np.random.default_rng(dim)
    x = rows(rng, 300, 3, dim, kind)
    pool = ref.Pool(40, 3, 8, dim, group, kind)
    cache = on_gpu(pool)
    slots = torch.from_numpy(rng.permutation(320)[:300].astype(np.int32)).to(DEV)
    WRITE[kind](x, x, slots, cache)
    k, v = (torch.empty((300, 3, dim), dtype=x.dtype, device=DEV) for _ in "kv")
    READ[kind](cache, slots, k, v)
    sync()
    assert torch.equal(k, v)
    a = x.cpu().double().numpy().reshape(300, 3, -1, group)
    span = (a.max(-1) - a.min(-1))[..., None]
    step = span / 15 * (1 + ref.HALF[kind])
    far = np.abs(k.cpu().double().numpy().reshape(a.shape) - a)
    # the top code falls short of the largest value, or passes it, by 15 roundings of the scale
    assert (far <= step * (0.5 + 15 * ref.HALF[kind]) + np.abs(a) * ref.HALF[kind] * 2 + span * 2.0 ** -8).all()


def test_rows_of_one_token_for_all_heads():
    """Strides of zero: one row of keys for every head, one token for every slot."""
    pool = ref.Pool(2, 4, 8, 64, 32, "bf16")
    cache = on_gpu(pool)
    row = rows(np.random.default_rng(1), 1, 1, 64, "bf16", 8)
    k = row.expand(5, 4, 64)
    slots = [3, 9, 0, 15, 8]
    WRITE["bf16"](k, k, torch.tensor(slots, dtype=torch.int32, device=DEV), cache)
    codes, scale, least = ref.quantise(k.cpu(), 32, "bf16")
    for which in (0, 1):
        for t, slot in enumerate(slots):
            pool.put(which, slot, codes[t], scale[t], least[t])
    sync()
    check_pool(cache, pool)


def test_no_tokens_and_another_stream():
    rng = np.random.default_rng(2)
    pool = ref.Pool(2, 2, 8, 64, 64, "f16")
    cache = on_gpu(pool)
    empty = torch.empty((0, 2, 64), dtype=torch.float16, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    WRITE["f16"](empty, empty, none, cache)
    READ["f16"](cache, none, empty, empty.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        store(rng, pool, cache, [0, 8, 3], "f16")
    side.synchronize()
    check_pool(cache, pool)


def test_pool_beyond_32_bit_offsets():
    """Pages more than 2^32 bytes apart, for codes and for scales."""
    rng = np.random.default_rng(4)
    dim, group, page = 128, 32, 8
    pool = ref.Pool(3, 2, page, dim, group, "bf16")
    say("kv pool of 3 pages 2.5 GiB apart")
    far = 5 << 29                                   # bytes between pages
    parts = []
    for which in (0, 1):
        codes = torch.empty(2 * far + (1 << 20), dtype=torch.uint8, device=DEV)
        scale = torch.empty(2 * far // 2 + (1 << 20), dtype=torch.bfloat16, device=DEV)
        ck = codes.as_strided((3, 2, page, dim // 2), (far, page * dim // 2, dim // 2, 1))
        sk = scale.as_strided((3, 2, dim // group, page, 2), (far // 2, dim // group * page * 2, 2 * page, 2, 1))
        ck.copy_(torch.from_numpy(pool.codes[which]).view(3, 2, page, dim // 2).to(DEV))
        sk.copy_(pool.scales[which].to(DEV))
        parts += [ck, sk]
    cache = bq.KvI4(parts[0], parts[2], parts[1], parts[3], group=group)
    slots = [23, 0, 17, 9, 8]
    store(rng, pool, cache, slots, "bf16")
    sync()
    check_pool(cache, pool)
    k, v = (torch.empty((5, 2, dim), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    READ["bf16"](cache, torch.tensor(slots, dtype=torch.int32, device=DEV), k, v)
    sync()
    assert same_bits(k, ref.read(pool, 0, slots)) and same_bits(v, ref.read(pool, 1, slots))


def test_captured_write_and_read():
    rng = np.random.default_rng(6)
    pool = ref.Pool(3, 2, 16, 128, 128, "bf16")
    cache = on_gpu(pool)
    k, v = (rows(rng, 7, 2, 128, "bf16") for _ in "kv")
    slots = torch.zeros(7, dtype=torch.int32, device=DEV)
    back = [torch.zeros((7, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        WRITE["bf16"](k, v, slots, cache)
        READ["bf16"](cache, slots, *back)
    for turn in range(4):
        k.copy_(rows(rng, 7, 2, 128, "bf16"))
        v.copy_(rows(rng, 7, 2, 128, "bf16"))
        places = rng.permutation(48)[:7]
        slots.copy_(torch.from_numpy(places.astype(np.int32)))
        graph.replay()
        sync()
        for which, x in enumerate((k, v)):
            codes, scale, least = ref.quantise(x.cpu(), 128, "bf16")
            for t, slot in enumerate(places.tolist()):
                pool.put(which, slot, codes[t], scale[t], least[t])
        check_pool(cache, pool)
        for which in (0, 1):
            assert same_bits(back[which], ref.read(pool, which, places))
