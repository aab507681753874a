"""What the Python binding of the 4-bit cache refuses before it passes a pointer on: tensors of
another type, shape, layout, length or device than the cache goes with.

The library behind it is a stand-in that records its arguments, so nothing is launched."""
from __future__ import annotations

import pytest
import torch

import block_quantized_wire_amd as bq

P, H, S, D, G = 6, 2, 16, 128, 64
I32, BF, F16 = torch.int32, torch.bfloat16, torch.float16


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    recorder = Recorder()
    bq._L()
    monkeypatch.setattr(bq, "_lib", recorder)
    monkeypatch.setattr(bq, "_raw_device", lambda: -1)      # tensors on the host stand for the GPU's
    return recorder


def arrays(dtype=BF, **new):
    a = dict(k=torch.zeros((P, H, S, D // 2), dtype=torch.uint8), v=torch.zeros((P, H, S, D // 2), dtype=torch.uint8),
             ks=torch.zeros((P, H, D // G, S, 2), dtype=dtype), vs=torch.zeros((P, H, D // G, S, 2), dtype=dtype))
    return {**a, **new}


def cache(dtype=BF):
    return bq.KvI4(**arrays(dtype), group=G)


def test_description_of_a_cache(lib):
    a = arrays()
    c = bq.KvI4(**a, group=G)
    s = c.struct
    assert (s.k, s.v, s.ks, s.vs) == tuple(a[n].data_ptr() for n in ("k", "v", "ks", "vs"))
    assert (s.page_stride, s.head_stride) == (H * S * D // 2, S * D // 2)
    assert (s.spage_stride, s.shead_stride) == (H * (D // G) * S * 2, (D // G) * S * 2)
    assert (s.pages, s.page_size, s.heads, s.dim, s.group) == (P, S, H, D, G)
    turned = {n: t.transpose(0, 1).contiguous().transpose(0, 1) for n, t in a.items()}
    s = bq.KvI4(**turned, group=G).struct
    assert (s.page_stride, s.head_stride) == (S * D // 2, P * S * D // 2)


def test_caches_that_are_refused(lib):
    for bad in (dict(k=torch.zeros((P, H, S, D // 2), dtype=torch.int8)), dict(v=torch.zeros((P, H, S, D // 2))),
                dict(ks=torch.zeros((P, H, D // G, S, 2))), dict(vs=torch.zeros((P, H, D // G, S, 2), dtype=F16)),
                dict(ks=torch.zeros((P, H, D // G, S, 2), dtype=torch.int16))):
        with pytest.raises(TypeError):
            bq.KvI4(**arrays(**bad), group=G)
    u8 = torch.uint8
    for bad in (dict(v=torch.zeros((P, H, S + 8, D // 2), dtype=u8)), dict(ks=torch.zeros((P, H, 1, S, 2), dtype=BF)),
                dict(vs=torch.zeros((P, H, 1, S, 2), dtype=BF)),
                dict(v=torch.zeros((P + 1, H, S, D // 2), dtype=u8)[1:].transpose(0, 1).contiguous().transpose(0, 1)),
                dict(k=torch.zeros((P, H, S, D), dtype=u8)[..., ::2], v=torch.zeros((P, H, S, D), dtype=u8)[..., ::2]),
                dict(k=torch.zeros((P, H, S, D), dtype=u8)[..., :D // 2],
                     v=torch.zeros((P, H, S, D), dtype=u8)[..., :D // 2]),
                dict(ks=torch.zeros((P, H, D // G, S, 4), dtype=BF)[..., :2],
                     vs=torch.zeros((P, H, D // G, S, 4), dtype=BF)[..., :2]),
                dict(k=torch.zeros((P, H, S, D // 2), dtype=u8, device="meta")),
                dict(ks=torch.zeros((P, H, D // G, S, 2), dtype=BF, device="meta"))):
        with pytest.raises(ValueError):
            bq.KvI4(**arrays(**bad), group=G)
    for group in (0, -64, 32, 128, 48):
        with pytest.raises(ValueError):
            bq.KvI4(**arrays(), group=group)


def rows(n=5, dtype=BF):
    return torch.zeros((n, H, D), dtype=dtype)


@pytest.mark.parametrize("name", ["bq_kv_write_i4", "bq_kv_read_i4"])
def test_rows(lib, name):
    def call(k, v, slots, c, suffix=""):
        f = getattr(bq, name + suffix)
        return f(k, v, slots, c, stream=0) if "write" in name else f(c, slots, k, v, stream=0)
    slots = torch.zeros(5, dtype=I32)
    c = cache()
    wide = torch.zeros((5, 3 * H, D + 8), dtype=BF)
    k, v = wide[:, :H, :D], wide[:, H:2 * H, :D]
    call(k, v, slots, c)
    fn, args = lib.calls.pop()
    assert fn == name
    want = [k.data_ptr(), 3 * H * (D + 8), D + 8, v.data_ptr(), 3 * H * (D + 8), D + 8]
    if "write" in name:
        assert list(args) == want + [slots.data_ptr(), 5, c.address, 0]
    else:
        assert list(args) == [c.address, slots.data_ptr(), 5] + want + [0]
    call(rows(dtype=F16), rows(dtype=F16), slots, cache(F16), "_f16")
    assert lib.calls.pop()[0] == name + "_f16"
    for bad in ((rows(dtype=F16), rows(), slots, c), (rows(), rows(dtype=torch.float32), slots, c),
                (rows(), rows(), slots.long(), c), (rows(dtype=F16), rows(dtype=F16), slots, c),
                (rows(), rows(), slots, cache(F16))):
        with pytest.raises(TypeError):
            call(*bad)
    with pytest.raises(TypeError):
        call(rows(), rows(), slots, c, "_f16")
    for bad in ((rows(4), rows(), slots, c), (rows(), rows(6), slots, c), (rows(), rows()[:, :1], slots, c),
                (rows(), torch.zeros((5, H, 2 * D), dtype=BF)[..., ::2], slots, c),
                (rows(), rows(), torch.zeros(10, dtype=I32)[::2], c)):
        with pytest.raises(ValueError):
            call(*bad)
    assert not lib.calls


def attn_args(**new):
    a = dict(q=torch.zeros((7, 4, D), dtype=BF), cache=cache(), table=torch.zeros((3, 5), dtype=I32),
             lens=torch.zeros(3, dtype=I32), out=torch.zeros((7, 4, D), dtype=BF),
             starts=torch.zeros(4, dtype=I32), max_q=4, lse=torch.zeros((7, 4)),
             ws=torch.zeros(100), stream=0)
    return {**a, **new}


def test_attention_passes_on(lib):
    a = attn_args(window=9, causal=False)
    bq.bq_attn_i4(**a)
    fn, args = lib.calls.pop()
    assert fn == "bq_attn_i4"
    p = {n: t.data_ptr() for n, t in a.items() if isinstance(t, torch.Tensor)}
    assert list(args) == [p["q"], 4 * D, D, a["cache"].address, p["table"], 5, 5, p["lens"], p["starts"], 3, 7, 4,
                          5 * S, 4, False, 9, D ** -0.5, p["out"], 4 * D, D, p["lse"], p["ws"], 400, 0]
    part = torch.zeros((3, 9), dtype=I32)[:, 2:7]
    bq.bq_attn_i4(**attn_args(starts=None, max_q=None, table=part, lse=None, ws=None, max_len=33, scale=2.0,
                              q=torch.zeros((3, 4, D), dtype=BF), out=torch.zeros((3, 4, D), dtype=BF)))
    args = lib.calls.pop()[1]
    assert args[5:7] == (9, 5) and args[8] is None and args[11:13] == (1, 33) and args[16] == 2.0
    assert args[20:23] == (None, None, 0)


def test_attention_refusals(lib):
    z = torch.zeros
    for bad in (dict(q=z((7, 4, D), dtype=F16)), dict(out=z((7, 4, D))), dict(table=z((3, 5), dtype=torch.int64)),
                dict(lens=z(3, dtype=torch.int64)), dict(starts=z(4)), dict(lse=z((7, 4), dtype=BF)),
                dict(cache=cache(F16))):
        with pytest.raises(TypeError):
            bq.bq_attn_i4(**attn_args(**bad))
    with pytest.raises(TypeError):
        bq.bq_attn_i4_f16(**attn_args())
    for bad in (dict(q=z((7, 4, D // 2), dtype=BF)), dict(out=z((6, 4, D), dtype=BF)),
                dict(out=z((7, 2, D), dtype=BF)), dict(q=z((7, 4, 2 * D), dtype=BF)[..., ::2]),
                dict(table=z((3, 10), dtype=I32)[:, ::2]), dict(lens=z(2, dtype=I32)), dict(lens=z(4, dtype=I32)),
                dict(lens=z(6, dtype=I32)[::2]), dict(starts=z(3, dtype=I32)), dict(starts=z(5, dtype=I32)),
                dict(lse=z(27)), dict(lse=z((4, 7)).t()), dict(max_q=None), dict(ws=z(10, 10).t())):
        with pytest.raises(ValueError):
            bq.bq_attn_i4(**attn_args(**bad))
    assert not lib.calls


class There:
    """A tensor that says it is on another device."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return (lambda: 1) if name == "get_device" else getattr(self.t, name)


def test_tensors_on_another_device_than_the_cache(lib):
    slots, c = torch.zeros(5, dtype=I32), cache()
    for bad in ((There(rows()), rows(), slots), (rows(), There(rows()), slots), (rows(), rows(), There(slots))):
        with pytest.raises(ValueError):
            bq.bq_kv_write_i4(*bad, c, stream=0)
        with pytest.raises(ValueError):
            bq.bq_kv_read_i4(c, bad[2], bad[0], bad[1], stream=0)
    good = attn_args()
    for name in ("q", "table", "lens", "out", "starts", "lse", "ws"):
        with pytest.raises(ValueError):
            bq.bq_attn_i4(**attn_args(**{name: There(good[name])}))
    assert not lib.calls


def test_another_device_than_the_current_one(lib, monkeypatch):
    """The launch would go to the current device's stream."""
    c = cache()
    monkeypatch.setattr(bq, "_raw_device", lambda: 0)
    for call in (lambda: bq.bq_kv_write_i4(rows(), rows(), torch.zeros(5, dtype=I32), c, stream=0),
                 lambda: bq.bq_attn_i4(**attn_args(cache=c))):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert not lib.calls
