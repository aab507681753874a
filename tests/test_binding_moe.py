"""What the Python binding of the expert layer refuses before it passes a pointer on: index and
weight tensors of another type, a layout that is not the one documented, arrays shorter than
the call reads, and a count of choices that was left out where it is not 1.

The library behind it is a stand-in that records its arguments, so nothing is launched."""
from __future__ import annotations

import pytest
import torch

import block_quantized_wire_amd as bq


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
    bq._L()                       # whatever loading sets up
    monkeypatch.setattr(bq, "_lib", recorder)
    return recorder


T, K, E, H = 6, 4, 5, 16
I32, F32 = torch.int32, torch.float32
SUFFIX = {"": torch.bfloat16, "_f16": torch.float16, "_f32": torch.float32}


def ints(n):
    return torch.zeros(n, dtype=I32)


def sort_args():
    return dict(expert=torch.zeros((T, K), dtype=I32), experts=E, off=ints(E + 1), src=ints(T * K),
                pos=ints(T * K), stream=0)


def gather_args():
    return dict(x=torch.zeros(T, H), pos=ints(T * K), off=ints(E + 1), out=torch.zeros(T * K, H),
                topk=K, stream=0)


def combine_args(dtype=F32):
    return dict(rows=torch.zeros((T * K, H), dtype=dtype), pos=ints(T * K), off=ints(E + 1),
                y=torch.zeros((T, H), dtype=dtype), weight=torch.zeros(T, K), topk=K, stream=0)


def bwd_args(dtype=F32):
    return dict(dy=torch.zeros((T, H), dtype=dtype), rows=torch.zeros((T * K, H), dtype=dtype),
                pos=ints(T * K), off=ints(E + 1), weight=torch.zeros(T, K),
                drows=torch.zeros((T * K, H), dtype=dtype), dweight=torch.zeros(T, K), stream=0)


def mm_args(dtype=torch.bfloat16):
    return dict(x=torch.zeros((T, 64), dtype=dtype), off=ints(E + 1),
                c=torch.zeros((E, H, 32), dtype=torch.uint8), scale=torch.zeros((E, H, 4), dtype=dtype),
                y=torch.zeros((T * K, H), dtype=dtype), group=64, src=ints(T * K), topk=K, stream=0)


def calls():
    yield "bq_moe_sort", sort_args(), ("expert", "off", "src", "pos"), ()
    yield "bq_moe_gather", gather_args(), ("pos", "off"), ()
    for s, d in SUFFIX.items():
        yield "bq_moe_combine" + s, combine_args(d), ("pos", "off"), ("weight",)
        yield "bq_moe_combine_bwd" + s, bwd_args(d), ("pos", "off"), ("weight", "dweight")
    for s in ("", "_f16"):
        yield "bq_moe_mm_i4" + s, mm_args(SUFFIX[s]), ("off", "src"), ()


@pytest.mark.parametrize("name,args,ints32,floats", calls(), ids=lambda v: v if isinstance(v, str) else "")
def test_types_and_layouts(lib, name, args, ints32, floats):
    fn = getattr(bq, name)
    fn(**args)
    assert [n for n, _ in lib.calls] == [name]
    for arg in ints32 + floats:
        for dtype in (torch.int64, torch.int16, torch.bfloat16, torch.float64):
            with pytest.raises(TypeError, match=arg):
                fn(**{**args, arg: args[arg].to(dtype)})
        wide = torch.zeros(args[arg].shape + (2,), dtype=args[arg].dtype)[..., 0]
        with pytest.raises(ValueError, match=arg):
            fn(**{**args, arg: wide})
    for arg in floats:
        with pytest.raises(ValueError, match=arg):
            fn(**{**args, arg: torch.zeros(K, T).t()})
    assert len(lib.calls) == 1


def test_arrays_that_end_too_soon(lib):
    for fn, args, short in ((bq.bq_moe_sort, sort_args(), {"src": T * K - 1, "pos": T * K - 1, "off": E}),
                            (bq.bq_moe_gather, gather_args(), {"pos": T * K - 1}),
                            (bq.bq_moe_combine_f32, combine_args(), {"pos": T * K - 1, "weight": T * K - 1}),
                            (bq.bq_moe_combine_bwd_f32, bwd_args(), {"pos": T * K - 1, "dweight": T * K - 1})):
        for arg, n in short.items():
            with pytest.raises(ValueError, match=arg):
                fn(**{**args, arg: torch.zeros(n, dtype=args[arg].dtype)})
    assert not lib.calls


def test_a_count_of_choices_left_out(lib):
    """It is the weights' second size; without weights, or for sources, it may be left out only
    where every token has one slot."""
    args = combine_args()
    del args["topk"]
    bq.bq_moe_combine_f32(**args)
    assert lib.calls[-1][1][6] == K
    bq.bq_moe_combine_f32(**{**args, "weight": torch.zeros(T, 1)})
    assert lib.calls[-1][1][6] == 1
    for weight in (None, torch.zeros(T * K)):
        with pytest.raises(ValueError, match="topk"):
            bq.bq_moe_combine_f32(**{**args, "weight": weight})
    bq.bq_moe_combine_f32(**{**args, "weight": None, "pos": ints(T)})
    assert lib.calls[-1][1][6] == 1

    args = mm_args()
    del args["topk"]
    with pytest.raises(ValueError, match="topk"):
        bq.bq_moe_mm_i4(**args)
    bq.bq_moe_mm_i4(**{**args, "src": ints(T), "y": args["y"][:T]})
    assert lib.calls[-1][1][4] == 1
    bq.bq_moe_mm_i4(**{**args, "x": torch.zeros((T * K, 64), dtype=torch.bfloat16), "src": None})
    assert lib.calls[-1][1][3] is None
    bq.bq_moe_mm_i4(**{**mm_args(), "topk": 0})     # the library's to refuse
    assert lib.calls[-1][1][4] == 0


def test_what_was_taken_before_still_is(lib):
    """Weights as one row of slots, arrays longer than the call reads, a step without weights."""
    args = combine_args()
    bq.bq_moe_combine_f32(**{**args, "weight": torch.zeros(T * K)})
    bq.bq_moe_combine_f32(**{**args, "weight": torch.zeros(T * K, 1), "pos": ints(T * K + 9)})
    bq.bq_moe_combine_f32(**{**args, "weight": None})
    bq.bq_moe_gather(**{**gather_args(), "pos": ints(100)})
    bq.bq_moe_mm_i4(**{**mm_args(), "src": ints(100)})
    assert lib.calls[-1][1][7] == T * K
    # rows of y past the sources belong to no expert, and the sources are not read there
    bq.bq_moe_mm_i4(**{**mm_args(), "src": ints(K)})
    assert lib.calls[-1][1][7] == K
    bq.bq_moe_sort(**{**sort_args(), "src": ints(100), "pos": ints(100)})
    bq.bq_moe_sort(**{**sort_args(), "expert": torch.zeros((0, K), dtype=I32), "src": ints(0),
                      "pos": ints(0)})
    # addresses in place of the index and weight tensors
    bq.bq_moe_sort(**{**sort_args(), "off": 64, "src": 128, "pos": 192})
    bq.bq_moe_gather(**{**gather_args(), "pos": 64})
    bq.bq_moe_combine_f32(**{**combine_args(), "pos": 64, "weight": 128})
    assert lib.calls[-1][1][2] == 64 and lib.calls[-1][1][4] == 128
    bq.bq_moe_combine_bwd_f32(**{**bwd_args(), "pos": 64, "dweight": 128})
    args = mm_args()
    del args["topk"]
    bq.bq_moe_mm_i4(**{**args, "src": 64})
    assert lib.calls[-1][1][3:5] == (64, 1)
    with pytest.raises(TypeError, match="off"):
        bq.bq_moe_sort(**{**sort_args(), "src": 128, "off": torch.zeros(E + 1, dtype=torch.int64)})
    assert len(lib.calls) == 13
