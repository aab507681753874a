"""The C ABI of the expert layer on the host: include/blockq_moe.h is plain C, every entry
point is exported, and every invalid argument is refused with its status before a launch.

No call here reaches a kernel; the addresses are never dereferenced.
"""
from __future__ import annotations

import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

from block_quantized_wire_amd import build as _build  # noqa: E402

if _build.stale():
    _build.build()

import block_quantized_wire_amd as bq  # noqa: E402

# every call below passes fake device addresses; see tests/test_abi_host.py
import torch  # noqa: E402

if torch.cuda.device_count() > 0:
    pytest.skip("host-only ABI tests run where no GPU is visible", allow_module_level=True)

L = bq.lib
OK, NULL, SIZE, ALIGN, BOUNDS, NSRC, ALIAS, LAUNCH, SCRATCH = range(9)
A = 1 << 40


def at(i):
    """The i-th of many far apart, aligned fake addresses."""
    return A + (i << 32)


class Call:
    """An entry point with a set of valid named arguments, some replaced per case."""

    def __init__(self, name, **args):
        self.fn, self.args = getattr(L, name), args

    def __call__(self, **new):
        assert not set(new) - set(self.args)
        return self.fn(*{**self.args, **new}.values())


QUANT = dict(x=at(1), rows=8, cols=256, ldx=256, group=64, c=at(2), ldc=128, scale=at(3), lds=4,
             stream=0)
DEQUANT = dict(c=at(2), ldc=128, scale=at(3), lds=4, zero=at(4), ldz=4, rows=8, cols=256, group=64,
               y=at(5), ldy=256, stream=0)
MM = dict(x=at(1), ldx=256, c=at(2), ldc=128, scale=at(3), lds=4, zero=at(4), ldz=4, M=3, N=8,
          K=256, group=64, y=at(5), ldy=8, stream=0)
MOE_MM = dict(x=at(1), ldx=256, x_rows=6, src=at(6), topk=2, off=at(7), experts=4, rows=12,
              c=at(2), ldc=128, stride_c=1024, scale=at(3), lds=4, stride_s=32, zero=at(4), ldz=4,
              stride_z=32, N=8, K=256, group=64, y=at(5), ldy=8, stream=0)
SORT = dict(expert=at(1), tokens=10000, topk=2, experts=8, off=at(2), src=at(3), pos=at(4),
            ws=at(5), ws_bytes=1024 * 9, stream=0)
GATHER = dict(x=at(1), ldx=32, pos=at(2), off=at(3), tokens=5, topk=2, experts=4, cols=31, esize=2,
              out=at(4), ldo=32, stream=0)
COMBINE = dict(rows=at(1), ldr=32, pos=at(2), off=at(3), weight=at(5), tokens=5, topk=2, experts=4,
               cols=31, y=at(4), ldy=32, stream=0)
BWD = dict(dy=at(1), lddy=32, rows=at(2), ldr=32, pos=at(3), off=at(4), weight=at(5), tokens=5,
           topk=2, experts=4, cols=31, drows=at(6), lddr=32, dweight=at(7), stream=0)


def refuse(call, status, **new):
    assert call(**new) == status, new


def header_text():
    return open(os.path.join(ROOT, "include", "blockq_moe.h")).read()


def test_every_declared_entry_point_is_exported_and_bound():
    names = set(re.findall(r"\b(bq_[a-z0-9_]+)\s*\(", header_text())) - {"bq_status"}
    assert len(names) == 17
    for name in names:
        assert hasattr(L, name), name
        assert callable(getattr(bq, name)), name
        assert name in bq.__all__, name


@pytest.mark.parametrize("lang", ["c99", "c++17"])
def test_header_is_plain_c(tmp_path, lang):
    src = tmp_path / ("p.c" if lang == "c99" else "p.cpp")
    src.write_text('#include "blockq_moe.h"\n'
                   "int main(void) { return bq_moe_sort_ws_bytes(9000, 1, 4) == 5120 ? 0 : 1; }\n")
    cc = ["gcc", "-std=c99", "-pedantic"] if lang == "c99" else ["g++", "-std=c++17"]
    libdir = os.path.dirname(bq.LIB_PATH)
    exe = tmp_path / "p"
    subprocess.run(cc + ["-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                         "-o", str(exe), f"-L{libdir}", "-lblockq", f"-Wl,-rpath,{libdir}"],
                   check=True, timeout=300)
    assert subprocess.run([str(exe)], timeout=300).returncode == 0


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_codec_refusals(suffix):
    q, d = Call("bq_quant_i4" + suffix, **QUANT), Call("bq_dequant_i4" + suffix, **DEQUANT)
    for call in (q, d):
        for bad in (dict(group=16), dict(group=0), dict(group=256), dict(cols=96), dict(rows=-1),
                    dict(cols=-64), dict(rows=1 << 31, cols=64)):
            refuse(call, SIZE, **bad)
        refuse(call, OK, rows=0)
        refuse(call, OK, cols=0)
        for bad in (dict(c=None), dict(scale=None)):
            refuse(call, NULL, **bad)
        for bad in (dict(ldc=112), dict(lds=3), dict(ldc=1 << 46)):
            refuse(call, BOUNDS, **bad)
        for bad in (dict(c=at(2) + 8), dict(ldc=136), dict(scale=at(3) + 4), dict(lds=6)):
            refuse(call, ALIGN, **bad)
    refuse(q, NULL, x=None)
    refuse(q, BOUNDS, ldx=248)
    refuse(q, ALIGN, x=at(1) + 2)
    refuse(q, ALIGN, ldx=260)
    refuse(q, ALIAS, c=at(1) + 256)
    refuse(q, ALIAS, scale=at(1) + 64)
    refuse(q, ALIAS, scale=at(2) + 64)
    refuse(d, NULL, y=None)
    refuse(d, BOUNDS, ldz=2)
    refuse(d, BOUNDS, ldy=128)
    refuse(d, ALIGN, zero=at(4) + 1)
    refuse(d, ALIGN, ldz=6)
    refuse(d, ALIGN, y=at(5) + 8)
    for k in ("c", "scale", "zero"):
        refuse(d, ALIAS, y=DEQUANT[k])


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_product_refusals(suffix):
    for call, base in ((Call("bq_mm_i4" + suffix, **MM), MM),
                       (Call("bq_moe_mm_i4" + suffix, **MOE_MM), MOE_MM)):
        for bad in (dict(K=0), dict(K=-64), dict(K=96), dict(N=-1), dict(group=48),
                    dict(N=(1 << 26) + 1), dict(K=(1 << 30) + 64)):
            refuse(call, SIZE, **bad)
        refuse(call, OK, N=0)
        for k in ("x", "c", "scale", "y"):
            refuse(call, NULL, **{k: None})
        for bad in (dict(ldx=248), dict(ldc=112), dict(lds=3), dict(ldz=3), dict(ldy=7),
                    dict(ldx=1 << 48), dict(ldy=1 << 48)):
            refuse(call, BOUNDS, **bad)
        for bad in (dict(x=at(1) + 8), dict(ldx=260), dict(c=at(2) + 4), dict(ldc=136),
                    dict(scale=at(3) + 4), dict(lds=5), dict(zero=at(4) + 2), dict(ldz=5),
                    dict(y=at(5) + 1)):
            refuse(call, ALIGN, **bad)
        for k in ("x", "c", "scale", "zero"):
            refuse(call, ALIAS, y=base[k])
    mm = Call("bq_mm_i4" + suffix, **MM)
    refuse(mm, OK, M=0)
    refuse(mm, SIZE, M=-1)
    refuse(mm, SIZE, M=(1 << 30) + 1)


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_expert_product_refusals(suffix):
    call = Call("bq_moe_mm_i4" + suffix, **MOE_MM)
    for bad in (dict(experts=0), dict(experts=1025), dict(topk=0), dict(topk=65)):
        refuse(call, NSRC, **bad)
    for bad in (dict(rows=-1), dict(x_rows=-1), dict(rows=1 << 30), dict(x_rows=(1 << 30) + 1)):
        refuse(call, SIZE, **bad)
    refuse(call, OK, rows=0)
    refuse(call, NULL, off=None)
    refuse(call, BOUNDS, src=None)                      # 12 rows of y, 6 of x
    refuse(call, BOUNDS, stride_c=1008)
    refuse(call, BOUNDS, stride_s=28)
    refuse(call, BOUNDS, stride_z=28)
    refuse(call, BOUNDS, stride_c=1 << 47)
    refuse(call, ALIGN, stride_c=1032)
    refuse(call, ALIGN, stride_s=34)
    refuse(call, ALIGN, stride_z=34)
    refuse(call, ALIGN, off=at(7) + 2)
    refuse(call, ALIGN, src=at(6) + 2)
    refuse(call, ALIAS, y=at(6))
    refuse(call, ALIAS, y=at(7))
    refuse(call, ALIAS, y=at(2) + 3 * 1024)             # the last expert's codes


def test_sort_refusals():
    call = Call("bq_moe_sort", **SORT)
    for bad in (dict(topk=0), dict(topk=65), dict(experts=0), dict(experts=1025)):
        refuse(call, NSRC, **bad)
    for bad in (dict(tokens=-1), dict(tokens=1 << 29)):
        refuse(call, SIZE, **bad)
    for k in ("expert", "off", "src", "pos"):
        refuse(call, NULL, **{k: None})
    refuse(call, NULL, tokens=0, off=None)
    refuse(call, SCRATCH, ws=None)
    refuse(call, SCRATCH, ws_bytes=1024 * 9 - 1)
    for k in ("expert", "off", "src", "pos", "ws"):
        refuse(call, ALIGN, **{k: SORT[k] + 2})
    for k in ("off", "src", "pos", "ws"):
        refuse(call, ALIAS, **{k: SORT["expert"] + 400})
    refuse(call, ALIAS, src=at(4))
    assert bq.bq_moe_sort_ws_bytes(4096, 1, 8) == 0
    assert bq.bq_moe_sort_ws_bytes(512, 8, 1024) == 0
    assert bq.bq_moe_sort_ws_bytes(4097, 1, 8) == 1024 * 9
    for bad in ((-1, 1, 8), (1, 0, 8), (1, 1, 0), (1, 65, 8), (1, 1, 1025), (1 << 30, 1, 8)):
        assert bq.bq_moe_sort_ws_bytes(*bad) == -1


def test_gather_refusals():
    call = Call("bq_moe_gather", **GATHER)
    for bad in (dict(topk=0), dict(experts=0), dict(topk=65), dict(experts=1025)):
        refuse(call, NSRC, **bad)
    for bad in (dict(tokens=-1), dict(cols=-1), dict(esize=1), dict(esize=8), dict(tokens=1 << 29)):
        refuse(call, SIZE, **bad)
    refuse(call, OK, tokens=0)
    refuse(call, OK, cols=0)
    for k in ("x", "pos", "off", "out"):
        refuse(call, NULL, **{k: None})
    for bad in (dict(ldx=30), dict(ldo=30), dict(ldx=1 << 47), dict(ldo=1 << 47)):
        refuse(call, BOUNDS, **bad)
    for k in ("x", "out"):
        refuse(call, ALIGN, **{k: GATHER[k] + 1})
        refuse(call, ALIGN, esize=4, **{k: GATHER[k] + 2})
    for k in ("pos", "off"):
        refuse(call, ALIGN, **{k: GATHER[k] + 2})
    for k in ("x", "pos", "off"):
        refuse(call, ALIAS, out=GATHER[k])


@pytest.mark.parametrize("suffix", ["", "_f16", "_f32"])
def test_combine_refusals(suffix):
    size = 4 if suffix == "_f32" else 2
    fwd, bwd = Call("bq_moe_combine" + suffix, **COMBINE), Call("bq_moe_combine_bwd" + suffix, **BWD)
    for call in (fwd, bwd):
        for bad in (dict(topk=0), dict(experts=0), dict(topk=65), dict(experts=1025)):
            refuse(call, NSRC, **bad)
        for bad in (dict(tokens=-1), dict(cols=-1), dict(tokens=1 << 29)):
            refuse(call, SIZE, **bad)
        refuse(call, OK, tokens=0)
        for k in ("rows", "pos", "off"):
            refuse(call, NULL, **{k: None})
        refuse(call, BOUNDS, ldr=30)
        for k in ("pos", "off", "weight"):
            refuse(call, ALIGN, **{k: call.args[k] + 2})
        refuse(call, ALIGN, rows=call.args["rows"] + size // 2)
    refuse(fwd, OK, cols=0)
    refuse(fwd, NULL, y=None)
    refuse(fwd, BOUNDS, ldy=30)
    for k in ("rows", "pos", "off", "weight"):
        refuse(fwd, ALIAS, y=COMBINE[k])
    for k in ("dy", "weight", "drows", "dweight"):
        refuse(bwd, NULL, **{k: None})
    refuse(bwd, BOUNDS, lddy=30)
    refuse(bwd, BOUNDS, lddr=30)
    refuse(bwd, ALIGN, dweight=at(7) + 2)
    for k in ("dy", "rows", "pos", "off", "weight", "dweight"):
        refuse(bwd, ALIAS, drows=BWD[k])
    refuse(bwd, ALIAS, dweight=at(5))
