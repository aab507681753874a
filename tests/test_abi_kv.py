"""The C ABI of the 4-bit cache on the host: include/blockq_kv.h is plain C, every entry point is
exported, and every invalid argument is refused with its status before a launch.

No call here reaches a kernel; the addresses are never dereferenced.
"""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

from block_quantized_wire_amd import build as _build  # noqa: E402

if _build.stale():
    _build.build()

import block_quantized_wire_amd as bq  # noqa: E402
import torch  # noqa: E402

if torch.cuda.device_count() > 0:
    pytest.skip("host-only ABI tests run where no GPU is visible", allow_module_level=True)

L = bq.lib
OK, NULL, SIZE, ALIGN, BOUNDS, NSRC, ALIAS, LAUNCH, SCRATCH = range(9)


def at(i):
    """The i-th of many far apart, aligned fake addresses."""
    return (1 << 40) + (i << 34)


POOL = dict(k=at(1), v=at(2), ks=at(3), vs=at(4), page_stride=2 * 16 * 64, head_stride=16 * 64,
            spage_stride=2 * 2 * 16 * 2, shead_stride=2 * 16 * 2, pages=10, page_size=16, heads=2, dim=128,
            group=64)
WRITE = dict(k=at(5), ldk=256, hsk=128, v=at(6), ldv=256, hsv=128, slot=at(7), tokens=9, cache=POOL, stream=0)
READ = dict(cache=POOL, slot=at(7), tokens=9, k=at(5), ldk=256, hsk=128, v=at(6), ldv=256, hsv=128, stream=0)
ATTN = dict(q=at(5), ldq=512, hsq=128, cache=POOL, table=at(6), ldt=8, table_cols=8, lens=at(7),
            starts=at(8), seqs=3, rows=7, max_q=4, max_len=128, heads=4, causal=1, window=0, scale=0.1,
            out=at(9), ldo=512, hso=128, lse=at(10), ws=at(11), ws_bytes=0, stream=0)


class Call:
    """An entry point with a set of valid named arguments; those of the pool by their own names, with
    a cache_ before them."""

    def __init__(self, name, args):
        self.fn, self.args = getattr(L, name), args

    def __call__(self, **new):
        pool = {**POOL, **{k[6:]: v for k, v in new.items() if k.startswith("cache_")}}
        args = {**self.args, **{k: v for k, v in new.items() if not k.startswith("cache_")}}
        assert set(args) == set(self.args) and set(pool) == set(POOL)
        if args["cache"] is POOL:
            struct = bq._KvI4(*pool.values())
            args["cache"] = ctypes.addressof(struct)
        return self.fn(*args.values())


def refuse(call, status, **new):
    assert call(**new) == status, new


def header_text():
    return open(os.path.join(ROOT, "include", "blockq_kv.h")).read()


def test_every_declared_entry_point_is_exported_and_bound():
    names = set(re.findall(r"\b(bq_[a-z0-9_]+)\(", header_text()))
    assert names == {"bq_kv_write_i4", "bq_kv_write_i4_f16", "bq_kv_read_i4", "bq_kv_read_i4_f16",
                     "bq_attn_i4", "bq_attn_i4_f16", "bq_attn_i4_ws_bytes"}
    for name in names:
        assert hasattr(L, name) and callable(getattr(bq, name)) and name in bq.__all__, name


@pytest.mark.parametrize("lang", ["c99", "c++17"])
def test_header_is_plain_c(tmp_path, lang):
    src = tmp_path / ("p.c" if lang == "c99" else "p.cpp")
    src.write_text('#include "blockq_kv.h"\n'
                   f"typedef char same_size[sizeof(bq_kv_i4) == {ctypes.sizeof(bq._KvI4)} ? 1 : -1];\n"
                   "int main(void) { same_size s; s[0] = 0;\n"
                   "  return s[0] + (bq_attn_i4_ws_bytes(1, 1, 1, 100, 8, 8, 128) == 0 ? 0 : 1); }\n")
    cc = ["gcc", "-std=c99", "-pedantic"] if lang == "c99" else ["g++", "-std=c++17"]
    libdir = os.path.dirname(bq.LIB_PATH)
    exe = tmp_path / "p"
    subprocess.run(cc + ["-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                         "-o", str(exe), f"-L{libdir}", "-lblockq", f"-Wl,-rpath,{libdir}"],
                   check=True, timeout=300)
    assert subprocess.run([str(exe)], timeout=300).returncode == 0


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_pools_that_are_refused(suffix):
    for name, args in (("bq_kv_write_i4", WRITE), ("bq_kv_read_i4", READ), ("bq_attn_i4", ATTN)):
        call = Call(name + suffix, args)
        refuse(call, NULL, cache=None)
        for bad in (dict(dim=32), dict(dim=96), dict(dim=512), dict(dim=0), dict(group=16), dict(group=256),
                    dict(group=0), dict(dim=64, group=128), dict(heads=0), dict(heads=-1), dict(heads=1025),
                    dict(pages=0), dict(pages=-1), dict(page_size=0), dict(page_size=-8), dict(page_size=12),
                    dict(page_size=4), dict(pages=1 << 27), dict(pages=1 << 30, page_size=1 << 30)):
            refuse(call, SIZE, **{"cache_" + k: v for k, v in bad.items()})
        for p in ("k", "v", "ks", "vs"):
            refuse(call, NULL, **{"cache_" + p: None})
            refuse(call, ALIGN, **{"cache_" + p: POOL[p] + 8})
        for bad in (dict(head_stride=1023), dict(head_stride=512), dict(page_stride=1024), dict(page_stride=0),
                    dict(head_stride=-1024), dict(page_stride=1 << 50), dict(spage_stride=64),
                    dict(shead_stride=32), dict(shead_stride=0), dict(spage_stride=-128),
                    dict(spage_stride=-(1 << 63)), dict(shead_stride=-(1 << 63)),
                    dict(spage_stride=1 << 62), dict(shead_stride=1 << 48), dict(page_stride=1 << 62)):
            refuse(call, BOUNDS, **{"cache_" + k: v for k, v in bad.items()})
        for bad in (dict(page_stride=2056), dict(head_stride=1032, page_stride=4096), dict(spage_stride=132),
                    dict(shead_stride=68, spage_stride=256)):
            refuse(call, ALIGN, **{"cache_" + k: v for k, v in bad.items()})


@pytest.mark.parametrize("suffix", ["", "_f16"])
@pytest.mark.parametrize("name,args", [("bq_kv_write_i4", WRITE), ("bq_kv_read_i4", READ)])
def test_row_refusals(name, args, suffix):
    call = Call(name + suffix, args)
    refuse(call, OK, tokens=0)
    refuse(call, OK, tokens=0, k=None, v=None, slot=None)
    refuse(call, SIZE, tokens=-1)
    refuse(call, SIZE, tokens=1 << 30)
    refuse(call, NULL, slot=None)
    refuse(call, ALIGN, slot=at(7) + 2)
    for x, ld, hs in (("k", "ldk", "hsk"), ("v", "ldv", "hsv")):
        refuse(call, NULL, **{x: None})
        for bad in ({x: args[x] + 8}, {ld: 260}, {hs: 132, ld: 512}):
            refuse(call, ALIGN, **bad)
        for bad in ({ld: -256}, {hs: -128}, {ld: 1 << 46}, {ld: 1 << 62}, {hs: 1 << 62}):
            refuse(call, BOUNDS, **bad)
        for cached in ("k", "v", "ks", "vs"):
            refuse(call, ALIAS, **{x: POOL[cached] + 64})
    if name == "bq_kv_read_i4":
        for bad in (dict(ldk=248), dict(hsk=120), dict(ldv=0), dict(hsv=0)):
            refuse(call, BOUNDS, **bad)
        refuse(call, ALIAS, k=at(6))
        refuse(call, ALIAS, slot=at(5) + 32)
    else:
        refuse(call, ALIAS, slot=POOL["ks"] + 32)
        refuse(call, ALIAS, cache_k=at(2))
        refuse(call, ALIAS, cache_vs=at(3))


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_attention_refusals(suffix):
    call = Call("bq_attn_i4" + suffix, ATTN)
    for ok in (dict(seqs=0), dict(rows=0), dict(max_q=0), dict(seqs=0, q=None, out=None, table=None, lens=None)):
        refuse(call, OK, **ok)
    for bad in (dict(seqs=-1), dict(seqs=(1 << 20) + 1), dict(rows=-1), dict(rows=1 << 29), dict(max_q=-1),
                dict(max_q=(1 << 20) + 1), dict(max_len=-1), dict(max_len=1 << 30), dict(heads=0),
                dict(heads=-2), dict(heads=3), dict(heads=130), dict(table_cols=-1), dict(window=-1),
                dict(seqs=1 << 20, max_q=1 << 20), dict(seqs=1 << 20, max_q=512, rows=7),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-float("inf"))):
        refuse(call, SIZE, **bad)
    for bad in ("q", "table", "lens", "out"):
        refuse(call, NULL, **{bad: None})
    for bad in (dict(q=at(5) + 2), dict(out=at(9) + 8), dict(ldq=514), dict(hsq=132, ldq=1024),
                dict(ldo=516), dict(table=at(6) + 2), dict(lens=at(7) + 1), dict(starts=at(8) + 2),
                dict(lse=at(10) + 2)):
        refuse(call, ALIGN, **bad)
    for bad in (dict(ldt=7), dict(ldq=-8), dict(hsq=-8), dict(ldq=1 << 47), dict(ldo=504), dict(hso=64),
                dict(ldo=0), dict(hso=0), dict(ldt=1 << 46)):
        refuse(call, BOUNDS, **bad)
    for inside in (POOL["k"], POOL["v"], POOL["ks"], POOL["vs"], ATTN["q"], ATTN["table"], ATTN["lens"],
                   ATTN["starts"]):
        refuse(call, ALIAS, out=inside)
        refuse(call, ALIAS, lse=inside)
    refuse(call, ALIAS, lse=ATTN["out"] + 64)


def test_workspace():
    size = bq.bq_attn_i4_ws_bytes
    for bad in (dict(seqs=-1), dict(rows=-1), dict(max_q=1 << 21), dict(max_len=1 << 30), dict(heads=5),
                dict(kv_heads=0), dict(kv_heads=-2), dict(heads=0), dict(dim=96), dict(rows=1 << 30)):
        assert size(**{**dict(seqs=1, rows=1, max_q=1, max_len=9999, heads=8, kv_heads=2, dim=128), **bad}) == -1
    assert size(0, 0, 0, 9999, 8, 2, 128) == 0 and size(1, 1, 1, 100, 8, 2, 128) == 0
    for dim in (64, 128, 256):
        for rows in (1, 3, 1 << 20):
            for max_len in (1, 5000, (1 << 30) - 1):
                for heads, kv in ((1, 1), (64, 1), (1024, 1024), (128, 2)):
                    if rows * heads < 1 << 31:
                        assert 0 <= size(1, rows, min(rows, 1 << 20), max_len, heads, kv, dim) <= 64 << 20
    call = Call("bq_attn_i4", ATTN)
    how = dict(seqs=1, rows=1, max_q=1, max_len=100000, starts=None)
    need = size(1, 1, 1, 100000, 4, 2, 128)
    assert need > 0
    refuse(call, SCRATCH, **how)
    refuse(call, SCRATCH, ws_bytes=need - 1, **how)
    refuse(call, SCRATCH, ws=None, ws_bytes=need, **how)
    refuse(call, ALIGN, ws=at(11) + 4, ws_bytes=need, **how)
    refuse(call, ALIAS, ws=at(9), ws_bytes=need, **how)
    refuse(call, ALIAS, ws=POOL["vs"], ws_bytes=need, **how)


def test_pools_that_are_taken_reach_the_launch():
    """Pages outside heads and heads outside pages, gaps, one page, shared rows: valid, so only the
    launch can fail where there is no GPU."""
    for name, args in (("bq_kv_write_i4", WRITE), ("bq_kv_read_i4", READ), ("bq_attn_i4", ATTN)):
        call = Call(name, args)
        for good in ({}, dict(page_stride=1024, head_stride=10240), dict(pages=1, page_stride=0),
                     dict(heads=1, head_stride=0), dict(page_stride=4096, spage_stride=1024),
                     dict(spage_stride=64, shead_stride=640)):
            refuse(call, LAUNCH, **{"cache_" + k: v for k, v in good.items()})
    refuse(Call("bq_kv_write_i4", WRITE), LAUNCH, ldk=0, hsk=0, v=at(5))
    refuse(Call("bq_attn_i4", ATTN), LAUNCH, ldq=0, hsq=0, lse=None, starts=None, window=1 << 50)
