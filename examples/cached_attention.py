"""An attention layer on libblockq as a server runs it: 4-bit projections, keys and values written
into a 4-bit paged cache, and attention over it, for prompts in chunks and for tokens one by one.

    python examples/cached_attention.py [--seqs 5] [--prompt 300] [--heads 16] [--kv-heads 4]
                                        [--dim 128] [--group 64] [--page 16] [--hidden 512]

Writes the prompts of a ragged batch in two chunks, then takes decode steps, first as single calls
and then as one captured graph that is replayed, and compares every result with plain torch in
binary32 on what the cache holds.  Every buffer is the caller's and is made once.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_wire_amd as bq  # noqa: E402


class Linear4:
    """y = x W^T with 4-bit weights, quantized from bf16 (rows, cols)."""

    def __init__(self, w: torch.Tensor, group: int):
        n, k = w.shape
        self.group = group
        self.codes = torch.empty((n, -(-(k // 2) // 16) * 16), dtype=torch.uint8, device=w.device)
        self.scale = torch.zeros((n, -(-(k // group) // 4) * 4), dtype=w.dtype, device=w.device)
        bq.bq_quant_i4(w, self.codes, self.scale, group=group)

    def __call__(self, x, y):
        bq.bq_mm_i4(x, self.codes, self.scale, y, group=self.group)


class Cache:
    """A pool of pages and who has them.  A server's allocator: a page is taken when a sequence's
    last one is full."""

    def __init__(self, pages, seqs, heads, page, dim, group, dtype, dev):
        codes = lambda: torch.zeros((pages, heads, page, dim // 2), dtype=torch.uint8, device=dev)  # noqa: E731
        scales = lambda: torch.zeros((pages, heads, dim // group, page, 2), dtype=dtype, device=dev)  # noqa: E731
        self.kv = bq.KvI4(codes(), codes(), scales(), scales(), group=group)
        self.page, self.free = page, list(range(pages))[::-1]
        self.table = [[] for _ in range(seqs)]
        self.lens = [0] * seqs

    def slots(self, new):
        """Slots of `new[b]` more tokens of every sequence b, in order."""
        out = []
        for b, n in enumerate(new):
            for t in range(self.lens[b], self.lens[b] + n):
                if t // self.page == len(self.table[b]):
                    self.table[b].append(self.free.pop())
                out.append(self.table[b][t // self.page] * self.page + t % self.page)
            self.lens[b] += n
        return out

    def values(self, which: str) -> torch.Tensor:
        """What the cache holds, in binary32: (pages, heads, page, dim).  (bq_kv_read_i4 rounds the
        same to the cache's type.)"""
        kv, d = self.kv, self.kv.dim
        codes, scales = getattr(kv, which), getattr(kv, which + "s")
        p, h, s, _ = codes.shape
        two = lambda c: torch.stack((c & 15, c >> 4), -1)  # noqa: E731
        if which == "k":        # words (g, i) hold numbers 32i + 8g ..
            c = two(codes.reshape(p, h, s, 4, d // 32, 4)).transpose(3, 4)
        else:                   # blocks of 8 tokens: words (r, pair, 4j ..) of two tokens' half-words
            c = two(codes.reshape(p, h, s // 8, 16, 4, d // 64, 2, 2)).permute(0, 1, 2, 4, 6, 5, 7, 8, 3)
        c = c.reshape(p, h, s, d // kv.group, kv.group).float()
        pair = scales.float().transpose(2, 3)[..., None]
        return (c * pair[..., 0, :] + pair[..., 1, :]).reshape(p, h, s, d)


class Attention:
    """hidden -> hidden, for up to max_rows rows at once."""

    def __init__(self, qkv: torch.Tensor, out: torch.Tensor, heads, kv_heads, dim, max_rows, max_len, seqs,
                 group=128):
        dev, dt = qkv.device, qkv.dtype
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.qkv, self.out = Linear4(qkv, group), Linear4(out, group)
        self.rows = torch.empty((max_rows, (heads + 2 * kv_heads) * dim), dtype=dt, device=dev)
        self.mixed = torch.empty((max_rows, heads * dim), dtype=dt, device=dev)
        self.lse = torch.empty((max_rows, heads), device=dev)
        # one workspace for every call of the layer, one after the other
        need = max(bq.bq_attn_i4_ws_bytes(seqs, r, q, max_len, heads, kv_heads, dim)
                   for r, q in ((seqs, 1), (max_rows, max_rows)))
        self.ws = torch.empty(max(need, 64 << 20), dtype=torch.uint8, device=dev)

    def __call__(self, x, cache, slots, table, lens, y, starts=None, max_q=None, max_len=None):
        n, h, kv, d = x.shape[0], self.heads, self.kv_heads, self.dim
        rows = self.rows[:n]
        self.qkv(x, rows)
        # queries, keys and values lie in the rows of one projection
        q = rows[:, : h * d].view(n, h, d)
        k = rows[:, h * d: (h + kv) * d].view(n, kv, d)
        v = rows[:, (h + kv) * d:].view(n, kv, d)
        bq.bq_kv_write_i4(k, v, slots, cache.kv)
        bq.bq_attn_i4(q, cache.kv, table, lens, self.mixed[:n].view(n, h, d), starts=starts, max_q=max_q,
                      max_len=max_len, lse=self.lse[:n], ws=self.ws)
        self.out(self.mixed[:n], y)
        return q

    def plain(self, q, cache, lens, new):
        """The attention of rows q over what the cache holds, sequence by sequence, in binary32."""
        k, v = cache.values("k"), cache.values("v")
        out, row = [], 0
        for b, n in enumerate(lens):
            pages = torch.tensor(cache.table[b], device=q.device, dtype=torch.int64)
            kb = k[pages].transpose(0, 1).reshape(self.kv_heads, -1, self.dim)[:, :n]
            vb = v[pages].transpose(0, 1).reshape(self.kv_heads, -1, self.dim)[:, :n]
            share = self.heads // self.kv_heads
            x = q[row:row + new[b]].float().transpose(0, 1)
            score = x @ kb.repeat_interleave(share, 0).transpose(1, 2) * self.dim ** -0.5
            at = torch.arange(n - new[b], n, device=q.device)
            score.masked_fill_(torch.arange(n, device=q.device) > at[:, None], -torch.inf)
            out.append((torch.softmax(score, -1) @ vb.repeat_interleave(share, 0)).transpose(0, 1))
            row += new[b]
        return torch.cat(out).reshape(row, -1)


def distance(got, want):
    return float((got.float() - want.float()).norm() / want.float().norm())


def run(seqs=5, prompt=300, heads=16, kv_heads=4, dim=128, group=64, page=16, hidden=512, steps=3, seed=1):
    """Distances (relative, 2-norm) of the attention's rows from plain torch: of the two chunks of the
    prompts, of single decode steps, of the replayed graph's."""
    dev, dt = "cuda", torch.bfloat16
    g = torch.Generator(device=dev).manual_seed(seed)
    norm = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    width = (heads + 2 * kv_heads) * dim
    longest = prompt + 2 * steps
    first = [max(1, prompt // 2 - 17 * b) for b in range(seqs)]
    second = [max(1, prompt // 3 - 5 * b) for b in range(seqs)]
    pages = seqs * (-(-longest // page))
    layer = Attention((norm(width, hidden) * hidden ** -0.5 * 2).to(dt),
                      (norm(hidden, heads * dim) * (heads * dim) ** -0.5).to(dt), heads, kv_heads, dim,
                      max(sum(first), sum(second), seqs), longest, seqs)
    cache = Cache(pages, seqs, kv_heads, page, dim, group, dt, dev)
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731

    def table():
        cols = -(-longest // page)
        return ints([t + [0] * (cols - len(t)) for t in cache.table])

    errors = {}
    for name, new in (("first chunk", first), ("second chunk", second)):
        slots = ints(cache.slots(new))
        starts = ints([sum(new[:b]) for b in range(seqs + 1)])
        x, y = norm(sum(new), hidden).to(dt), torch.empty((sum(new), hidden), dtype=dt, device=dev)
        q = layer(x, cache, slots, table(), ints(cache.lens), y, starts=starts, max_q=max(new), max_len=longest)
        errors[name] = distance(layer.mixed[: sum(new)], layer.plain(q, cache, cache.lens, new))

    # a decode step's buffers, which the graph goes by
    x, y = norm(seqs, hidden).to(dt), torch.empty((seqs, hidden), dtype=dt, device=dev)
    slots, tab, lens = ints([0] * seqs), table(), ints(cache.lens)

    def set_step():
        slots.copy_(ints(cache.slots([1] * seqs)))
        tab.copy_(table())
        lens.copy_(ints(cache.lens))
        x.copy_(norm(seqs, hidden).to(dt))

    worst = 0.0
    for _ in range(steps):
        set_step()
        q = layer(x, cache, slots, tab, lens, y, max_len=longest)
        worst = max(worst, distance(layer.mixed[:seqs], layer.plain(q, cache, cache.lens, [1] * seqs)))
    errors["steps"] = worst
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = layer(x, cache, slots, tab, lens, y, max_len=longest)
    worst = 0.0
    for _ in range(steps):
        set_step()
        graph.replay()
        worst = max(worst, distance(layer.mixed[:seqs], layer.plain(q, cache, cache.lens, [1] * seqs)))
    errors["graph"] = worst
    return errors


def close(errors) -> bool:
    """Whether the rows are as near as one rounding to bf16 (2^-8 at most of a value) leaves them."""
    return all(v < 2.0 ** -8 for v in errors.values())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("seqs", 5), ("prompt", 300), ("heads", 16), ("kv-heads", 4), ("dim", 128), ("group", 64),
                        ("page", 16), ("hidden", 512), ("steps", 3)):
        ap.add_argument("--" + name, type=int, default=value)
    found = run(**{k.replace("-", "_"): v for k, v in vars(ap.parse_args()).items()})
    for k, v in found.items():
        print(f"{k:14s} {v:.2e}")
    sys.exit(0 if close(found) else 1)
