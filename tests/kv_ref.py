"""Plain implementations, on the host and in 64 bits where values are computed, of the 4-bit
cache of keys and values and of attention over it.  They share no code with the library: codes
are found number by number from the places that include/blockq_kv.h gives them."""
from __future__ import annotations

import math

import numpy as np
import torch

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}      # what one rounding may cost, relative
# a weight times a scale, relative: binary16 has 11 significant bits, so a number in [2^e, 2^(e+1)) lies
# within half of 2^(e-10) of its rounding, 2^-11 of 2^e or less; two such parts hold it to 2^-22
HELD = {"bf16": 2.0 ** -11, "f16": 2.0 ** -20}
TINY = {"bf16": 0.0, "f16": 2.0 ** -25}            # ... and absolute


def k_place(dim):
    """(byte within a token's row, odd nibble) of every number of a key."""
    d = np.arange(dim)
    word = (d % 32) // 8 * (dim // 32) + d // 32
    return word * 4 + d % 8 // 2, d % 2


def v_place(dim, t):
    """(byte within a block of 8 tokens, odd nibble) of every number of token t's value."""
    d = np.arange(dim)
    j, r = d // 16, d % 16
    word = (r * 4 + t // 2) * (dim // 64) + j // 4
    return word * 4 + t % 2 * 2 + j % 4 // 2, j % 2


class Pool:
    """The arrays of a cache on the host, in the layout of the library."""

    def __init__(self, pages, heads, page, dim, group, kind, fill=0xA5):
        self.pages, self.heads, self.page, self.dim, self.group, self.kind = pages, heads, page, dim, group, kind
        self.codes = [np.full((pages, heads, page * dim // 2), fill, np.uint8) for _ in "kv"]
        bits = np.full((pages, heads, dim // group, page, 2), fill * 0x0101, np.uint16).view(np.int16)
        self.scales = [torch.from_numpy(bits.copy()).view(TORCH[kind]) for _ in "kv"]

    def where(self, which, place):
        if which == 0:
            byte, odd = k_place(self.dim)
            return byte + place * (self.dim // 2), odd
        byte, odd = v_place(self.dim, place % 8)
        return byte + place // 8 * (4 * self.dim), odd

    def put(self, which, slot, codes, scale, least):
        """codes [heads, dim], scale and least [heads, dim / group] of one slot."""
        page, place = divmod(slot, self.page)
        byte, odd = self.where(which, place)
        row = self.codes[which][page]
        for nib in (0, 1):
            at = byte[odd == nib]
            keep = 0xF0 if nib == 0 else 0x0F
            row[:, at] = (row[:, at] & keep) | (codes[:, odd == nib] << (4 * nib))
        self.scales[which][page, :, :, place, 0] = scale
        self.scales[which][page, :, :, place, 1] = least

    def get(self, which, slots):
        """codes, scale, least of slots, [n, heads, dim] in 64 bits."""
        slots = np.asarray(slots, np.int64)
        n, dim = len(slots), self.dim
        codes = np.empty((n, self.heads, dim))
        for place in np.unique(slots % self.page):
            on = np.nonzero(slots % self.page == place)[0]
            byte, odd = self.where(which, int(place))
            b = self.codes[which][slots[on] // self.page][:, :, byte]
            codes[on] = np.where(odd == 1, b >> 4, b & 15)
        pairs = self.scales[which].double().numpy()[slots // self.page, :, :, slots % self.page]
        s = np.repeat(pairs[..., 0], self.group, 2)
        m = np.repeat(pairs[..., 1], self.group, 2)
        return codes, s, m

    def random(self, rng, spread=0.3):
        """Every code and scale; values of about one."""
        for which in (0, 1):
            c = np.clip(np.rint(rng.normal(7.5, 2.6, self.codes[which].shape + (2,))), 0, 15).astype(np.uint8)
            self.codes[which][:] = c[..., 0] | (c[..., 1] << 4)
            shape = tuple(self.scales[which].shape[:-1])
            s = rng.uniform(0.2, 0.2 + spread, shape)
            m = s * rng.normal(-7.5, 0.7, shape)
            self.scales[which][..., 0] = torch.from_numpy(s).to(TORCH[self.kind])
            self.scales[which][..., 1] = torch.from_numpy(m).to(TORCH[self.kind])
        return self


def quantise(x, group, kind):
    """codes [.., dim], scale and least [.., dim / group] (16-bit) of rows x, by the definition."""
    v = x.float().numpy().astype(np.float64)
    g = v.reshape(v.shape[:-1] + (-1, group))
    lo, hi = g.min(-1), g.max(-1)
    with np.errstate(all="ignore"):
        unit = torch.from_numpy(((hi - lo) / 15.0).astype(np.float32)).to(TORCH[kind])
        s = unit.double().numpy()[..., None]
        q = np.where(s > 0, np.rint(((g - lo[..., None]) / s).astype(np.float32)), 0.0)
        bad = ~np.isfinite(g).all(-1)
    codes = np.where(bad[..., None], 0, np.clip(np.nan_to_num(q), 0, 15)).astype(np.uint8)
    least = torch.from_numpy(np.where(bad, np.nan, lo).astype(np.float32)).to(TORCH[kind])
    unit = torch.where(torch.from_numpy(bad), torch.full_like(unit, float("nan")), unit)
    return codes.reshape(v.shape), unit, least


def read(pool, which, slots):
    """The rows of slots in the type; zeros for slots outside."""
    slots = np.asarray(slots, np.int64)
    inside = (slots >= 0) & (slots < pool.pages * pool.page)
    c, s, m = pool.get(which, np.where(inside, slots, 0))
    with np.errstate(all="ignore"):
        y = (c * s + m).astype(np.float32)      # c * s is exact, one rounding to binary32
    y[~inside] = 0
    return torch.from_numpy(y).to(TORCH[pool.kind])


def attend(pool, q, table, lens, starts, causal, window, scale, kind):
    """out, lse and bounds on the kernel's distance from them, in 64 bits.

    A score's binary32 error: the products with the codes and the group's sum of q, each a sum of at
    most dim terms in any order and 2^-23 a step (which covers any rounding of the matrix
    cores), over the sum of the terms' sizes; q's own rounding (2^-25 of the largest of its row, 2^4
    times that for half of its numbers) is below a step.  A weight is off by that and by exp2's and
    the reference's rounding; weights times scales are held to 2^-20 (for bf16 results to 11 bits:
    half a step is 2^-11 at most); where there are many rows a value is a binary16 number, c s + m
    rounded once: 2^-11 of it at most; sums over the tokens take a step for 8 tokens and a few more
    to join, over the sizes of (c - 8) s and of m + 8 s."""
    rows, heads, dim = q.shape
    share = heads // pool.heads
    out, lse = np.zeros((rows, heads, dim)), np.full((rows, heads), -np.inf)
    eo, el = np.zeros((rows, heads, dim)), np.zeros((rows, heads))
    x = q.double().numpy()
    ulp = 2.0 ** -23
    for b, n in enumerate(lens):
        r0, r1 = (b, b + 1) if starts is None else (int(starts[b]), int(starts[b + 1]))
        if n == 0 or r1 <= r0:
            continue
        tok = np.arange(n)
        page = np.asarray(table[b])[tok // pool.page]
        good = (page >= 0) & (page < pool.pages)
        slot = np.where(good, page, 0) * pool.page + tok % pool.page
        kc, ks, km = pool.get(0, slot)
        vc, vs, vm = pool.get(1, slot)
        for i in range(r1 - r0):
            p = n - (r1 - r0) + i
            sees = good.copy()
            if causal:
                sees &= tok <= p
            if window:
                sees &= tok > max(-1, p - window)
            if not sees.any():
                continue
            on = np.nonzero(sees)[0]
            for h in range(heads):
                c = h // share
                a = x[r0 + i, h]
                kk = kc[on, c] * ks[on, c] + km[on, c]
                s = scale * (kk @ a)
                size = abs(scale) * ((kc[on, c] * np.abs(ks[on, c]) + np.abs(km[on, c])) @ np.abs(a))
                top = s.max()
                w = np.exp(s - top)
                total = w.sum()
                lse[r0 + i, h] = top + math.log(total)
                w /= total
                v = vc[on, c] * vs[on, c] + vm[on, c]
                out[r0 + i, h] = w @ v
                steps = dim + 16
                off = ulp * (steps * size + np.abs(s) + np.abs(s - top) + 4)
                mean = (w * off).sum()
                parts = np.abs(vc[on, c] - 8) * np.abs(vs[on, c]) + np.abs(vm[on, c] + 8 * vs[on, c])
                sums = ulp * (n / 8 + 32)
                e = ((w * (off + mean + HELD[kind] + sums))[:, None] * parts).sum(0)
                e += (w[:, None] * np.abs(v)).sum(0) * 2.0 ** -11
                # m + 8 s is rounded for each token
                e += ((w * ulp)[:, None] * (np.abs(vm[on, c]) + 8 * np.abs(vs[on, c]))).sum(0)
                eo[r0 + i, h] = e + (np.abs(out[r0 + i, h]) + e) * HALF[kind] + TINY[kind]
                el[r0 + i, h] = mean + sums + ulp * (abs(lse[r0 + i, h]) + abs(top) + 4)
    return out, lse, eo, el
