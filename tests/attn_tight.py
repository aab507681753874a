"""Closer bounds than kv_ref's on attention over a binary16 cache, whose values are held to 2^-22."""
from __future__ import annotations

import math

import numpy as np

ULP = 2.0 ** -23


def attend(pool, q, table, lens, scale, held=None):
    """out and its bound for one row a sequence.  held: a rounding of the weights times scales, planted.

    As in kv_ref: a score is a binary32 sum of dim + 16 steps, weights are off by that and by exp2's and the
    reference's rounding, sums over tokens take a step for 8 of them and a few more.  A weight times a
    scale is two binary16 numbers, 2^-11 of 2^-11 at most, and the first takes up to half a step of what is
    below 2^-14: 2^-20 covers the first, and the second is at most 2^-25, times a code's distance of 8, where
    the largest scale has 2^6 or more: 2^-28 of it, or 2^-8 of the weight's own part."""
    rows, heads, dim = q.shape
    share = heads // pool.heads
    x = q.double().numpy()
    out, eo = np.zeros((rows, heads, dim)), np.zeros((rows, heads, dim))
    for b, n in enumerate(lens):
        tok = np.arange(n)
        slot = np.asarray(table[b])[tok // pool.page].astype(np.int64) * pool.page + tok % pool.page
        kc, ks, km = pool.get(0, slot)
        vc, vs, vm = pool.get(1, slot)
        for h in range(heads):
            c, a = h // share, x[b, h]
            s = scale * ((kc[:, c] * ks[:, c] + km[:, c]) @ a)
            size = abs(scale) * ((kc[:, c] * np.abs(ks[:, c]) + np.abs(km[:, c])) @ np.abs(a))
            w = np.exp(s - s.max())
            total = w.sum()
            least = vm[:, c] + 8 * vs[:, c]
            ps = w[:, None] * vs[:, c]
            if held is not None:
                ps = held(ps)
            out[b, h] = (ps * (vc[:, c] - 8) + w[:, None] * least).sum(0) / total
            w /= total
            off = ULP * ((dim + 16) * size + np.abs(s) + np.abs(s - s.max()) + 4)
            sums = ULP * (n / 8 + 32)
            parts = np.abs(vc[:, c] - 8) * np.abs(vs[:, c]) + np.abs(least)
            e = ((w * (off + (w * off).sum() + 2.0 ** -20 + sums))[:, None] * parts).sum(0)
            e += ((w * ULP)[:, None] * (np.abs(vm[:, c]) + 8 * np.abs(vs[:, c]))).sum(0)
            e += np.minimum(2.0 ** -28 * np.abs(vs[:, c]).max(), 2.0 ** -8 * w[:, None] * np.abs(vs[:, c])).sum(0)
            eo[b, h] = e + (np.abs(out[b, h]) + e) * 2.0 ** -11 + 2.0 ** -25
    return out, eo


def attend_rows(pool, q, table, n, scale, held=None):
    """out and its bound for many rows of one sequence, each of which sees all n tokens.  held: a rounding of
    the values, planted.

    Scores, weights and sums as above.  A value is two binary16 numbers: 2^-22 of it, or 2^-25 where the second
    is below 2^-14.  A weight times 2^6 is two as well: 2^-22 of it, or 2^-25, 2^-31 of the weight of the
    reference, which the weights' sum is not below; the product of the second ones, 2^-22 of the whole, is left out."""
    rows, heads, dim = q.shape
    share = heads // pool.heads
    x = q.double().numpy()
    out, eo = np.zeros((rows, heads, dim)), np.zeros((rows, heads, dim))
    tok = np.arange(n)
    slot = np.asarray(table)[tok // pool.page].astype(np.int64) * pool.page + tok % pool.page
    kc, ks, km = pool.get(0, slot)
    vc, vs, vm = pool.get(1, slot)
    for h in range(heads):
        c = h // share
        k, v = kc[:, c] * ks[:, c] + km[:, c], vc[:, c] * vs[:, c] + vm[:, c]
        if held is not None:
            v = held(v)
        for i in range(rows):
            a = x[i, h]
            s = scale * (k @ a)
            size = abs(scale) * ((kc[:, c] * np.abs(ks[:, c]) + np.abs(km[:, c])) @ np.abs(a))
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ v
            off = ULP * ((dim + 16) * size + np.abs(s) + np.abs(s - s.max()) + 4)
            rel = (w * (off + (w * off).sum() + 3 * 2.0 ** -22 + ULP * (n / 8 + 32)))[:, None]
            e = (rel * np.abs(v) + w[:, None] * 2.0 ** -25 + 2.0 ** -31 * np.abs(v)).sum(0)
            eo[i, h] = e + (np.abs(out[i, h]) + e) * 2.0 ** -11 + 2.0 ** -25
    return out, eo


def binary16(x):
    return x.astype(np.float16).astype(np.float64)


def case(make, dim, group, n):
    """Scores of about 0, so that their own rounding is small beside what is looked for."""
    return make([dim, group, n], (n,), None, 4, 2, dim, group, 16, "f16", q_size=2.0 ** -9)


def case_rows(make, dim, group, n):
    return make([dim, group, n, 1], (n,), (40,), 4, 2, dim, group, 16, "f16", q_size=2.0 ** -9)
