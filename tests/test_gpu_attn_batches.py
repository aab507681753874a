"""Attention over the 4-bit cache for batches of many sequences: 64 at a time are looked at, up to 256
are ordered by length and dealt out, and more are taken as they come."""
from __future__ import annotations

import numpy as np
import pytest

from gpu_util import say
from test_gpu_attn import Case

import block_quantized_wire_amd as bq

pytestmark = pytest.mark.gpu


def ragged(seed, seqs, short, long_at, long_len):
    """Short lengths, empty ones among them, and a few long ones."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, short, seqs)
    for i, at in enumerate(long_at):
        lens[at] = long_len - 100 * i
    return [int(n) for n in lens]


@pytest.mark.parametrize("kind,dim,group", [("bf16", 128, 64), ("f16", 64, 32), ("bf16", 256, 128)])
@pytest.mark.parametrize("seqs,long_at", [(63, (62,)), (64, (0, 63)), (65, (64,)), (70, (3, 66)), (128, (127,)),
                                          (130, (64, 129)), (193, (0, 192)), (255, (254,)), (256, (70, 255))])
def test_turns_of_many_sequences_dealt_out(kind, dim, group, seqs, long_at):
    lens = ragged([seqs, dim], seqs, 60, long_at, 4500)
    say(f"attn {seqs} sequences dealt out D={dim} {kind}")
    c = Case([seqs, dim], lens, None, 2, 1, dim, group, 16, kind)
    assert bq.bq_attn_i4_ws_bytes(seqs, seqs, 1, max(lens), 2, 1, dim) > 0
    c.check()


@pytest.mark.parametrize("seqs", [67, 129, 190])
def test_rows_of_many_sequences_dealt_out(seqs):
    """Sequences of no row, one and a few, two tiles among them."""
    rng = np.random.default_rng(seqs)
    new = [int(n) for n in rng.integers(0, 6, seqs)]
    lens = ragged([seqs], seqs, 40, (seqs - 1, 5, 65), 9000 if seqs < 190 else 20000)
    say(f"attn {seqs} sequences of up to 5 rows")
    c = Case([seqs], lens, new, 3, 1, 64, 64, 24, "bf16")
    assert bq.bq_attn_i4_ws_bytes(seqs, c.q.shape[0], c.max_q, max(lens), 3, 1, 64) > 0
    c.check(extra=2)
    c.check(window=50)


@pytest.mark.parametrize("seqs", [64, 65, 127, 200, 256, 257, 300, 700])
@pytest.mark.parametrize("new", [1, 3])
def test_many_sequences_each_in_a_workgroup(seqs, new):
    lens = ragged([seqs, new], seqs, 90, (seqs - 1, seqs // 2), 260)
    say(f"attn {seqs} sequences, {new} rows")
    c = Case([seqs, new], lens, None if new == 1 else [new] * seqs, 4, 2, 64, 32, 8, "f16")
    assert bq.bq_attn_i4_ws_bytes(seqs, c.q.shape[0], c.max_q, max(lens), 4, 2, 64) == 0
    c.check()


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("seqs", [65, 130, 256, 257, 300])
def test_many_rows_of_many_sequences(kind, dim, seqs):
    rng = np.random.default_rng(seqs)
    lens = ragged([seqs, dim], seqs, 50, (seqs - 1, seqs // 3), 200)
    new = [int(n) for n in rng.integers(0, 4, seqs)]
    new[seqs - 1], new[64], new[2] = 9, 9, 5
    say(f"attn {seqs} sequences of many rows {kind}")
    c = Case([seqs, dim], lens, new, 16, 2, dim, 64, 16, kind)
    assert c.max_q * 8 > 64
    c.check(extra=1)
