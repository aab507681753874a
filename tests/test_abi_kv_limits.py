"""Sizes at which attention over the 4-bit cache is cut another way or refused, on the host: nothing
is launched."""
from __future__ import annotations

import ctypes

import pytest

import block_quantized_wire_amd as bq
from block_quantized_wire_amd import build as _build

if _build.stale():
    _build.build()

MOST = (1 << 30) - 1


def test_turns_that_are_dealt_out_can_be_counted():
    """Turns of 128 tokens are counted in 32 bits: with 2^31 of them or more, each unit keeps its own, for
    which a workspace is not needed."""
    size = bq.bq_attn_i4_ws_bytes
    assert size(256, 256, 1, MOST, 1, 1, 128) == 0
    assert size(1, 1, 1, MOST, 380, 380, 64) == 0
    assert size(1, 16, 16, MOST, 96 * 16, 96, 256) == 0
    assert size(255, 255, 1, MOST, 1, 1, 128) > 0
    assert size(256, 256, 1, 1 << 29, 1, 1, 128) > 0
    for dim in (64, 128, 256):
        for base in (1, 7, 200, 255, 256, 300, 383):
            for max_len in (MOST, 1 << 29, (1 << 29) + 1, 900000000, 800000000):
                if base * ((max_len + 127) // 128 + 1) >= 1 << 31:
                    assert size(1, 1, 1, max_len, base, base, dim) == 0
                else:
                    assert size(1, 1, 1, max_len, base, base, dim) > 0


@pytest.mark.parametrize("name", ["bq_attn_i4", "bq_attn_i4_f16"])
def test_scales_whose_product_with_log2_e_is_not_finite(name):
    """|scale| up to 2^126 is taken; beyond it every row that sees something would be NaN."""
    pool = bq._KvI4(16, 32, 48, 64, 2048, 1024, 128, 64, 10, 16, 2, 128, 64)

    def call(scale):        # no sequence: the arguments are looked at, and no pointer is read
        return getattr(bq.lib, name)(None, 0, 0, ctypes.addressof(pool), None, 0, 0, None, None, 0, 0, 0, 0, 4, 1, 0,
                                     scale, None, 0, 0, None, None, 0, 0)
    for scale in (2.0 ** 126, -2.0 ** 126, 0.0, 1e-45):
        assert call(scale) == 0
    for scale in (2.0 ** 126 * (1 + 2.0 ** -23), -2.0 ** 127, 3.4e38, float("inf"), -float("inf"), float("nan")):
        assert call(scale) == 2
