"""What the binding of the 4-bit cache passes on where a table has room for more tokens than a sequence may
have.  The library behind it is a stand-in, so nothing is launched."""
from __future__ import annotations

import torch

import block_quantized_wire_amd as bq
from test_binding_kv import attn_args, lib  # noqa: F401


def test_longest_sequence_of_a_wide_table(lib):  # noqa: F811
    for cols, most in ((5, 80), ((1 << 26) - 1, (1 << 30) - 16), (1 << 26, (1 << 30) - 1), (1 << 27, (1 << 30) - 1)):
        bq.bq_attn_i4(**attn_args(table=Wide(cols)))
        assert lib.calls.pop()[1][12] == most


class Wide:
    """A table of many columns without its memory."""

    dtype, device = torch.int32, torch.device("cpu")

    def __init__(self, cols):
        self.shape = (3, cols)

    def stride(self):
        return (self.shape[1], 1)

    def get_device(self):
        return -1

    def data_ptr(self):
        return 64
