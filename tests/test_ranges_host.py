"""The arithmetic that turns the expert layer's int32 arrays into row numbers, compiled for the
host from the header that the kernels include, over the extremes of int32 (with overflow
trapped): whatever the arrays hold, a row that is used as an address is inside."""
from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_quantized_wire_amd", "csrc")

VALUES = """
static const int32_t kAny[] = {INT32_MIN, INT32_MIN + 1, -0x60000000, -(1 << 30), -65536, -300, -64,
                               -3, -2, -1, 0, 1, 2, 3, 5, 63, 64, 65, 127, 128, 299, 300, 301, 65536,
                               (1 << 29) + 7, (1 << 30) - 1, 1 << 30, 0x60000000, INT32_MAX - 1,
                               INT32_MAX};
static const int32_t kRows[] = {1, 2, 63, 64, 300, 4096, (1 << 30) - 1, 1 << 30};
"""


def run(tmp_path, body):
    src = tmp_path / "p.cpp"
    src.write_text('#include "bq_ranges.h"\n#include <initializer_list>\n#include <stdint.h>\n#include <stdio.h>\n' + VALUES + body)
    exe = tmp_path / "p"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-ftrapv",
                    "-I", CSRC, str(src), "-o", str(exe)], check=True, timeout=300)
    got = subprocess.run([str(exe)], timeout=300, capture_output=True, text=True)
    assert got.returncode == 0, got.stdout + got.stderr


def test_an_experts_rows_are_inside(tmp_path):
    """0 <= lo <= hi <= rows for any pair of offsets, the pair itself where it is valid, and a
    count of row blocks that fits the launch's bound of rows / tile + 1."""
    run(tmp_path, """
int main() {
    for (int32_t rows : kRows)
        for (int32_t first : kAny)
            for (int32_t end : kAny) {
                const bq::RowRange r = bq::expert_rows(first, end, rows);
                bool ok = 0 <= r.lo && r.lo <= r.hi && r.hi <= rows;
                if (0 <= first && first <= end && end <= rows)
                    ok = ok && r.lo == first && r.hi == end;
                if (first >= end || first >= rows || end <= 0)
                    ok = ok && r.lo == r.hi;
                for (int tile : {64, 128})
                    ok = ok && (r.hi - r.lo + tile - 1) / tile <= rows / tile + 1;
                if (!ok)
                    return printf("rows %d offsets %d %d: [%d, %d)\\n", rows, first, end, r.lo, r.hi), 1;
            }
    return 0;
}
""")


def test_a_source_names_a_row_of_x_or_none(tmp_path):
    """A slot in [0, x_rows * topk) names row slot / topk; every other value names none, those
    between -topk and 0 too."""
    run(tmp_path, """
int main() {
    for (int32_t rows : kRows)
        for (int32_t topk : {1, 2, 7, 64})
            for (int32_t slot : kAny) {
                const int32_t r = bq::source_row(slot, topk, rows);
                const bool there = slot >= 0 && slot < (int64_t)rows * topk;
                if (there ? r != slot / topk : r != -1)
                    return printf("rows %d topk %d slot %d: row %d\\n", rows, topk, slot, r), 1;
            }
    return 0;
}
""")
