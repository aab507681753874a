// bq_ranges.h -- which rows the expert layer's int32 arrays name, for arrays with anything in
// them.
//
// Offsets are read on the device, where nothing has checked them, and a row number that is
// used as an address comes out of here.  Everything is constexpr, so the kernels and a host
// program compile the same arithmetic; none of it overflows for any int32 input.
#pragma once

#include <stdint.h>

namespace bq {

// Rows [lo, hi) of an expert whose offsets are `first` and `end`: 0 <= lo <= hi <= rows.
// Both ends are brought inside before they are compared: the difference of two offsets wraps.
struct RowRange {
    int32_t lo, hi;
};
constexpr RowRange expert_rows(int32_t first, int32_t end, int32_t rows) {
    const int32_t lo = first < 0 ? 0 : first < rows ? first : rows;
    return RowRange{lo, end < lo ? lo : end < rows ? end : rows};
}

// The row of x that a slot's token is, or -1 where there is none.  The sign is tested before the
// division, which rounds towards 0.
constexpr int32_t source_row(int32_t slot, int32_t topk, int32_t x_rows) {
    return slot < 0 || slot / topk >= x_rows ? -1 : slot / topk;
}

}  // namespace bq
