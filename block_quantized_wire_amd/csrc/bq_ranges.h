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

}  // namespace bq
