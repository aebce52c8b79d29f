// Tensor maps of the grouped products' operands (host side).
#pragma once
#include <cuda.h>

namespace mg {

// bf16 [outer][rows][cols], rows ld elements apart (0: cols); box box_cols x
// box_rows x 1, 128-byte swizzle, zeros outside.  outer = 0: two-dimensional.
// False if the driver has no encoder or refuses.
bool group_map(CUtensorMap* map, const void* base, long long outer, long long rows, long long cols, long long ld,
               int box_cols, int box_rows);

}  // namespace mg
