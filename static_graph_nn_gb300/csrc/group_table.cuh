// The row ranges of the groups of a grouped product and their tile counts,
// read from the offsets in device memory by one warp into shared memory.
#pragma once
#include <stdint.h>

namespace mg {

// Entries [0, groups): the groups.  With zero_rest two more: the rows before
// the first group and behind the last one, which belong to none.
struct GroupTable {
  int* lo;    // first row
  int* hi;    // one past the last row
  int* cum;   // inclusive prefix sum of row tiles
  int n;      // entries
};

constexpr int kGroupTableInts(int max_groups) { return 3 * (max_groups + 2); }

// Called by all 32 lanes of one warp; the others read it after a barrier.
// Offsets that decrease or leave [0, rows] are clamped: a group then has the
// rows that no earlier one has, and no index leaves [0, rows].
static __device__ __forceinline__ void load_group_table(const GroupTable& t, const int* offsets, int groups,
                                                        int rows, int tile_rows) {
  const int lane = threadIdx.x & 31;
  auto clamp = [&](int v) { return min(max(v, 0), rows); };
  const int first = clamp(offsets[0]);
  int row = first, tiles = 0;
  for (int b = 0; b < groups; b += 32) {
    const int e = b + lane;
    int hi = e < groups ? clamp(offsets[e + 1]) : 0;
    hi = max(hi, row);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, hi, o);
      if (lane >= o) hi = max(hi, y);
    }
    int lo = __shfl_up_sync(0xffffffffu, hi, 1);
    if (lane == 0) lo = row;
    int c = (hi - lo + tile_rows - 1) / tile_rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += y;
    }
    if (e < groups) {
      t.lo[e] = lo;
      t.hi[e] = hi;
      t.cum[e] = tiles + c;
    }
    row = __shfl_sync(0xffffffffu, hi, 31);
    tiles += __shfl_sync(0xffffffffu, c, 31);
  }
  if (lane == 0 && t.n > groups) {
    t.lo[groups] = 0;
    t.hi[groups] = first;
    t.cum[groups] = tiles + (first + tile_rows - 1) / tile_rows;
    t.lo[groups + 1] = row;
    t.hi[groups + 1] = rows;
    t.cum[groups + 1] = t.cum[groups] + (rows - row + tile_rows - 1) / tile_rows;
  }
}

}  // namespace mg
