// parts.cuh -- where the sums of a row block that was cut lie in the workspace (compiled for the device, and for the
// host in the tests).
#pragma once

#include <cstdint>

#include "drain.cuh"  // SPECREJ_HD

namespace specrej {

// Whether a row block cut into `count` parts (0: not cut), of which the first is that of block `first`, lies within
// the `blocks` of a call.  What the join of shared prefixes reads there is only written as the row block is begun:
// after a wait that gave up it may be anything that the workspace held before.
SPECREJ_HD inline bool parts_within(int32_t first, int32_t count, int32_t blocks)
{
    return count == 0 || (count > 0 && count <= blocks && first >= 0 && first <= blocks - count);
}

// The place of row `row` of part j: a block has max_rows places for the row block that came to it from the block
// before, and as many behind them for the one that begins in it and goes on.
SPECREJ_HD inline int64_t part_place(int32_t first, int32_t j, int32_t max_rows, int32_t row)
{
    return ((int64_t)(first + j) * 2 + (j == 0)) * max_rows + row;
}

}  // namespace specrej
