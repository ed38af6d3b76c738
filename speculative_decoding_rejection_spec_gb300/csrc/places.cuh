// places.cuh -- how many places of the list of work a request's row blocks can take (compiled for the device, and for
// the host in the tests).
#pragma once

#include <cstdint>

#include "drain.cuh"  // SPECREJ_HD

namespace specrej {

// At most so many for one head: every row block begins with `begin` places and has at most one tile of `tile_keys` more
// than `keys` fill, of `tile` places each.  Costs are 32-bit, so requests above INT32_MAX are refused; the bound itself
// is 64-bit.
SPECREJ_HD inline int64_t most_places(int64_t row_blocks, int64_t keys, int begin, int tile, int tile_keys)
{
    return row_blocks * (begin + tile * (1 + keys / tile_keys));
}

// The keys of a row block over at most `tokens` tokens of a window: those tokens' own, the window of the first, the
// sinks, and what copies of `box` keys bring at the end of the sinks and before the window.
SPECREJ_HD inline int64_t most_window_keys(int64_t context, int64_t tokens, int64_t window, int64_t sinks, int box)
{
    const int64_t keys = tokens + window + sinks + 2 * box;
    return keys < context ? keys : context;
}

}  // namespace specrej
