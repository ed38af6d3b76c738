// drain.cuh -- how a block that gave up a wait ends the phases of its barriers whose copies are in flight
// (compiled for the device, and for the host in the tests).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SPECREJ_HD __host__ __device__
#else
#define SPECREJ_HD
#endif

namespace specrej {

// A barrier of `count` arrivals a phase, of which `arrivals` have been made in all, each after the phase
// before its own had completed; copies that complete on it were announced with them.  The last phase
// begun has arrivals outstanding (those of roles that stopped) and completes with `missing` more and the
// bytes announced; waiting for `parity` then is waiting for it.  Nothing was begun without an arrival.
struct Drain {
    bool begun;
    uint32_t missing, parity;
};

SPECREJ_HD inline Drain drain_of(uint32_t arrivals, uint32_t count)
{
    const uint32_t phases = (arrivals + count - 1) / count;
    return Drain{arrivals > 0, phases * count - arrivals, (phases - 1) & 1};
}

}  // namespace specrej
