// bulk_ring.cuh -- which copies of a ring in shared memory may still be under way.
//
// One thread issues copies 0, 1, 2, ...: copy x goes to place x % slots and completes phase x / slots of that place's
// mbarrier.  It issues copy x only after it has itself waited for copy x - slots.  So when it stops, wherever that is,
// all copies but the last `slots` have landed, and each of those is the newest of its place: its parity names it.
// (What the loop around it has counted by then says nothing of that: the loop may go on without copies.)
//
// Plain arithmetic, host code too: tests/test_ring_drain.py goes through every stopping point.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MOE_RING_FN __host__ __device__ __forceinline__
#else
#define MOE_RING_FN inline
#endif

namespace moe {

// The first of the `issued` copies that may not have landed, and a copy's place and parity.
MOE_RING_FN uint32_t ring_first_open(uint32_t issued, uint32_t slots) { return issued > slots ? issued - slots : 0u; }
MOE_RING_FN uint32_t ring_place(uint32_t x, uint32_t slots) { return x % slots; }
MOE_RING_FN uint32_t ring_parity(uint32_t x, uint32_t slots) { return (x / slots) & 1u; }

}  // namespace moe
