// wc_ring.cuh -- which copies into a ring of stages may still be in flight.
#pragma once

#include <stdint.h>

#ifndef __CUDACC__
#define __host__
#define __device__
#endif

namespace wc {

// After `fills` copies into `stages` stages in turn: calls f(stage, parity) for the
// last copy into each stage that had one, oldest first. Copy k lies in stage
// k % stages and completes that stage's phase k / stages, which a wait names by its
// parity. Earlier copies into a stage have landed, or it could not have been filled
// again. A block may end only when these have landed as well, whichever of its roles
// gave up: its shared memory goes to another block.
template <typename F>
__host__ __device__ inline void ring_last_fills(uint32_t fills, uint32_t stages, F f) {
    for (uint32_t k = fills < stages ? 0u : fills - stages; k < fills; ++k)
        f(k % stages, (k / stages) & 1u);
}

}  // namespace wc
