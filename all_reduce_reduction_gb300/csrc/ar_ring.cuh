// The steps of a ring of stages that one warp fills and empties: which stage and which
// phase of the stage's barrier a step has, and what may still be on its way.
#pragma once

#include <stdint.h>

namespace ar {

struct RingSteps {
    uint32_t bits;                    // 2^bits stages
    uint32_t sent;                    // copies on their way or landed; of the sending lane
    uint32_t used;                    // steps waited for

    __host__ __device__ __forceinline__ uint32_t stage(uint32_t step) const {
        return step & ((1u << bits) - 1u);
    }
    __host__ __device__ __forceinline__ uint32_t parity(uint32_t step) const {
        return step >> bits & 1;
    }
    // The first step whose copy may not have landed.  A wait that gave up counts as a step
    // too, so `used` does not say: of each stage the last copy that was sent is looked at.
    __host__ __device__ __forceinline__ uint32_t oldest_open() const {
        return sent > 1u << bits ? sent - (1u << bits) : 0u;
    }
};

}  // namespace ar
