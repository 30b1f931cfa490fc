// ring.cuh -- which waits cover the loads of a ring of stages.
//
// Loaders fill the stages of a ring in turn, each on its own: fill number i goes to stage
// i % stages and completes that stage's barrier in phase i / stages. A loader begins a
// fill only after the stage's last one was consumed, which takes every loader's part of
// it: the loaders are never a whole ring apart, and of all fills begun only the last
// `stages` can still be in flight.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define EM_RING __host__ __device__ __forceinline__
#else
#define EM_RING inline
#endif

namespace em {

// The first fill that may be in flight when the loader that is ahead has begun `begun`.
EM_RING uint32_t ring_first(uint32_t begun, uint32_t stages) { return begun > stages ? begun - stages : 0u; }
EM_RING uint32_t ring_stage(uint32_t fill, uint32_t stages) { return fill % stages; }
EM_RING uint32_t ring_parity(uint32_t fill, uint32_t stages) { return fill / stages & 1u; }

}  // namespace em
