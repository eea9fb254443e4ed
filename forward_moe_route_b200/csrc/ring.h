// The copies of a ring in shared memory that are still in flight when a wait has
// run out.  Plain C++, so that a host program can step through it.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

// A ring of `stages` slots is filled in turn; copy number k goes to slot
// k % stages and completes the phase of that slot's barrier whose parity is
// (k / stages) & 1.  `next` and `parity` are those of the first copy that was not
// issued.  A block may not leave shared memory to the next one while a copy is
// on its way: wait(slot, parity) is called for each slot with the parity of the
// last copy issued to it, or of the phase before a barrier's first where there was
// none, which counts as complete.
template <class Wait>
MOE_HD void ring_drain(int next, uint32_t parity, int stages, Wait wait) {
#ifdef __CUDACC__
#pragma unroll 1
#endif
  for (int s = 0; s < stages; ++s) wait(s, s < next ? parity : parity ^ 1u);
}

// `parity` of ring_drain for a reader that is at slot `at`, in a phase of parity
// `reading`, when the ring is filled up to slot `next` and holds at least one copy
MOE_HD uint32_t ring_parity(int next, int at, uint32_t reading) {
  return next > at ? reading : reading ^ 1u;
}

}  // namespace moe
