// tq_ring.cuh -- a ring of shared-memory stages filled by bulk copies, item i
// into stage i % stages: what a thread block that gives up has to wait for.
// The host compiles it too.
#pragma once

namespace tq {

#ifdef __CUDACC__
__host__ __device__ __forceinline__
#else
inline
#endif
// The parity of the phase that the last of `issued` items of a stage completes
// on its barrier, -1 if it had none. `issued` has to be what was issued: waiting
// for an item that was not can end at once, on the phase before the one whose
// copies are still in flight.
int last_phase(int issued, int stage, int stages) {
  return issued > stage ? ((issued - 1 - stage) / stages) & 1 : -1;
}

}  // namespace tq
