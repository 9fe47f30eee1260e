// kvk_chunk_stop.cuh -- what a stopped chunk attention still has to wait for: the loads that a
// pair of CTAs has in flight when a bounded wait has run out.
//
// Both CTAs of a pair load their halves of step i of a ring of `slots` slots, counted on the
// leader's barrier of slot i % slots: the leader arms a phase with both halves' bytes just ahead
// of its own loads.  A CTA issues step i only once step i - slots has been used, which takes both
// halves, so every phase but the last of each slot is complete, and the last `slots` steps issued
// by either CTA cover all that may be in flight.  A stop finds the CTAs at different steps, since
// each goes on until one of its own waits fails.  With the number of steps that each has issued,
// the leader completes what the other never will:
//   issued by both             its phase completes when the loads land
//   issued by the leader only  the other's bytes never come: counted as if they had
//   issued by the other only   the phase was never armed: armed with the other's bytes
// and then every phase that was used completes once the loads in flight have landed, none earlier.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KVK_STOP_FN __host__ __device__ __forceinline__
#else
#define KVK_STOP_FN inline
#endif

namespace kvk {
namespace chunk {

struct StopStep {
  int slot;
  uint32_t parity;   // of the step's phase of its barrier
  bool arm;          // the leader arrives and expects the other CTA's bytes
  bool complete;     // the leader counts the other CTA's bytes as landed
};

// The first step that may be in flight, after `own` steps of the leader and `peer` of the other.
KVK_STOP_FN int stop_first(int slots, int own, int peer) {
  const int top = own > peer ? own : peer;
  return top > slots ? top - slots : 0;
}
KVK_STOP_FN StopStep stop_step(int i, int slots, int own, int peer) {
  StopStep s;
  s.slot = i % slots;
  s.parity = (uint32_t)(i / slots) & 1u;
  s.arm = i >= own;
  s.complete = i < own && i >= peer;
  return s;
}

}  // namespace chunk
}  // namespace kvk
