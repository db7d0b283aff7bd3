// ring.cuh — the copies of a ring of shared-memory slots that may still be in flight.
#pragma once
#include <cstdint>

namespace jattn {

// Copy i of a ring fills slot i % slots and completes phase i / slots of the slot's
// barrier.  Calls wait(slot, parity) so that, when those waits have returned, each
// of `issued` copies has landed: by a barrier's phase, or by a wait that runs out its
// limit.  own: the copies complete on this CTA's barriers.  If not (the second CTA of
// a pair, whose copies complete on the first one's), its own barriers stay in their
// first phase, in which a wait for parity 1 returns at once and one for parity 0 runs
// out its limit: one such wait.
template <typename Wait>
__host__ __device__ __forceinline__ void drain_ring(int issued, int slots, bool own, Wait wait) {
  if (issued == 0) return;
  if (!own) {
    wait(0, 0u);
    return;
  }
  for (int i = issued > slots ? issued - slots : 0; i < issued; ++i)
    wait(i % slots, static_cast<uint32_t>(i / slots) & 1u);
}

}  // namespace jattn
