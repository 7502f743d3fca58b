// Bounded waits of the kernels whose roles are whole warps.
//
// A wait that gives up on its own limit may end with one answer in one lane and
// another in the next: the lanes poll one after another, and the barrier can
// complete, or another role can fail, between two of them.  What follows a wait
// is for whole warps (__syncwarp, votes, tcgen05.ld), so lanes that part there
// wait for each other for good.  The warp forms therefore vote: every lane gets
// the same answer, and a warp of which one lane gave up gives up.
//
// Uses mbar_try_wait and global_timer_ns of dsa_common.cuh.
#pragma once

namespace dsa {

// a bounded wait of a converged warp, which also gives up as soon as another role
// has failed; every step is the whole warp's
__device__ __forceinline__ bool wait_or_fail(uint64_t *bar, uint32_t parity, uint64_t limit_ns,
                                             volatile uint32_t *failed) {
  // the first tries do without the timer, whose reading takes hundreds of cycles
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *failed != 0u || global_timer_ns() - t0 > limit_ns)) {
      *failed = 1u;
      return false;
    }
  }
}
// whether any role has failed, the same answer in every lane of a converged warp
__device__ __forceinline__ bool warp_failed(const volatile uint32_t *failed) {
  return __any_sync(0xffffffffu, *failed != 0u) != 0;
}

}  // namespace dsa
