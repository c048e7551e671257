// What the kernels whose warps have tasks of their own share beyond ptx.cuh: the thread that issues for its warp, and a
// wait that leaves the issue slots to the warps that work.
#pragma once
#include "ptx.cuh"

namespace msa {

// One thread of a converged warp, the same one each time.  Products are issued under this predicate: with one that the
// compiler cannot tell to hold for a single thread (lane == 0) it serialises each issue over the lanes, 66 cycles a
// product where these take 15 to 40 (M = 128, N = 16 to 64).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// mbar_wait whose polls suspend for a while each (a hint of kSuspendNs; 3.8 us were measured on a barrier that nothing
// reaches): polls of warps that wait would take a third of the issue slots from those that work.  Gives up once *gave_up
// is set (nullptr: never) or limit_ns have passed since the first kPollsAtATime polls, looking at both that often.
constexpr uint32_t kSuspendNs = 1000, kPollsAtATime = 16;
__device__ __forceinline__ bool mbar_wait_long(uint64_t* bar, uint32_t parity, const volatile uint32_t* gave_up,
                                               uint64_t limit_ns = MSA_WAIT_LIMIT_NS) {
  uint64_t since = 0;
  for (uint32_t polls = 1;; ++polls) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendNs)
        : "memory");
    if (ok) return true;
    if (polls % kPollsAtATime == 0) {
      const uint64_t now = global_timer_ns();
      if (gave_up && *gave_up) return false;
      if (since == 0) since = now;
      else if (now - since > limit_ns) return false;
    }
  }
}

}  // namespace msa
