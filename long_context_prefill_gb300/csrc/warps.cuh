// What the kernels whose warps have tasks of their own share beyond ptx.cuh: the thread that issues for its warp.
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

}  // namespace msa
