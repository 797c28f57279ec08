// Warps that share a named barrier and can give up a wait leave it together.
#pragma once

#include <cstdint>

namespace rag {

// named_bar_sync that tells every thread whether one of them came with `leave`.
// Warps that share a named barrier and can give up a wait between its rounds
// have to leave together: one that just left would be missed at the next round,
// and bar.sync has no limit. So whoever gives up still comes to its next round,
// once, with `leave`, and whoever is told so leaves at that round; a warp that
// has no rounds left comes once more, for one that gave up meanwhile. Each then
// comes to every round up to the last one exactly once. (Against bar.sync it
// costs a step of the 8-bit attention 0.1-0.2 us of 8.4-35, the streamed append
// 0.8 of 101.6; a word in shared memory that names the round costs the same.)
__device__ __forceinline__ bool named_bar_leave(uint32_t id, uint32_t nthreads, bool leave) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"(uint32_t(leave))
      : "memory");
  return r != 0;
}
// How such a warp's run went: on to the next round, a wait of its own gave up
// (it owes a round), or it was told to leave.
enum class Run { kOn, kGaveUp, kTold };

}  // namespace rag
