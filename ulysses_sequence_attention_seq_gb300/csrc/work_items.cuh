// work_items.cuh -- attention kernels whose blocks go on with the work of blocks
// that have not started (cluster launch control).
//
// The grid has one block per work item, longest first where the causal flag
// makes some longer.  A block that is resident asks for one that has not started
// while its own item still runs, so that the next item's facts, first tiles and
// rows arrive before it is done, and barriers, tensor memory and descriptors are
// set up once.  Who computes an item, never what, depends on the timing.
#pragma once

#include <stdint.h>

namespace ulysses {
namespace dev {

// A running block takes over one that has not started (cluster launch control):
// the 16-byte answer lands at `slot` and completes 16 bytes of `bar`'s
// transaction count.  Not to be asked again once the answer was "none".
__device__ __forceinline__ void take_block(uint32_t slot, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   slot),
               "r"(bar)
               : "memory");
}
// The blockIdx.x taken over, or -1.
__device__ __forceinline__ int taken_block(uint32_t slot) {
  uint64_t lo, hi;
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(lo), "=l"(hi) : "r"(slot) : "memory");
  uint32_t block;
  asm volatile(
      "{\n\t.reg .b128 answer;\n\t.reg .pred taken;\n\t"
      "mov.b128 answer, {%1, %2};\n\t"
      "mov.u32 %0, 0xffffffff;\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 taken, answer;\n\t"
      "@taken clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, answer;\n\t}"
      : "=r"(block)
      : "l"(lo), "l"(hi));
  return (int)block;
}

// A work item: its query tile (or pair of tiles; < 0: no item), head of the
// rank, rank * B + batch, first key tile and numbers of key tiles.
struct Item {
  int tile, j, rb, t0, nA, nB;
  float zero;  // 0 that the compiler does not know of
};
// Facts in shared memory, by the producer for every warp.
__device__ __forceinline__ void put_item(uint32_t at, const Item &it) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(it.tile), "r"(it.j), "r"(it.rb), "r"(it.t0)
               : "memory");
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %3};" ::"r"(at + 16), "r"(it.nA), "r"(it.nB), "r"(0) : "memory");
}
__device__ __forceinline__ Item get_item(uint32_t at) {
  Item it;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(it.tile), "=r"(it.j), "=r"(it.rb), "=r"(it.t0)
               : "r"(at)
               : "memory");
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(it.nA), "=r"(it.nB) : "r"(at + 16) : "memory");
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(it.zero) : "r"(at + 24) : "memory");
  return it;
}

}  // namespace dev
}  // namespace ulysses
