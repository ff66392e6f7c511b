// What the roles of a warp-specialised kernel share: one elected lane, waits of whole warps, plain bulk copies.
#pragma once

#include "common.cuh"

namespace jab {

// True in exactly one lane.  Issuing the tensor-core and TMA instructions under this predicate instead
// of lane == 0 lets the compiler treat the region as warp-uniform and keep matrix descriptors in
// uniform registers: eight back-to-back MMAs took 116 clocks to issue against 404 (measured on an
// idle tensor pipe), less than the 512 they take to run.
JAB_DEVICE bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// mbar_wait by a whole warp, with one verdict for all lanes: after a wait that gave up in some lanes only
// (the phase completed between their last looks) the warp would split and its next warp-wide step never end.
JAB_DEVICE bool mbar_wait_warp(uint64_t* bar, uint32_t parity, const KernelGuard& g, volatile uint32_t* abort_flag,
                               uint32_t where) {
  const bool ok = mbar_wait(bar, parity, g, abort_flag, where);
  return __all_sync(0xffffffffu, ok);
}

// Global -> shared copy of a multiple of 16 bytes, both addresses 16-byte aligned.
JAB_DEVICE void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

}  // namespace jab
