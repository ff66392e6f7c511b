// One lane of a converged warp, chosen by the hardware.
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

}  // namespace jab
