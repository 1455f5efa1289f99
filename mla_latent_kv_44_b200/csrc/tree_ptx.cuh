// Helpers shared by the tensor-core kernels of mla_decode_tree.
#pragma once

#include "tc_ptx.cuh"

namespace mla {
namespace {

// True in one lane of a converged warp. An MMA or a TMA load takes its operands from uniform
// registers; from a warp that runs the loop together they are at hand, from one thread in a
// divergent branch every operand is moved first (an MMA then took 132 cycles to issue against 25).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(p));
  return p != 0;
}

// Waits for a phase up to about 0.1 ms in hardware, which takes no issue slots from the warps that
// share the scheduler (a warp that polls does).
__device__ __forceinline__ bool mbar_try_long(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity), "r"(100000u) : "memory");
  return ok != 0;
}

// Shared-memory matrix descriptors of 128-byte swizzled slabs, 8-row groups 1024 bytes apart
// (as sdesc builds them): the high word is constant, the low word holds the start and the
// leading offset, and moves by bytes / 16.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3FFF) | ((lbo >> 4) << 16);
}

}  // namespace
}  // namespace mla
