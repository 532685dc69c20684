// Loads from memory straight into LDS (global_load_lds: 16 bytes a lane, lane L of a
// wave lands at lds_addr + 16 L), as the experts' products have them.  Inline assembly that the
// compiler does not track: whoever issues such loads waits for them with
// wait_barrier, also before the block ends.  An SALU write of M0 needs one
// wait state before the load reads it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

__device__ __forceinline__ void lds_dma16(const void* gaddr, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(gaddr), "s"(lds_addr) : "memory", "m0");
}
__device__ __forceinline__ void lds_dma16_s(const void* sbase, uint32_t voff, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(voff), "s"(sbase), "s"(lds_addr) : "memory", "m0");
}
// Wait until at most N of this wave's loads are outstanding, then block barrier.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(N) : "memory");
}

}  // namespace moe
