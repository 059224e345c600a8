// Untiled bulk copies between global and shared memory, for rings of stages that single warps own
// (addresses and sizes are multiples of 16 bytes; waits are those of tc_gemm.cuh, bounded in time), and
// the two ends of a launch that begins before the kernel ahead of it has ended.
#pragma once

#include "tc_gemm.cuh"

namespace fckl {

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

// Lets the next kernel of the stream begin, if it was launched to do so (launch_after), once every block
// of this one has come here or ended.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Returns when the kernel ahead has ended and its writes are visible: before the first access to memory.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace fckl
