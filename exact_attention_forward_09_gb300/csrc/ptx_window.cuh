// ptx_window.cuh -- what the windowed and paged kernels need beside ptx.cuh:
// 4-D TMA loads, dependent launches, one more device error.
#pragma once

#include "ptx.cuh"

namespace fa {

// Device error word: a bit of its own beside FA_DEVERR_TIMEOUT, for an index
// read from device memory that was out of range.
enum : int { FA_DEVERR_INDEX = 2 };

// tma_load_3d_hint for a 4-D map.
__device__ __forceinline__ void tma_load_4d_hint(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                                 int c1, int c2, int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}

// In a kernel launched with programmatic stream serialisation: waits until
// the kernel before it in the stream has ended and its writes are visible
// (returns at once otherwise).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel of the stream be launched, if it was asked for so,
// once every CTA of this one has come here or ended.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace fa
