// ptx_window.cuh -- what the windowed and paged kernels need beside ptx.cuh:
// 4-D TMA loads, dependent launches, one more device error.
#pragma once

#include "ptx.cuh"

namespace fa {

// An index read from device memory was out of range.  Kept in the word behind the
// one of FA_DEVERR_TIMEOUT, so that neither error hides the other.  (As two bits
// of one word the waits need an atomic OR where they have an exchange, which alone
// makes the windowed kernels 0.7 to 2% slower: 16384 tokens, 8/2 heads, window 4096,
// 169.2 -> 172.3 us; 4 x 2048 tokens over 4000 to 10000 keys 581 -> 592.)
enum : int { FA_DEVERR_INDEX = 1 };
__device__ __forceinline__ void report_index(int* err) { atomicOr(err + 1, FA_DEVERR_INDEX); }

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

// ------------------------------------------------------------- clusters --
__device__ __forceinline__ int cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return (int)n;
}
// Every thread of every CTA of the cluster; orders shared-memory accesses.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address, in the cluster's window, of a shared-memory address in CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

}  // namespace fa
