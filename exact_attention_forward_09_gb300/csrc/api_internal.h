// api_internal.h -- what the C-ABI files share (defined in api.cu): device
// state, argument checks and TMA descriptor encoding.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa.h"

namespace fa {

// Checks that the current device is an sm_103 and gives its number and the
// library's error word on it.
fa_status internal_device_setup(int* dev, int** err);
int internal_sm_count(int dev);

// Sizes, pointers and scale of a dense forward call (*empty: nothing to do).
fa_status internal_check_common(const void* q, const void* k, const void* v, const void* o, const float* lse, int64_t B,
                                int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d, float scale, bool* empty);

// 3-D map over a contiguous [BH, N, d] tensor: boxes of 128 bytes x box_rows.
fa_status internal_encode_map(CUtensorMap* map, const void* base, CUtensorMapDataType dt, int elem_bytes, int64_t BH,
                              int64_t N, int64_t d, uint32_t box_rows);
// Map of `rank` dimensions with the given byte strides (of dimensions 1 ..
// rank - 1), 128-byte swizzle, out-of-range elements read as 0.
fa_status internal_encode_map_nd(CUtensorMap* map, const void* base, CUtensorMapDataType dt, int rank,
                                 const uint64_t* dims, const uint64_t* strides, const uint32_t* box);

// The failure injection asked for by fa_debug_inject (bit 0), consumed.
bool internal_take_inject();

}  // namespace fa
