// tree.h -- launch interface of the kernel that lays out trees of drafted tokens.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

// Mask rows ([T, words], words at most 32) and positions of the nodes whose
// parents are given: see fa_tree_plan_window.
cudaError_t launch_tree_plan(const int* parents, const int* cu_q, const int* seq_k, int B, int T, uint32_t* mask, int words,
                             int* positions, int window, int sinks, int* err, cudaStream_t stream);

}  // namespace fa
