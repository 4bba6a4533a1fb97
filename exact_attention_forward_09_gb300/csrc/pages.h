// pages.h -- launch interfaces of the kernels that move, share and hand out a
// cache's pages.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

// The rows of a cache as the copying kernels see them: "planes" are the keys
// and the values of each layer.
struct PageRows {
  uint16_t *k, *v;
  long long layer_stride, page_stride, head_stride, token_stride;  // elements
  int layers, heads, num_pages, page_shift;
};

struct PoolParams {
  int* refs;                // [num_pages] how many rows of the table hold a page; 0: free
  int* table;               // [rows, table_stride]
  long long table_stride;
  int max_pages, num_pages, page_shift;
  int rows;
  int* seq_k;               // [rows] tokens that a row holds pages for
  int* err;
};

// Rows of the table shrink or grow to want[row] tokens.
cudaError_t launch_pages_resize(const PoolParams& prm, const int* want, cudaStream_t stream);

// Row dst[f] becomes a copy of row src[f]; fresh[f]: see fa_pages_fork.
cudaError_t launch_pages_fork(const PoolParams& prm, const PageRows& rows, int d, const int* src, const int* dst, int* fresh, int n,
                              cudaStream_t stream);

// Pages src[i] to pages dst[i].
cudaError_t launch_cache_copy(const PageRows& rows, int d, const int* src, const int* dst, int n, int* err, cudaStream_t stream);

struct CompactParams {
  PageRows rows;
  const int *table, *first, *keep, *keep_n;
  long long table_stride, keep_stride;
  int max_pages, max_keep, B;
  int* seq_k_out;           // [B] first + keep_n
  int* err;
};
cudaError_t launch_cache_compact(const CompactParams& prm, int d, int sms, cudaStream_t stream);

constexpr int kMaxResizeRows = 49152;   // their first ranks lie in shared memory
constexpr int kMaxForkRows = 1 << 18;   // three bits each in shared memory
constexpr int kMaxForks = 16384;        // ranks in shared memory

}  // namespace fa
