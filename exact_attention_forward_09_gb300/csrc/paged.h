// paged.h -- launch interfaces of the paged cache's small kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

// Joins the partial results of the units that attn_window_kernel<.., PAGED>
// cut: for CTA c with desc[c] = {parts, first token, kv head, rows}, part 0
// lies in slot 2 c + 1 and part s >= 1 in slot 2 (c + s); a slot holds
// slot_rows rows of o_part ([d] fp32) and lse_part.  Row r of the unit goes
// to token first + r / g, head kv_head * g + r % g of o [T, Hq, d] and lse
// [T, Hq].  max_units: the most units the call can have; max_rows: the rows a
// unit is expected to have at most (more are joined, if slower).
cudaError_t launch_paged_combine(const float* o_part, const float* lse_part, const int4* desc, void* o, float* lse,
                                 int sms, int ctas, int max_units, int slot_rows, int max_rows, int g, int Hq, int d,
                                 bool f16, cudaStream_t stream);

struct AppendParams {
  const uint16_t *q, *k, *v;   // new tokens: [T, heads, d], rows of a token contiguous
  uint16_t* q_out;             // [T, Hq, d], or null: no queries
  uint16_t *k_pages, *v_pages;
  long long q_stride, k_stride, v_stride;              // elements between tokens
  long long page_stride, head_stride, token_stride;    // of the pages, elements
  const int *table, *cu_q, *seq_k;
  long long table_stride;
  int max_pages, num_pages, page_shift;
  int B, T, Hq, Hkv;           // Hq = 0: no queries
  const float *cos, *sin;      // [rope_len, rope_dim / 2]; null: no rotation
  int rope_len, rope_dim;      // rope_dim: rotated columns, a multiple of 16
  const int* positions;        // [T] positions of the rotation; null: where the token is written
  int* err;
};
cudaError_t launch_cache_append(const AppendParams& prm, int d, bool f16, int rope_layout, cudaStream_t stream);

}  // namespace fa
