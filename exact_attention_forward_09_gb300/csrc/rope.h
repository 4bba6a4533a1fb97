// rope.h -- launch interfaces of the rotary position kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

// One array that is turned: element (b, h, n, c) of x lies at x + b * x_batch
// + h * x_head + n * x_token + c (16-bit elements), of y likewise.
struct RopeArray {
  const uint16_t* x;
  uint16_t* y;
  long long x_batch, x_head, x_token;
  long long y_batch, y_head, y_token;
  int heads;
  int same;            // y is x: columns behind the rotated ones are not touched
};

struct RopeParams {
  RopeArray a[2];      // the heads of both are taken as one list
  int heads;           // a[0].heads + a[1].heads
  int heads_per_block;
  int N, tiles;        // tokens per batch entry, blocks of tokens they make
  int r;               // rotated columns
  const int* positions;  // of token n of entry b at b * pos_stride + n; null: offset + n
  long long pos_stride;
  int offset;
  const float *cos, *sin;  // [rope_len, r / 2]
  int rope_len;
  int* err;
};
cudaError_t launch_rope(RopeParams prm, int64_t B, int d, bool f16, int layout, bool inverse, int sms, cudaStream_t stream);

struct RopeTableParams {
  float *cos, *sin;        // [n, half]
  int n, half;             // positions, pairs
  uint32_t start;          // the first position
  float amp_hi, amp_lo;    // the amplitude in two parts
  uint64_t turns[128];     // 2^64 times the turns per position of each pair
};
cudaError_t launch_rope_table(const RopeTableParams& prm, int sms, cudaStream_t stream);

}  // namespace fa
