// attn_bwd.h -- launch interface of the attention backward kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

struct BwdParams {
  float* dq_acc;       // [BHq, Nq, D] fp32, zeroed by the preprocessing kernel (added to through tm dq_acc)
  void* dk;            // [BHkv, Nk, D] bf16 / f16
  void* dv;            // [BHkv, Nk, D]
  // [BHq, nrec, 2, 64]: per 64-row record, -LSE_i * log2(e) (-inf for a
  // row with no key or past Nq) then -D_i (0 past Nq)
  const float* vecs;
  int nrec;            // records per query head (whole kernel steps)
  int* err;            // device error word
  int Nq, Nk;          // query rows / keys per head
  int Hq, Hkv;         // heads (Hq % Hkv == 0)
  int BHkv;            // batch x key/value heads
  float scale_log2;    // scale * log2(e)
  float scale;         // dK = scale * dS^T Q
  int drop_step;       // test hook: step whose Q/dO stage CTA 0 never fills (-1: none)
  // sliding window with sinks (the WIN instances): see BwdWindow
  int window, sinks;
  int sink_tiles, sink_split;
  int split_kt, tile_split;  // tiles from split_kt on in tile_split (>= 2) shares
  // sink_split > 1: [sink_tiles][BHkv][sink_split][dK, dV][128][D] fp32, then
  // [tiles from split_kt on][BHkv][tile_split][dK, dV][128][D]
  float* part;
};

// How the windowed backward shares out its key tiles' query steps, over CTAs
// that leave fp32 dK and dV to be summed.  The tiles that hold a sink are seen
// by every query from their first key on, the others by about window / 128 + 1
// query tiles: `split` shares of each of the first, `tile_split` of the others
// from tile split_kt on.
struct BwdWindow {
  int window, sinks;
  int sink_tiles, split;
  int split_kt, tile_split;
  size_t part_bytes;
};
BwdWindow bwd_window_plan(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int d, int64_t window,
                          int64_t sinks);

struct BwdLaunch {
  CUtensorMap q, dout;  // [BHq, Nq, D], 64-row boxes
  CUtensorMap k, v;     // [BHkv, Nk, D], 128-row boxes
  CUtensorMap dq_acc;   // fp32 [BHq, Nq, D], 32-column x step-row boxes, 128-byte swizzle
  CUtensorMap dk, dv;   // [BHkv, Nk, D], 128-row boxes (epilogue stores)
  BwdParams prm;
  cudaStream_t stream;
};

// ELEM: 0 bf16, 1 f16 (the forward's element kinds)
template <int ELEM, int D, bool CAUSAL, bool WIN = false>
cudaError_t launch_attn_bwd(const BwdLaunch& L);

// The end of the windowed backward: dq = RN(scale * dq_acc), and for the shared
// tiles (rows below Nk) dK = scale * sum of the shares' dK, dV = sum of theirs.
cudaError_t launch_bwd_window_finish(const BwdParams& prm, void* dq, long long elems, int d, bool f16,
                                     cudaStream_t stream);

// The rows of few keys.  D = dO . O carries O's rounding, which dS = P (dP - D)
// hands on to every key of a row, and which averages out over many keys only.  So
// under a window the rows that see at most 32 keys take D = sum_j P_j dP_j over
// them, in fp32: every row where window + sinks <= 32, in a preparation kernel of
// its own, else those at positions below 32, in blocks of their own.
// Relative error of dQ against 64 bits, bf16, 1000 tokens, d = 128, with dO . O and
// so (rounding dQ alone gives 1.66e-3): two keys to a row 3.74e-3 and 2.33e-3, 30
// and 2 sinks 2.47e-3 and 2.35e-3.  Cost: 0 within 0.5 us where only the first
// positions are such rows; where all are, 16/4 heads x 8192 rows, window 30, 2
// sinks, the backward takes 149 us instead of 119 (d = 64 92 instead of 81).
// blocks 0, not all: dO . O everywhere (fa_bwd).
struct BwdFewKeys {
  int blocks;
  int first, rows;  // rows first .. first + rows - 1 of every head
  bool all;         // every row
  const void *q, *k, *v, *dout;
  int Hq, Hkv, Nk;
  int window, sinks;
  float scale_log2;
};
// Which rows they are (a row before position 0 sees no key, and O = 0 gives it
// D = 0); the pointers, heads and scale are the caller's to fill in.
BwdFewKeys bwd_few_keys(int64_t BHq, int64_t Nq, int64_t Nk, int64_t window, int64_t sinks);

// Records of -LSE_i * log2(e) and -D_i (D_i = dO_i . O_i, see BwdFewKeys) for
// every query row, padded to nrec 64-row records per head, and dq_acc := 0.
cudaError_t launch_bwd_prep(const void* o, const void* dout, const float* lse, float* vecs, float* dq_acc,
                            long long bhq, int nq, int nrec, int d, bool f16, const BwdFewKeys& few,
                            cudaStream_t stream);

// Query rows per kernel step for head dimension d, and the records per
// query head the kernel reads (whole steps).
int bwd_step_rows(int d);
long long bwd_records_per_head(long long nq, int d);

// dq = RN(scale * dq_acc) in the element type.
cudaError_t launch_bwd_dq_convert(const float* dq_acc, void* dq, float scale, long long elems, bool f16,
                                  cudaStream_t stream);

// Zero `bytes` bytes (a multiple of 16, 16-byte aligned).
cudaError_t launch_zero_fill(void* p, long long bytes, cudaStream_t stream);

}  // namespace fa
