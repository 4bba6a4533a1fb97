// paged.cu -- the small kernels around paged attention: the join of cut
// units, and the write of new tokens into the cache with rotary positions.
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa.h"
#include "paged.h"
#include "paged_search.cuh"
#include "ptx_window.cuh"

namespace fa {
namespace {

// ---------------------------------------------------------------- join --
// Softmax over disjoint key sets is the LSE-weighted mean of the parts: with
// m = max_s LSE_s and w_s = e^(LSE_s - m), O = sum_s w_s O_s / sum_s w_s and
// LSE = m + ln sum_s w_s, summed in a fixed order.  Lane l holds columns l*E
// .. l*E+E-1 of a row.  A unit cut in a few parts (chunks: up to 256 rows, two
// or three parts) takes a warp per two rows; of one cut in many (a long
// context: as many parts as the GPU has SMs per head) a block takes up to
// eight rows at once, so that its rows take few rounds, and each row's share
// of the warps splits the parts and meets in shared memory.  The parts were
// just written and lie in L2, and what is left is latency: the loads of a
// row's parts go out before the weights they meet are known, and the blocks of
// a call with few units go to its cut units alone.
//   d = 128, one sequence of 12000 keys, 32/2 heads, 8 new tokens (128 rows
//   per head): 15.2 us in all; 25.0 with blocks spread over all CTAs' units, 40.9
//   with a whole block for one row after the other.  (Ranking the cut units
//   costs 0.5 us, so calls with many units or few rows keep a block per CTA.)
constexpr int kFewParts = 4;
constexpr int kThreads = 256;
constexpr int kMaxCtas = 2 * kThreads;

// x = columns lane*E .. of a row of parts
template <int E>
__device__ __forceinline__ void load_cols(float (&x)[E], const float* src) {
  if constexpr (E == 2) {
    *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(src);
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(x + e) = *reinterpret_cast<const float4*>(src + e);
  }
}

// e^(l - m), 0 for a part without visible keys (its columns are zeros); a part
// of a NaN row has weight NaN, and the row stays NaN
__device__ __forceinline__ float part_weight(float l, float m) { return l == -INFINITY ? 0.0f : expf(l - m); }

// (No pointer is __restrict__: what is read through a const one that is may be read
// ahead of pdl_wait, by the compiler's choice.)
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) paged_combine_kernel(
    const float* o_part, const float* lse_part, const int4* desc, void* o, float* lse, int ctas, int slot_rows, int g, int Hq) {
  constexpr int E = D / 32;
  __shared__ float red[8][D];
  __shared__ float red_w[8];
  __shared__ int warp_cut[8];
  __shared__ int4 shared_u;
  __shared__ int shared_cta;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch();
  pdl_wait();  // the parts and desc are the previous kernel's
  int4 u;
  int cta = blockIdx.x;
  if (gridDim.x == ctas) {
    u = desc[cta];
  } else {
    // fewer units than CTAs: the k-th cut unit goes to blocks (k, y)
    int4 mine[2];
    uint32_t has[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = i * kThreads + threadIdx.x;
      mine[i] = c < ctas ? desc[c] : make_int4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) has[i] = __ballot_sync(0xffffffffu, mine[i].x != 0);
    if (lane == 0) warp_cut[warp] = __popc(has[0]) + __popc(has[1]);
    if (threadIdx.x == 0) shared_u = make_int4(0, 0, 0, 0);
    __syncthreads();
    int rank = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w)
      if (w < warp) rank += warp_cut[w];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (mine[i].x != 0 && rank + __popc(has[i] & ((1u << lane) - 1)) == blockIdx.x) {
        shared_u = mine[i];
        shared_cta = i * kThreads + threadIdx.x;
      }
      rank += __popc(has[i]);
    }
    __syncthreads();
    u = shared_u;
    cta = shared_cta;
  }
  const int parts = u.x, rows = u.w, slot0 = 2 * cta;
  if (parts == 0) return;
  auto at = [&](int s, int row) -> long long {
    return (long long)(s == 0 ? slot0 + 1 : slot0 + 2 * s) * slot_rows + row;
  };
  auto out_row = [&](int row) -> long long { return (long long)(u.y + row / g) * Hq + u.z * g + row % g; };
  if (parts <= kFewParts) {
    for (int row0 = (blockIdx.y * 8 + warp) * 2; row0 < rows; row0 += gridDim.y * 16) {
      float x[2][kFewParts][E], l[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = min(row0 + i, rows - 1);
        l[i] = lane < parts ? lse_part[at(lane, row)] : -INFINITY;
#pragma unroll
        for (int s = 0; s < kFewParts; ++s)
          if (s < parts) load_cols<E>(x[i][s], o_part + at(s, row) * D + lane * E);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (row0 + i >= rows) break;
        float m = l[i];
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        m = __shfl_sync(0xffffffffu, m, 0);  // (lanes 0 .. 3 hold all parts)
        const float w = lane < parts ? part_weight(l[i], m) : 0.0f;
        float acc[E], total = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll
        for (int s = 0; s < kFewParts; ++s) {
          if (s < parts) {
            const float ws = __shfl_sync(0xffffffffu, w, s);
            total += ws;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(ws, x[i][s][e], acc[e]);
          }
        }
        const float inv = total != 0.0f ? 1.0f / total : 0.0f;
        const long long r = out_row(row0 + i);
        uint32_t pk[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2)
          pk[e / 2] = F16 ? pack_f16x2(acc[e] * inv, acc[e + 1] * inv) : pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
        uint32_t* dst = reinterpret_cast<uint32_t*>(o) + r * (D / 2) + lane * (E / 2);
        if constexpr (E == 2) dst[0] = pk[0];
        else if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(pk);
        else *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<uint4*>(pk);
        if (lane == 0) lse[r] = total == 0.0f ? -INFINITY : m + logf(total);
      }
    }
    return;
  }
  constexpr int AHEAD = E <= 4 ? 8 : 4;  // parts in flight per warp
  // rows that the block takes at once: enough for one round, at most a row per warp
  int lg = 0;
  while (lg < 3 && (int)(gridDim.y << lg) < rows) ++lg;
  const int share = 8 >> lg;  // warps per row
  const int sub = warp / share, first = warp % share;
  for (int base = blockIdx.y; base < rows; base += gridDim.y << lg) {
    const int row = base + sub * gridDim.y;
    const bool valid = row < rows;
    float m = -INFINITY;
    float acc[E], wsum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    if (valid) {
      for (int s = lane; s < parts; s += 32) m = fmaxf(m, lse_part[at(s, row)]);
      for (int s0 = first; s0 < parts; s0 += share * AHEAD) {  // this warp's parts: s0, s0 + share, ...
        const int n = min(AHEAD, (parts - s0 + share - 1) / share);
        float x[AHEAD][E];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          if (i < n) load_cols<E>(x[i], o_part + at(s0 + share * i, row) * D + lane * E);
        const float l = lane < n ? lse_part[at(s0 + share * lane, row)] : -INFINITY;
        if (s0 == first) {
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        }
        const float w = lane < n ? part_weight(l, m) : 0.0f;
        wsum += w;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, i);
          if (i < n) {
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(wi, x[i][e], acc[e]);
          }
        }
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, d);
#pragma unroll
    for (int e = 0; e < E; ++e) red[warp][lane * E + e] = acc[e];
    if (lane == 0) red_w[warp] = wsum;
    __syncthreads();
    if (valid) {
      float total = 0.0f;
      for (int w = 0; w < share; ++w) total += red_w[sub * share + w];
      const float inv = total != 0.0f ? 1.0f / total : 0.0f;
      const long long r = out_row(row);
      for (int c = first * 32 + lane; c < D / 2; c += share * 32) {
        float x = 0.0f, y = 0.0f;
        for (int w = 0; w < share; ++w) {
          x += red[sub * share + w][2 * c];
          y += red[sub * share + w][2 * c + 1];
        }
        reinterpret_cast<uint32_t*>(o)[r * (D / 2) + c] =
            F16 ? pack_f16x2(x * inv, y * inv) : pack_bf16x2(x * inv, y * inv);
      }
      // (a row's first warp has a part, so its maximum is the row's)
      if (first == 0 && lane == 0) lse[r] = total == 0.0f ? -INFINITY : m + logf(total);
    }
    __syncthreads();  // red is read before the next rows' sums
  }
}

// -------------------------------------------------------------- append --
// All bytes: each new q, k and v row is read once and written once.  One
// block per token (and one that looks the token ranges over): its threads are
// D/16 column chunks (16 columns each: the two 8-column halves of 8 rotary
// pairs) times 128/(D/16) heads, so a thread loads the 8 angles of its chunk
// once and uses them for every head it takes.  The pair (a, b) becomes (a c - b s, a s + b c) in fp32, each
// product rounded before the sum, rounded once to the element type.
//   9125 tokens, 32 + 2 x 8 heads, d = 128, read out of one projection: 229 MB
//   in 37.5 us, 6.1 TB/s (0.90 of the measured copy rate; 39.6 us with four
//   rows in flight per thread, which cost registers and so blocks; 43.8 with
//   256 threads per token, whose second round is half empty).  64 tokens: 2.9
//   us, three dependent look-ups (sequence, lengths, page) behind the launch.

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&x));
  else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (F16) return pack_f16x2(lo, hi);
  else return pack_bf16x2(lo, hi);
}

template <int D, bool F16, int LAYOUT>  // LAYOUT 0: no rotation
__global__ void __launch_bounds__(128) cache_append_kernel(const AppendParams prm) {
  constexpr int CL = D / 16;        // column chunks
  constexpr int HL = 128 / CL;      // heads at a time
  constexpr int MORE = 2;           // rows in flight per thread (4 take 72 registers and leave fewer blocks: see above)
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 31;
  if (t == prm.T) {
    // the last block: token ranges that do not fit T, or go back (those that no
    // token lies in are nobody else's to find)
    bool bad = false;
    for (int b = threadIdx.x; b < prm.B; b += 128) {
      const int a = prm.cu_q[b], e = prm.cu_q[b + 1];
      bad |= a < 0 || e < a || e > prm.T;
    }
    if (bad) report_index(prm.err);
    return;
  }
  const int c = threadIdx.x % CL, h0 = threadIdx.x / CL;
  const bool turn = LAYOUT != 0 && c < prm.rope_dim / 16;
  // columns of the two 8-element pieces of this chunk
  const int x0 = LAYOUT == FA_ROPE_HALF && turn ? 8 * c : 16 * c;
  const int x1 = LAYOUT == FA_ROPE_HALF && turn ? prm.rope_dim / 2 + 8 * c : 16 * c + 8;
  const int rows = prm.Hq + 2 * prm.Hkv;
  auto source = [&](int r) -> const uint16_t* {
    if (r < prm.Hq) return prm.q + t * prm.q_stride + (long long)r * D;
    r -= prm.Hq;
    return r < prm.Hkv ? prm.k + t * prm.k_stride + (long long)r * D : prm.v + t * prm.v_stride + (long long)(r - prm.Hkv) * D;
  };
  uint4 u[MORE], w[MORE];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < MORE; ++i) {
      const int r = r0 + i * HL;
      if (r < rows) {
        const uint16_t* src = source(r);
        u[i] = *reinterpret_cast<const uint4*>(src + x0);
        w[i] = *reinterpret_cast<const uint4*>(src + x1);
      }
    }
  };
  // the first rows do not depend on where they go: their latency and that of
  // the three dependent look-ups (sequence, lengths, page) pass together
  load(h0);
  const int given = LAYOUT != 0 && prm.positions ? prm.positions[t] : 0;
  const int b = find_sequence(prm.cu_q, prm.B, t, lane);
  // (a range is cut to the T tokens there are, as fa_fwd_paged does)
  const int q0 = max(0, prm.cu_q[b]), q1 = min(prm.T, prm.cu_q[b + 1]);
  if (t < q0 || t >= q1) return;  // a row that belongs to no sequence
  const long long pos = (long long)prm.seq_k[b] - (q1 - q0) + (t - q0);
  const long long angle = LAYOUT != 0 && prm.positions ? given : pos;  // the row of the tables
  // device data that leads out of range: nothing is written for the token
  int page = -1;
  if (pos >= 0 && (pos >> prm.page_shift) < prm.max_pages && (LAYOUT == 0 || (angle >= 0 && angle < prm.rope_len)))
    page = prm.table[b * prm.table_stride + (pos >> prm.page_shift)];
  if ((unsigned)page >= (unsigned)prm.num_pages) {
    if (threadIdx.x == 0) report_index(prm.err);
    return;
  }
  float cs[8], sn[8];
  if (LAYOUT != 0 && turn) {
    const float4* pc = reinterpret_cast<const float4*>(prm.cos + angle * (prm.rope_dim / 2) + 8 * c);
    const float4* ps = reinterpret_cast<const float4*>(prm.sin + angle * (prm.rope_dim / 2) + 8 * c);
    *reinterpret_cast<float4*>(cs) = pc[0];
    *reinterpret_cast<float4*>(cs + 4) = pc[1];
    *reinterpret_cast<float4*>(sn) = ps[0];
    *reinterpret_cast<float4*>(sn + 4) = ps[1];
  }
  const long long slot = page * prm.page_stride + (pos & ((1 << prm.page_shift) - 1)) * prm.token_stride;
  for (int r0 = h0; r0 < rows; r0 += MORE * HL) {
    if (r0 != h0) load(r0);
#pragma unroll
    for (int j = 0; j < MORE; ++j) {
      const int r = r0 + j * HL;
      if (r >= rows) break;
      uint16_t* dst;
      if (r < prm.Hq) dst = prm.q_out + ((long long)t * prm.Hq + r) * D;
      else if (r < prm.Hq + prm.Hkv) dst = prm.k_pages + slot + (r - prm.Hq) * prm.head_stride;
      else dst = prm.v_pages + slot + (r - prm.Hq - prm.Hkv) * prm.head_stride;
      if (LAYOUT != 0 && turn && r < prm.Hq + prm.Hkv) {
        uint32_t uu[4] = {u[j].x, u[j].y, u[j].z, u[j].w}, ww[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
        float a[8], z[8];  // the pairs' first and second elements
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2<F16>(uu[i]), h = unpack2<F16>(ww[i]);
          if constexpr (LAYOUT == FA_ROPE_HALF) {
            a[2 * i] = f.x, a[2 * i + 1] = f.y, z[2 * i] = h.x, z[2 * i + 1] = h.y;
          } else {
            a[i] = f.x, z[i] = f.y, a[4 + i] = h.x, z[4 + i] = h.y;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = __fsub_rn(__fmul_rn(a[i], cs[i]), __fmul_rn(z[i], sn[i]));
          const float q = __fadd_rn(__fmul_rn(a[i], sn[i]), __fmul_rn(z[i], cs[i]));
          a[i] = p;
          z[i] = q;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (LAYOUT == FA_ROPE_HALF) {
            uu[i] = pack2<F16>(a[2 * i], a[2 * i + 1]);
            ww[i] = pack2<F16>(z[2 * i], z[2 * i + 1]);
          } else {
            uu[i] = pack2<F16>(a[i], z[i]);
            ww[i] = pack2<F16>(a[4 + i], z[4 + i]);
          }
        }
        u[j] = make_uint4(uu[0], uu[1], uu[2], uu[3]);
        w[j] = make_uint4(ww[0], ww[1], ww[2], ww[3]);
      }
      *reinterpret_cast<uint4*>(dst + x0) = u[j];
      *reinterpret_cast<uint4*>(dst + x1) = w[j];
    }
  }
}

template <int D, bool F16>
cudaError_t append_layout(const AppendParams& prm, int layout, cudaStream_t stream) {
  const unsigned grid = (unsigned)prm.T + 1;  // (the last block looks the token ranges over)
  if (layout == 0) cache_append_kernel<D, F16, 0><<<grid, 128, 0, stream>>>(prm);
  else if (layout == FA_ROPE_HALF) cache_append_kernel<D, F16, FA_ROPE_HALF><<<grid, 128, 0, stream>>>(prm);
  else cache_append_kernel<D, F16, FA_ROPE_INTERLEAVED><<<grid, 128, 0, stream>>>(prm);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& prm, int d, bool f16, int layout, cudaStream_t stream) {
  switch (d) {
    case 64: return f16 ? append_layout<64, true>(prm, layout, stream) : append_layout<64, false>(prm, layout, stream);
    case 128: return f16 ? append_layout<128, true>(prm, layout, stream) : append_layout<128, false>(prm, layout, stream);
    case 256: return f16 ? append_layout<256, true>(prm, layout, stream) : append_layout<256, false>(prm, layout, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_paged_combine(const float* o_part, const float* lse_part, const int4* desc, void* o, float* lse,
                                 int sms, int ctas, int max_units, int slot_rows, int max_rows, int g, int Hq, int d,
                                 bool f16, cudaStream_t stream) {
  // launched while the attention kernel still runs; it waits for it itself
  cudaLaunchConfig_t cfg = {};
  if (ctas > kMaxCtas) return cudaErrorInvalidValue;
  // a block per CTA and 16 rows of a unit cut in few parts, or one row of a
  // unit cut in many; with so few units that their blocks would leave SMs
  // idle, a block per unit and as many rows as fill the GPU four times
  const int few = (max_rows + 15) / 16, many = max_rows < 8 ? max_rows : 8;
  int x = ctas, y = few > many ? few : many;
  const int spread = 4 * sms / (max_units < ctas ? max_units : ctas);
  if (spread > y && max_rows > y) {
    x = max_units;
    y = spread < max_rows ? spread : max_rows;
  }
  cfg.gridDim = dim3((unsigned)x, (unsigned)y, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto kern) {
    return cudaLaunchKernelEx(&cfg, kern, o_part, lse_part, desc, o, lse, ctas, slot_rows, g, Hq);
  };
  switch (d) {
    case 64: return f16 ? go(paged_combine_kernel<64, true>) : go(paged_combine_kernel<64, false>);
    case 128: return f16 ? go(paged_combine_kernel<128, true>) : go(paged_combine_kernel<128, false>);
    case 256: return f16 ? go(paged_combine_kernel<256, true>) : go(paged_combine_kernel<256, false>);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
