// paged.cu -- the small kernels around paged attention: the join of cut
// units, and the write of new tokens into the cache with rotary positions.
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa.h"
#include "paged.h"
#include "ptx.cuh"

namespace fa {
namespace {

// ---------------------------------------------------------------- join --
// Softmax over disjoint key sets is the LSE-weighted mean of the parts: with
// m = max_s LSE_s and w_s = e^(LSE_s - m), O = sum_s w_s O_s / sum_s w_s and
// LSE = m + ln sum_s w_s.  One block per row of a cut unit: its 8 warps take
// the parts in turn (a single long context is cut into as many parts as half
// the GPU has SMs), lane l holding columns l*E .. l*E+E-1, and meet in shared
// memory in a fixed order.
template <int D, bool F16>
__global__ void __launch_bounds__(256) paged_combine_kernel(const float* __restrict__ o_part,
                                                            const float* __restrict__ lse_part,
                                                            const int4* __restrict__ desc, void* __restrict__ o,
                                                            float* __restrict__ lse, int slot_rows, int g, int Hq) {
  constexpr int E = D / 32;
  __shared__ float red[8][D];
  __shared__ float red_w[8];
  const int4 u = desc[blockIdx.x];
  const int parts = u.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int row = blockIdx.y; parts > 0 && row < u.w; row += gridDim.y) {
    auto at = [&](int s) -> long long {
      const long long slot = s == 0 ? 2LL * blockIdx.x + 1 : 2LL * (blockIdx.x + s);
      return slot * slot_rows + row;
    };
    float m = -INFINITY;
    for (int s = lane; s < parts; s += 32) m = fmaxf(m, lse_part[at(s)]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float acc[E], wsum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    for (int s = warp; s < parts; s += 8) {
      const float ls = lse_part[at(s)];
      if (ls == -INFINITY) continue;  // a run without visible keys; a NaN row stays NaN
      const float w = expf(ls - m);
      wsum += w;
      const float* src = o_part + at(s) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 x = *reinterpret_cast<const float2*>(src + e);
        acc[e] = fmaf(w, x.x, acc[e]);
        acc[e + 1] = fmaf(w, x.y, acc[e + 1]);
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) red[warp][lane * E + e] = acc[e];
    if (lane == 0) red_w[warp] = wsum;
    __syncthreads();
    const long long orow = (long long)(u.y + row / g) * Hq + u.z * g + row % g;
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) total += red_w[w];
    const float inv = total != 0.0f ? 1.0f / total : 0.0f;
    if (threadIdx.x < D / 2) {
      float a = 0.0f, b = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        a += red[w][2 * threadIdx.x];
        b += red[w][2 * threadIdx.x + 1];
      }
      reinterpret_cast<uint32_t*>(o)[orow * (D / 2) + threadIdx.x] =
          F16 ? pack_f16x2(a * inv, b * inv) : pack_bf16x2(a * inv, b * inv);
    }
    if (threadIdx.x == 0) lse[orow] = total == 0.0f ? -INFINITY : m + logf(total);
    __syncthreads();  // red is read before the next row's sums
  }
}

// -------------------------------------------------------------- append --
// All bytes: each new q, k and v row is read once and written once.  One
// block per token: its threads are D/16 column chunks (16 columns each: the
// two 8-column halves of 8 rotary pairs) times 256/(D/16) heads, so a thread
// loads the 8 angles of its chunk once and uses them for every head it
// takes.  The pair (a, b) becomes (a c - b s, a s + b c) in fp32, each
// product rounded before the sum, rounded once to the element type.

// the last b with cu[b] <= t, by 32-way search over cu[0 .. B-1]
__device__ __forceinline__ int find_sequence(const int* __restrict__ cu, int B, int t, int lane) {
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const uint32_t yes = __ballot_sync(0xffffffffu, i < n && cu[lo + i] <= t);
    const int last = yes == 0u ? 0 : 31 - __clz(yes);
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

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
__global__ void __launch_bounds__(256) cache_append_kernel(const AppendParams prm) {
  constexpr int CL = D / 16;        // column chunks
  constexpr int HL = 256 / CL;      // heads at a time
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int b = find_sequence(prm.cu_q, prm.B, t, lane);
  const int q0 = prm.cu_q[b], q1 = prm.cu_q[b + 1];
  if (t < q0 || t >= q1) return;  // a row that belongs to no sequence
  const long long pos = (long long)prm.seq_k[b] - (q1 - q0) + (t - q0);
  // device data that leads out of range: nothing is written for the token
  int page = -1;
  if (pos >= 0 && (pos >> prm.page_shift) < prm.max_pages && (LAYOUT == 0 || pos < prm.rope_len))
    page = prm.table[b * prm.table_stride + (pos >> prm.page_shift)];
  if ((unsigned)page >= (unsigned)prm.num_pages) {
    if (threadIdx.x == 0) atomicOr(prm.err, FA_DEVERR_INDEX);
    return;
  }
  const int c = threadIdx.x % CL, h0 = threadIdx.x / CL;
  // columns of the two 8-element pieces of this chunk
  const int x0 = LAYOUT == FA_ROPE_HALF ? 8 * c : 16 * c;
  const int x1 = LAYOUT == FA_ROPE_HALF ? D / 2 + 8 * c : 16 * c + 8;
  float cs[8], sn[8];
  if constexpr (LAYOUT != 0) {
    const float4* pc = reinterpret_cast<const float4*>(prm.cos + pos * (D / 2) + 8 * c);
    const float4* ps = reinterpret_cast<const float4*>(prm.sin + pos * (D / 2) + 8 * c);
    *reinterpret_cast<float4*>(cs) = pc[0];
    *reinterpret_cast<float4*>(cs + 4) = pc[1];
    *reinterpret_cast<float4*>(sn) = ps[0];
    *reinterpret_cast<float4*>(sn + 4) = ps[1];
  }
  const long long slot = page * prm.page_stride + (pos & ((1 << prm.page_shift) - 1)) * prm.token_stride;
  const int rows = prm.Hq + 2 * prm.Hkv;
  for (int r = h0; r < rows; r += HL) {
    const uint16_t* src;
    uint16_t* dst;
    bool turn = LAYOUT != 0;
    if (r < prm.Hq) {
      src = prm.q + t * prm.q_stride + (long long)r * D;
      dst = prm.q_out + ((long long)t * prm.Hq + r) * D;
    } else if (r < prm.Hq + prm.Hkv) {
      const int h = r - prm.Hq;
      src = prm.k + t * prm.k_stride + (long long)h * D;
      dst = prm.k_pages + slot + h * prm.head_stride;
    } else {
      const int h = r - prm.Hq - prm.Hkv;
      src = prm.v + t * prm.v_stride + (long long)h * D;
      dst = prm.v_pages + slot + h * prm.head_stride;
      turn = false;
    }
    uint4 u = *reinterpret_cast<const uint4*>(src + x0), w = *reinterpret_cast<const uint4*>(src + x1);
    if (turn) {
      uint32_t uu[4] = {u.x, u.y, u.z, u.w}, ww[4] = {w.x, w.y, w.z, w.w};
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
      u = make_uint4(uu[0], uu[1], uu[2], uu[3]);
      w = make_uint4(ww[0], ww[1], ww[2], ww[3]);
    }
    *reinterpret_cast<uint4*>(dst + x0) = u;
    *reinterpret_cast<uint4*>(dst + x1) = w;
  }
}

template <int D, bool F16>
cudaError_t append_layout(const AppendParams& prm, int layout, cudaStream_t stream) {
  const unsigned grid = (unsigned)prm.T;
  if (layout == 0) cache_append_kernel<D, F16, 0><<<grid, 256, 0, stream>>>(prm);
  else if (layout == FA_ROPE_HALF) cache_append_kernel<D, F16, FA_ROPE_HALF><<<grid, 256, 0, stream>>>(prm);
  else cache_append_kernel<D, F16, FA_ROPE_INTERLEAVED><<<grid, 256, 0, stream>>>(prm);
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
                                 int ctas, int slot_rows, int max_rows, int g, int Hq, int d, bool f16,
                                 cudaStream_t stream) {
  const dim3 grid((unsigned)ctas, (unsigned)(max_rows < 32 ? max_rows : 32), 1);
  auto go = [&](auto kern) { kern<<<grid, 256, 0, stream>>>(o_part, lse_part, desc, o, lse, slot_rows, g, Hq); };
  switch (d) {
    case 64: f16 ? go(paged_combine_kernel<64, true>) : go(paged_combine_kernel<64, false>); break;
    case 128: f16 ? go(paged_combine_kernel<128, true>) : go(paged_combine_kernel<128, false>); break;
    case 256: f16 ? go(paged_combine_kernel<256, true>) : go(paged_combine_kernel<256, false>); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace fa
