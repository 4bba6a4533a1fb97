// rope.cu -- rotary positions: queries and keys turned (and their gradients
// turned back), and the tables of angles.
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa.h"
#include "ptx_window.cuh"
#include "rope.h"

namespace fa {
namespace {

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

// ---------------------------------------------------------------- rope --
// The pair (a, b) becomes (a c - b s, a s + b c) in fp32, each product rounded
// before the sum, rounded once to the element type.  The inverse takes -s: the
// transpose of the same matrix, and so its gradient (also where the tables carry
// an amplitude).
//
// All bytes: every element is read once and written once.  A thread has 16
// columns of one token, as two 8-column pieces r/2 apart, so that in both layouts
// a row's threads read whole runs of 16-byte pieces (half: the pieces are the
// pairs' first and second elements; interleaved: four pairs each).  It loads their
// eight angles once and takes one head after the other, so the tables are read
// once per block and not once per head; a block is 256/(d/16) tokens in a row,
// which lie together in either order of heads and tokens.  The first rows' loads
// go out before the position and its angles are known.
//   2 x 8192 tokens, 16 + 4 heads, d = 128: 168 MB in 27.4 us, 6.1 TB/s (0.90 of the
//   measured copy rate; 29.2 with four rows in flight; forward and back in a stream
//   56.2 us, 60.5 where each is launched at the end of the one before); 8 x 4096 of 32 + 8 heads
//   103 us, 6.5 TB/s; 64 columns of d = 256 in place 15.6 us where copying the others
//   takes 22.8; 65 tokens 2.3 us.
constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 2;  // rows in flight per thread (four take 80 registers and leave three blocks to an SM)

template <int D, bool F16, int LAYOUT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams prm, const float sign) {
  constexpr int CL = D / 16;  // column chunks of a row
  constexpr int TB = kRopeThreads / CL;
  pdl_launch();  // (the gradients' rotation, say, may be launched; it waits for this kernel's end)
  pdl_wait();
  const int c = threadIdx.x % CL;
  const int batch = blockIdx.x / prm.tiles;
  const int n = (blockIdx.x - batch * prm.tiles) * TB + threadIdx.x / CL;
  if (n >= prm.N) return;
  const bool turn = c < prm.r / 16;
  const int x0 = turn ? 8 * c : prm.r + 8 * (c - prm.r / 16);
  const int x1 = x0 + (turn ? prm.r / 2 : (D - prm.r) / 2);
  const int h0 = blockIdx.y * prm.heads_per_block, h1 = min(h0 + prm.heads_per_block, prm.heads);
  auto array = [&](int& h) -> const RopeArray& {
    if (h < prm.a[0].heads) return prm.a[0];
    h -= prm.a[0].heads;
    return prm.a[1];
  };
  uint4 u[kRopeRows], w[kRopeRows];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i) {
      int k = h + i;
      if (k < h1) {
        const RopeArray& a = array(k);
        const uint16_t* src = a.x + batch * a.x_batch + k * a.x_head + n * a.x_token;
        if (turn || !a.same) {
          u[i] = *reinterpret_cast<const uint4*>(src + x0);
          w[i] = *reinterpret_cast<const uint4*>(src + x1);
        }
      }
    }
  };
  load(h0);
  const int pos = prm.positions ? prm.positions[batch * prm.pos_stride + n] : prm.offset + n;
  if ((unsigned)pos >= (unsigned)prm.rope_len) {  // (device data: the row is left as it is)
    if (c == 0) report_index(prm.err);
    return;
  }
  // half: the angles of pairs x0 .. x0 + 7; interleaved: of x0/2 .. x0/2 + 3 and x1/2 .. x1/2 + 3
  float cs[8], sn[8];
  if (turn) {
    const long long row = (long long)pos * (prm.r / 2);
    const int p0 = LAYOUT == FA_ROPE_HALF ? x0 : x0 / 2, p1 = LAYOUT == FA_ROPE_HALF ? x0 + 4 : x1 / 2;
    *reinterpret_cast<float4*>(cs) = *reinterpret_cast<const float4*>(prm.cos + row + p0);
    *reinterpret_cast<float4*>(cs + 4) = *reinterpret_cast<const float4*>(prm.cos + row + p1);
    *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(prm.sin + row + p0);
    *reinterpret_cast<float4*>(sn + 4) = *reinterpret_cast<const float4*>(prm.sin + row + p1);
#pragma unroll
    for (int i = 0; i < 8; ++i) sn[i] *= sign;
  }
  for (int h = h0; h < h1; h += kRopeRows) {
    if (h != h0) load(h);
#pragma unroll
    for (int j = 0; j < kRopeRows; ++j) {
      int k = h + j;
      if (k >= h1) break;
      const RopeArray& a = array(k);
      if (!turn && a.same) continue;
      uint16_t* dst = a.y + batch * a.y_batch + k * a.y_head + n * a.y_token;
      if (turn) {
        uint32_t uu[4] = {u[j].x, u[j].y, u[j].z, u[j].w}, ww[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
        auto pair = [&](float& p, float& q, int i) {
          const float y = __fsub_rn(__fmul_rn(p, cs[i]), __fmul_rn(q, sn[i]));
          q = __fadd_rn(__fmul_rn(p, sn[i]), __fmul_rn(q, cs[i]));
          p = y;
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 f = unpack2<F16>(uu[i]), g = unpack2<F16>(ww[i]);
          if constexpr (LAYOUT == FA_ROPE_HALF) {
            pair(f.x, g.x, 2 * i);
            pair(f.y, g.y, 2 * i + 1);
          } else {
            pair(f.x, f.y, i);
            pair(g.x, g.y, 4 + i);
          }
          uu[i] = pack2<F16>(f.x, f.y);
          ww[i] = pack2<F16>(g.x, g.y);
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
cudaError_t rope_layout(const RopeParams& prm, dim3 grid, int layout, float sign, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRopeThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return layout == FA_ROPE_HALF ? cudaLaunchKernelEx(&cfg, rope_kernel<D, F16, FA_ROPE_HALF>, prm, sign)
                                : cudaLaunchKernelEx(&cfg, rope_kernel<D, F16, FA_ROPE_INTERLEAVED>, prm, sign);
}

// --------------------------------------------------------------- table --
// The angle of pair i at position p is p f_i turns.  With f_i as a 64-bit
// fraction of a turn the product's whole turns fall off the top of a 64-bit
// integer, so its reduction is exact at any position: what is left of the angle
// carries the frequency's own error (the host rounds it to the nearest, 2^-65 turns,
// times p) alone, where an fp32 product would be off by p 2^-24 radians.  The nearest quarter turn is split off as
// two bits, and what remains (at most an eighth of a turn, exact in 62 bits) is
// rounded to fp32 relative to itself, so that values near zero keep their digits.
// A thread keeps four pairs and steps through positions by adding; two blocks to
// an SM, as a thread's start (four 64-bit products, frequencies at addresses that
// differ within the warp) costs as much as some positions (eight blocks: +1.3 us).
//   Instructions bound it: 131072 positions of 64 pairs in 12.4 us, 5.4 TB/s (a
//   fill of as many bytes takes 9.6); 16.5 with a conversion from 64 bits, which has
//   a small part of the rate of one from 32, and 17.9 with the library's sincospif.
constexpr int kTableThreads = 256, kTableBlocks = 2;

__device__ __forceinline__ void turn_of(uint64_t t, float& c, float& s) {
  const uint32_t h = (uint32_t)(t >> 32) + 0x20000000u;  // bits 31, 30: the nearest quarter turn
  const int top = (int)(h & 0x3fffffffu) - 0x20000000;   // the rest's upper word
  // The rest in half turns, at most a quarter, rounded once: its upper 24 bits are
  // exact in fp32, and the 32 behind them add to them.
  const float x = fmaf((float)(top >> 6), 0x1p-25f, (float)__funnelshift_r((uint32_t)t, (uint32_t)top, 6) * 0x1p-57f);
  // sin(pi x) and cos(pi x): polynomials in x^2 that are nearest to them over this
  // range (fitted by weighted least squares, the weights moved toward the largest
  // errors as Lawson's method does), with these coefficients to 1.3e-9 and 9.1e-9 (a
  // unit of fp32 just below 1 is 6e-8); pi in two parts
  const float u = x * x;
  const float ps = fmaf(u, fmaf(u, fmaf(u, fmaf(u, 0.0812298f, -0.59922882f), 2.5501636f), -5.1677128f), -8.7422777e-8f);
  const float pc = fmaf(u, fmaf(u, fmaf(u, 0.23212635f, -1.3351379f), 4.0587106f), -4.9348022f);
  const float a = fmaf(x, 3.14159274f, x * ps), b = fmaf(u, pc, 1.0f);
  // an odd quarter swaps the two; the sine's sign is the quarter's upper bit, the
  // cosine's that and the lower one
  const bool odd = h & 0x40000000u;
  c = __uint_as_float(__float_as_uint(odd ? a : b) ^ ((h ^ (h << 1)) & 0x80000000u));
  s = __uint_as_float(__float_as_uint(odd ? b : a) ^ (h & 0x80000000u));
}

template <bool AMP>  // whether there is an amplitude other than 1
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const __grid_constant__ RopeTableParams prm) {
  const int groups = prm.half / 4;                 // threads of a position
  const int per = kTableThreads / groups;          // positions of a block at a time
  const int g = threadIdx.x % groups;
  if ((int)threadIdx.x >= per * groups) return;
  long long p = (long long)blockIdx.x * per + threadIdx.x / groups;
  const long long step = (long long)gridDim.x * per;
  uint64_t t[4], dt[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t f = prm.turns[4 * g + i];
    t[i] = f * (uint64_t)(prm.start + p);
    dt[i] = f * (uint64_t)step;
  }
  for (; p < prm.n; p += step) {
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn_of(t[i], c[i], s[i]);
      t[i] += dt[i];
      if constexpr (AMP) {
        // rounded once
        c[i] = fmaf(c[i], prm.amp_hi, c[i] * prm.amp_lo);
        s[i] = fmaf(s[i], prm.amp_hi, s[i] * prm.amp_lo);
      }
    }
    const long long at = p * prm.half + 4 * g;
    *reinterpret_cast<float4*>(prm.cos + at) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(prm.sin + at) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

}  // namespace

cudaError_t launch_rope(RopeParams prm, int64_t B, int d, bool f16, int layout, bool inverse, int sms, cudaStream_t stream) {
  const int tb = kRopeThreads / (d / 16);
  prm.tiles = (prm.N + tb - 1) / tb;
  const int64_t blocks = B * prm.tiles;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  // As many heads to a block as leave 16 blocks per SM, so that a small call
  // spreads over the GPU and a large one reads its angles seldom.
  int64_t groups = (16LL * sms + blocks - 1) / blocks;
  if (groups > prm.heads) groups = prm.heads;
  if (groups < 1) groups = 1;
  prm.heads_per_block = (int)((prm.heads + groups - 1) / groups);
  if (prm.heads_per_block < (prm.heads + 65534) / 65535) prm.heads_per_block = (prm.heads + 65534) / 65535;
  const dim3 grid((unsigned)blocks, (unsigned)((prm.heads + prm.heads_per_block - 1) / prm.heads_per_block), 1);
  const float sign = inverse ? -1.0f : 1.0f;
  switch (d) {
    case 64: return f16 ? rope_layout<64, true>(prm, grid, layout, sign, stream) : rope_layout<64, false>(prm, grid, layout, sign, stream);
    case 128: return f16 ? rope_layout<128, true>(prm, grid, layout, sign, stream) : rope_layout<128, false>(prm, grid, layout, sign, stream);
    case 256: return f16 ? rope_layout<256, true>(prm, grid, layout, sign, stream) : rope_layout<256, false>(prm, grid, layout, sign, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_rope_table(const RopeTableParams& prm, int sms, cudaStream_t stream) {
  const int per = kTableThreads / (prm.half / 4);
  int64_t blocks = ((int64_t)prm.n + per - 1) / per;
  if (blocks > kTableBlocks * (int64_t)sms) blocks = kTableBlocks * (int64_t)sms;  // (then each steps on)
  if (prm.amp_hi == 1.0f && prm.amp_lo == 0.0f) rope_table_kernel<false><<<(unsigned)blocks, kTableThreads, 0, stream>>>(prm);
  else rope_table_kernel<true><<<(unsigned)blocks, kTableThreads, 0, stream>>>(prm);
  return cudaGetLastError();
}

}  // namespace fa
