// rope_api.cu -- the C ABI of the rotary position operators (declared in
// include/fa.h): argument checks, frequencies and launch on the caller's stream.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "fa.h"
#include "api_internal.h"
#include "rope.h"

namespace {

constexpr int64_t kMaxLen = (int64_t)1 << 30;
constexpr double kTurn = 6.283185307179586476925;  // 2 pi

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool rope_dim_ok(int64_t r, int64_t most) { return r >= 16 && r <= most && r % 16 == 0; }

// A number as the sum of two doubles, about 104 bits.  An angle far out is a
// frequency times its position, and so is its error: with a double's, 2^-53 of it,
// small sines near position 2^30 were off by 250 times what fa_rope_table states.
struct Two {
  double hi, lo;
};
Two sum(double a, double b) {  // exact
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
Two operator+(Two a, Two b) {
  const Two s = sum(a.hi, b.hi);
  return sum(s.hi, s.lo + (a.lo + b.lo));
}
Two operator-(Two a, Two b) { return a + Two{-b.hi, -b.lo}; }
Two operator*(Two a, Two b) {
  const double p = a.hi * b.hi;
  return sum(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
Two operator/(Two a, Two b) {
  const double q = a.hi / b.hi;
  return Two{q, 0.0} + Two{(a - b * Two{q, 0.0}).hi / b.hi, 0.0};
}
Two one(double x) { return {x, 0.0}; }

// x^(-1/n), x >= 1: a double, and one step of Newton's method for y^n x = 1, whose
// error is the square of the double's.
Two root(double x, int n) {
  const Two y = one(std::pow(x, -1.0 / n));
  Two p = one(x), square = y;
  for (int k = n; k > 0; k >>= 1, square = square * square)
    if (k & 1) p = p * square;
  return y - y * (p - one(1.0)) / one(n);
}

const Two kTurns = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / 2 pi

// The angle per position of pair i of r/2.
bool scaled_frequencies(int64_t r, double theta, const fa_rope_scaling* sc, Two* f) {
  const int half = (int)(r / 2);
  const int kind = sc ? sc->kind : FA_ROPE_SCALE_NONE;
  const double s = sc ? sc->factor : 1.0;
  if (!std::isfinite(theta) || theta <= 1.0) return false;
  if (kind < FA_ROPE_SCALE_NONE || kind > FA_ROPE_SCALE_INDEX) return false;
  if (sc && !std::isfinite((float)sc->amplitude)) return false;  // (the tables are fp32)
  if (kind != FA_ROPE_SCALE_NONE && (!std::isfinite(s) || s < 1.0)) return false;
  const bool parts = kind == FA_ROPE_SCALE_TURNS || kind == FA_ROPE_SCALE_INDEX;
  if (parts) {
    if (!std::isfinite(sc->original) || !std::isfinite(sc->low) || !std::isfinite(sc->high)) return false;
    if (sc->original < 1.0 || sc->low < 0.0 || sc->high <= sc->low) return false;
    if (kind == FA_ROPE_SCALE_INDEX && sc->low <= 0.0) return false;
  }
  // from one pair to the next: theta^(-1/half), and where the base is scaled, by
  // factor^(half/(half - 1)), that of it
  Two step = root(theta, half);
  if (kind == FA_ROPE_SCALE_BASE) {
    if (!std::isfinite(theta * std::pow(s, (double)r / (double)(r - 2)))) return false;
    step = step * root(s, half - 1);
  }
  // keep = start + (a pair's frequency, or its number) * rise, clamped
  Two start = one(1.0), rise = one(0.0);
  if (kind == FA_ROPE_SCALE_LINEAR) start = one(0.0);
  if (kind == FA_ROPE_SCALE_TURNS) {
    const Two width = sum(sc->high, -sc->low);
    start = one(0.0) - one(sc->low) / width;
    rise = one(sc->original) * kTurns / width;
  }
  if (kind == FA_ROPE_SCALE_INDEX) {
    auto at = [&](double turns) { return (double)r * std::log(sc->original / (turns * kTurn)) / (2.0 * std::log(theta)); };
    const double lo = std::fmax(0.0, std::floor(at(sc->high)));
    const double hi = std::fmin((double)(r - 1), std::ceil(at(sc->low)));
    rise = one(-1.0) / one(std::fmax(hi - lo, 0.001));
    start = one(1.0) - one(lo) * rise;
  }
  const bool scaled = parts || kind == FA_ROPE_SCALE_LINEAR;
  const Two inverse = one(1.0) / one(scaled ? s : 1.0), rest = one(1.0) - inverse;
  Two base = one(1.0);
  for (int i = 0; i < half; ++i, base = base * step) {
    f[i] = base;
    if (!scaled) continue;
    Two keep = parts ? start + (kind == FA_ROPE_SCALE_TURNS ? base : one(i)) * rise : start;
    if (!std::isfinite(keep.hi)) keep = one((sc->original * base.hi / kTurn - sc->low) / (sc->high - sc->low));  // (past 1e308)
    if (!(keep.hi > 0.0)) f[i] = base * inverse;
    else if ((keep - one(1.0)).hi < 0.0) f[i] = base * (inverse + keep * rest);
  }
  return true;
}

// 2^64 times the turns that f radians are, to the nearest.  (f is at most one
// radian, so this stays below 2^62, and what a double's 53 bits leave is an integer.)
uint64_t turns_of(Two f) {
  const Two t = f * kTurns;
  const double hi = std::ldexp(t.hi, 64), whole = std::floor(hi);
  return (uint64_t)whole + (uint64_t)(int64_t)std::floor((hi - whole) + std::ldexp(t.lo, 64) + 0.5);
}

}  // namespace

extern "C" {

fa_status fa_rope_table(float* rope_cos, float* rope_sin, int64_t n, int64_t rope_dim, double theta, int64_t start,
                        const fa_rope_scaling* scaling, cudaStream_t stream) {
  if (n < 0 || start < 0) return FA_ERR_INVALID_ARG;
  if (!rope_dim_ok(rope_dim, 256)) return FA_ERR_UNSUPPORTED;
  Two f[128];
  if (!scaled_frequencies(rope_dim, theta, scaling, f)) return FA_ERR_INVALID_ARG;
  if (n > kMaxLen || start > kMaxLen) return FA_ERR_UNSUPPORTED;
  if (n == 0) return FA_OK;
  if (!rope_cos || !rope_sin || !aligned16(rope_cos) || !aligned16(rope_sin)) return FA_ERR_INVALID_ARG;
  int dev = 0;
  int* err = nullptr;
  fa_status st = fa::internal_device_setup(&dev, &err);
  if (st != FA_OK) return st;
  fa::RopeTableParams p;
  std::memset(&p, 0, sizeof(p));
  p.cos = rope_cos;
  p.sin = rope_sin;
  p.n = (int)n;
  p.half = (int)(rope_dim / 2);
  p.start = (uint32_t)start;
  const double amp = scaling ? scaling->amplitude : 1.0;
  p.amp_hi = (float)amp;
  p.amp_lo = (float)(amp - (double)p.amp_hi);
  for (int i = 0; i < p.half; ++i) p.turns[i] = turns_of(f[i]);
  return fa::launch_rope_table(p, fa::internal_sm_count(dev), stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_rope(const fa_rope_array* arrays, int64_t count, int64_t B, int64_t N, int64_t d, const int32_t* positions,
                  int64_t pos_stride, int64_t offset, const float* rope_cos, const float* rope_sin, int64_t rope_len,
                  int64_t rope_dim, int rope_layout, int inverse, int dtype, cudaStream_t stream) {
  if (B < 0 || N < 0 || offset < 0 || pos_stride < 0 || rope_len < 0) return FA_ERR_INVALID_ARG;
  if (!arrays || count < 1 || count > 2) return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP16) return FA_ERR_INVALID_ARG;
  if (rope_layout != FA_ROPE_INTERLEAVED && rope_layout != FA_ROPE_HALF) return FA_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (!rope_dim_ok(rope_dim, d)) return FA_ERR_UNSUPPORTED;
  int64_t heads = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (arrays[i].heads < 0) return FA_ERR_INVALID_ARG;
    if (arrays[i].heads > (1 << 20)) return FA_ERR_UNSUPPORTED;
    heads += arrays[i].heads;
  }
  if (N > kMaxLen || B > kMaxLen || rope_len > kMaxLen || offset > kMaxLen || B * ((N * (d / 16) + 255) / 256) > 0x7fffffffLL)
    return FA_ERR_UNSUPPORTED;
  if (B == 0 || N == 0 || heads == 0) return FA_OK;
  if (!rope_cos || !rope_sin || !aligned16(rope_cos) || !aligned16(rope_sin)) return FA_ERR_INVALID_ARG;
  if (positions ? !aligned4(positions) : offset + N > rope_len) return FA_ERR_INVALID_ARG;
  fa::RopeParams p;
  std::memset(&p, 0, sizeof(p));
  for (int64_t i = 0; i < count; ++i) {
    const fa_rope_array& a = arrays[i];
    if (a.heads == 0) continue;
    if (!a.x || !a.y || !aligned16(a.x) || !aligned16(a.y)) return FA_ERR_INVALID_ARG;
    const int64_t sizes[3] = {B, a.heads, N};
    const int64_t xs[3] = {a.x_batch, a.x_head, a.x_token}, ys[3] = {a.y_batch, a.y_head, a.y_token};
    for (int j = 0; j < 3; ++j) {
      if (sizes[j] == 1) continue;  // never stepped over
      if (xs[j] < 0 || xs[j] % 8 != 0 || ys[j] < d || ys[j] % 8 != 0) return FA_ERR_INVALID_ARG;
      if (xs[j] >= (int64_t)1 << 38 || ys[j] >= (int64_t)1 << 38) return FA_ERR_UNSUPPORTED;
    }
    fa::RopeArray& o = p.a[i];
    o.x = static_cast<const uint16_t*>(a.x);
    o.y = static_cast<uint16_t*>(a.y);
    o.heads = (int)a.heads;
    o.x_batch = B > 1 ? a.x_batch : 0;
    o.x_head = a.heads > 1 ? a.x_head : 0;
    o.x_token = N > 1 ? a.x_token : 0;
    o.y_batch = B > 1 ? a.y_batch : 0;
    o.y_head = a.heads > 1 ? a.y_head : 0;
    o.y_token = N > 1 ? a.y_token : 0;
    o.same = o.x == o.y;
    if (o.same && (o.x_batch != o.y_batch || o.x_head != o.y_head || o.x_token != o.y_token)) return FA_ERR_INVALID_ARG;
  }
  int dev = 0;
  int* err = nullptr;
  fa_status st = fa::internal_device_setup(&dev, &err);
  if (st != FA_OK) return st;
  p.heads = (int)heads;
  p.N = (int)N;
  p.r = (int)rope_dim;
  p.positions = positions;
  p.pos_stride = pos_stride;
  p.offset = (int)offset;
  p.cos = rope_cos;
  p.sin = rope_sin;
  p.rope_len = (int)rope_len;
  p.err = err;
  return fa::launch_rope(p, B, (int)d, dtype == FA_DTYPE_FP16, rope_layout, inverse != 0, fa::internal_sm_count(dev), stream) ==
                 cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // extern "C"
