// window_api.cu -- the C ABI of the windowed and paged operators (declared in
// include/fa.h): argument checks, TMA descriptors, kernel selection and
// launch on the caller's stream.  Nothing is allocated here.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "fa.h"
#include "api_internal.h"
#include "attn_window.cuh"
#include "paged.h"
#include "tree.h"

namespace fa {
#define FA_EXTERN_WINDOW(E, D, P, F) extern template cudaError_t launch_attn_window<E, D, P, F>(const WinLaunch&);
#define FA_EXTERN_PAGED(E, D, F)     \
  FA_EXTERN_WINDOW(E, D, true, F)      \
  extern template cudaError_t launch_attn_window<E, D, true, F, true>(const WinLaunch&);
#define FA_EXTERN_ELEM(E)                 \
  FA_EXTERN_WINDOW(E, 64, false, WIN_PAIR)  \
  FA_EXTERN_WINDOW(E, 128, false, WIN_PAIR) \
  FA_EXTERN_WINDOW(E, 256, false, WIN_ONE)  \
  FA_EXTERN_WINDOW(E, 64, false, WIN_TWO)    \
  FA_EXTERN_WINDOW(E, 64, false, WIN_SPLIT)  \
  FA_EXTERN_WINDOW(E, 128, false, WIN_SPLIT) \
  FA_EXTERN_WINDOW(E, 256, false, WIN_SPLIT) \
  FA_EXTERN_PAGED(E, 64, WIN_FEW2)      \
  FA_EXTERN_PAGED(E, 64, WIN_ONE)      \
  FA_EXTERN_PAGED(E, 64, WIN_PAIR)      \
  FA_EXTERN_PAGED(E, 128, WIN_FEW)      \
  FA_EXTERN_PAGED(E, 128, WIN_FEW2)      \
  FA_EXTERN_PAGED(E, 128, WIN_ONE)      \
  FA_EXTERN_PAGED(E, 128, WIN_PAIR)      \
  FA_EXTERN_PAGED(E, 256, WIN_FEW)      \
  FA_EXTERN_PAGED(E, 256, WIN_ONE)
FA_EXTERN_ELEM(kBF16)
FA_EXTERN_ELEM(kFP16)
#undef FA_EXTERN_ELEM
#undef FA_EXTERN_PAGED
#undef FA_EXTERN_WINDOW
}  // namespace fa

namespace {

constexpr int64_t kMaxWords = 32;              // of a mask row: a lane has one
constexpr int64_t kMaxLen = (int64_t)1 << 30;  // positions, windows and token counts fit int arithmetic

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// scale * log2(e); a zero scale becomes one so small that every score's
// product is zero against the row sum's rounding, while a masked score
// (infinite) still gives 2^-inf = 0 rather than 0 * inf
float log2_scale(float scale) {
  const float s = (float)((double)scale * 1.4426950408889634074);
  return s == 0.0f ? 1e-30f : s;
}

template <int ELEM>
fa_status launch_dense(const fa::WinLaunch& L, int64_t d, int form) {
  cudaError_t e = cudaErrorInvalidValue;
  if (d == 64) {
    if (form == fa::WIN_SPLIT) e = fa::launch_attn_window<ELEM, 64, false, fa::WIN_SPLIT>(L);
    if (form == fa::WIN_TWO) e = fa::launch_attn_window<ELEM, 64, false, fa::WIN_TWO>(L);
    if (form == fa::WIN_PAIR) e = fa::launch_attn_window<ELEM, 64, false, fa::WIN_PAIR>(L);
  } else if (d == 128) {
    if (form == fa::WIN_SPLIT) e = fa::launch_attn_window<ELEM, 128, false, fa::WIN_SPLIT>(L);
    if (form == fa::WIN_PAIR) e = fa::launch_attn_window<ELEM, 128, false, fa::WIN_PAIR>(L);
  } else {
    if (form == fa::WIN_SPLIT) e = fa::launch_attn_window<ELEM, 256, false, fa::WIN_SPLIT>(L);
    if (form == fa::WIN_ONE) e = fa::launch_attn_window<ELEM, 256, false, fa::WIN_ONE>(L);
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int ELEM, bool TREE>
fa_status launch_paged(const fa::WinLaunch& L, int64_t d, int form) {
  cudaError_t e = cudaErrorInvalidValue;
  if (d == 64) {
    if (form == fa::WIN_FEW2) e = fa::launch_attn_window<ELEM, 64, true, fa::WIN_FEW2, TREE>(L);
    if (form == fa::WIN_ONE) e = fa::launch_attn_window<ELEM, 64, true, fa::WIN_ONE, TREE>(L);
    if (form == fa::WIN_PAIR) e = fa::launch_attn_window<ELEM, 64, true, fa::WIN_PAIR, TREE>(L);
  } else if (d == 128) {
    if (form == fa::WIN_FEW) e = fa::launch_attn_window<ELEM, 128, true, fa::WIN_FEW, TREE>(L);
    if (form == fa::WIN_FEW2) e = fa::launch_attn_window<ELEM, 128, true, fa::WIN_FEW2, TREE>(L);
    if (form == fa::WIN_ONE) e = fa::launch_attn_window<ELEM, 128, true, fa::WIN_ONE, TREE>(L);
    if (form == fa::WIN_PAIR) e = fa::launch_attn_window<ELEM, 128, true, fa::WIN_PAIR, TREE>(L);
  } else {
    if (form == fa::WIN_FEW) e = fa::launch_attn_window<ELEM, 256, true, fa::WIN_FEW, TREE>(L);
    if (form == fa::WIN_ONE) e = fa::launch_attn_window<ELEM, 256, true, fa::WIN_ONE, TREE>(L);
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

CUtensorMapDataType map_type(int dtype) {
  return dtype == FA_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// Two partial results of all query rows that an SM works on (a pair of query
// tiles, or two CTAs of one), their LSE, and a descriptor per CTA.
struct PagedWorkspace {
  size_t lse_at, desc_at, bytes;
};
PagedWorkspace paged_workspace(int sms, int64_t d) {
  const size_t rows = (size_t)2 * sms * (d <= 128 ? 2 : 1) * fa::kBM;
  PagedWorkspace w;
  w.lse_at = rows * d * 4;
  w.desc_at = w.lse_at + rows * 4;
  w.bytes = w.desc_at + (size_t)2 * sms * sizeof(int4);
  return w;
}

// The layout of a cache: sizes, strides that a TMA map can describe, a page
// size that boxes of whole 8-row swizzle groups cover.
fa_status check_cache(const fa_kv_cache* c) {
  if (!c || !c->k || !c->v) return FA_ERR_INVALID_ARG;
  if (c->dtype != FA_DTYPE_BF16 && c->dtype != FA_DTYPE_FP16) return FA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->heads < 1 || c->page_size < 1) return FA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128 && c->d != 256) return FA_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0) return FA_ERR_UNSUPPORTED;
  if (c->num_pages > 0x7fffffffLL || c->heads > (1 << 20)) return FA_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v)) return FA_ERR_INVALID_ARG;
  const int64_t strides[3] = {c->token_stride, c->head_stride, c->page_stride};
  const int64_t sizes[3] = {c->page_size, c->heads, c->num_pages};
  for (int i = 0; i < 3; ++i) {
    if (sizes[i] == 1) continue;  // never stepped over
    if (strides[i] < c->d || strides[i] % 8 != 0) return FA_ERR_INVALID_ARG;
    if (strides[i] >= (int64_t)1 << 38) return FA_ERR_UNSUPPORTED;
  }
  return FA_OK;
}

// What a ragged batch over a cache needs of its index arrays.
fa_status check_batch(const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                      const int32_t* cu_q, const int32_t* seq_k, int64_t B, int64_t T) {
  if (max_pages < 1 || (B > 1 && table_stride < max_pages)) return FA_ERR_INVALID_ARG;
  if (!block_table || !cu_q || !seq_k) return FA_ERR_INVALID_ARG;
  if (!aligned4(block_table) || !aligned4(cu_q) || !aligned4(seq_k)) return FA_ERR_INVALID_ARG;
  if (B > (1 << 24) || T > kMaxLen || max_pages > kMaxLen) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int shift_of(int64_t page_size) {
  int s = 0;
  while (((int64_t)1 << s) < page_size) ++s;
  return s;
}

// fa_fwd_paged, and with a mask fa_fwd_tree.
fa_status fwd_paged(const void* q, const fa_kv_cache* cache, void* o, float* lse, const int32_t* block_table,
                    int64_t table_stride, int64_t max_pages, const int32_t* cu_q, const int32_t* seq_k, const uint32_t* mask,
                    int64_t words, const int32_t* positions, int64_t B, int64_t T, int64_t Hq, int64_t q_stride, int64_t max_q,
                    int64_t window, int64_t sinks, float scale, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (B < 0 || T < 0 || Hq < 0 || max_q < 0) return FA_ERR_INVALID_ARG;
  if (window < 1 || sinks < 0 || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  fa_status st = check_cache(cache);
  if (st != FA_OK) return st;
  const int64_t Hkv = cache->heads, d = cache->d;
  if (Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (Hq / Hkv > fa::kBM) return FA_ERR_UNSUPPORTED;  // a token's heads share one query tile
  if (B == 0 || T == 0 || Hq == 0) return FA_OK;
  if ((st = check_batch(block_table, table_stride, max_pages, cu_q, seq_k, B, T)) != FA_OK) return st;
  if (!q || !o || !lse || !aligned16(q) || !aligned16(o) || !aligned4(lse)) return FA_ERR_INVALID_ARG;
  if (T > 1 && (q_stride < Hq * d || q_stride % 8 != 0)) return FA_ERR_INVALID_ARG;
  if (q_stride >= (int64_t)1 << 38 || Hq > (1 << 20)) return FA_ERR_UNSUPPORTED;
  int dev = 0;
  int* err = nullptr;
  if ((st = fa::internal_device_setup(&dev, &err)) != FA_OK) return st;
  const int sms = fa::internal_sm_count(dev);
  const PagedWorkspace ws = paged_workspace(sms, d);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < ws.bytes)
    return FA_ERR_INVALID_ARG;

  fa::WinLaunch L;
  std::memset(&L, 0, sizeof(L));
  const int64_t g = Hq / Hkv;
  if (max_q < T && max_q * B < T) max_q = 0;  // too low for so many tokens: not a hint to size units by
  int64_t tpt = fa::kBM / g;  // tokens whose g heads fit a query tile
  if (max_q > 0 && max_q < tpt) tpt = max_q;
  // The form (see WinForm).  Few rows: no sequence brings more than their
  // tokens, or each brings one on average.  Two CTAs per SM with units for all.
  auto few_of = [&](int form) {
    const int64_t tokens = fa::few_rows((int)d, form) / g;
    return tokens > 0 && (max_q > 0 ? max_q <= tokens : T <= B) ? tokens : 0;
  };
  int64_t few = d == 64 || (d == 128 && B * Hkv >= sms) ? few_of(fa::WIN_FEW2) : 0;
  const bool few2 = few > 0;
  if (!few2) few = d == 64 ? 0 : few_of(fa::WIN_FEW);
  if (few > 0 && few < tpt) tpt = few;
  // Else query tiles per CTA: one where sequences bring few rows on average; or
  // up to a tile's, if there are enough of them that few are cut or if the
  // longest is far above the average, so that most are short.
  // (One tile against a pair at d = 64, 16/4 heads: 32 x 1 token over 3000 keys
  // 32 and 37 us; 33 sequences, 30 of them one token, 31 and 36; but 32 x 24
  // tokens over 1100 keys, cut into twice as many parts, 24 and 19.)  Trees, whose
  // line counts a step of one query tile as one of a pair: one where they bring up
  // to a tile's rows on average (one against a pair, 32/8 heads: 32 x 16 nodes over
  // 1000 to 8000 keys 72.6 and 87.4 us at d = 64, 110.4 and 110.9 at d = 128, under a
  // window of 1000 34.5 and 42.0, 43.5 and 49.3; 32 nodes 84.5 and 90.6, 117.3 and 117.6;
  // above, 33 to 40 nodes 137 and 109, 200 and 131).
  const bool pair = few == 0 && d <= 128 && (T * g > fa::kBM * B || (!mask && T * g > 32 * B && B * Hkv < 2 * sms &&
                                                                    (max_q < T ? max_q : T) * B <= 4 * T));
  const int form = few2 ? fa::WIN_FEW2 : few > 0 ? fa::WIN_FEW : pair ? fa::WIN_PAIR : fa::WIN_ONE;
  const int ctas = few2 || (form == fa::WIN_ONE && d == 64) ? 2 * sms : sms;
  const int slot_rows = (pair ? 2 : 1) * fa::kBM;
  const CUtensorMapDataType dt = map_type(cache->dtype);
  {
    const uint64_t dims[3] = {(uint64_t)d, (uint64_t)Hq, (uint64_t)T};
    const uint64_t strides[2] = {(uint64_t)d * 2, (uint64_t)(T > 1 ? q_stride : Hq * d) * 2};
    const uint32_t box[3] = {64, (uint32_t)g, (uint32_t)tpt};
    if ((st = fa::internal_encode_map_nd(&L.q, q, dt, 3, dims, strides, box)) != FA_OK) return st;
  }
  for (int i = 0; i < 2; ++i) {
    const uint64_t dims[4] = {(uint64_t)d, (uint64_t)cache->page_size, (uint64_t)Hkv, (uint64_t)cache->num_pages};
    // a stride that is never stepped over only has to be one that a map takes
    const uint64_t strides[3] = {(uint64_t)cache->token_stride * 2,
                                 (uint64_t)(Hkv > 1 ? cache->head_stride : cache->token_stride) * 2,
                                 (uint64_t)(cache->num_pages > 1 ? cache->page_stride : cache->token_stride) * 2};
    const uint32_t box[4] = {64, (uint32_t)(cache->page_size < 128 ? cache->page_size : 128), 1, 1};
    if ((st = fa::internal_encode_map_nd(i == 0 ? &L.k : &L.v, i == 0 ? cache->k : cache->v, dt, 4, dims, strides,
                                         box)) != FA_OK)
      return st;
  }
  L.o = L.q;  // (not used: a paged tile's rows are stored by their threads)
  fa::WinParams& p = L.prm;
  p.o = o;
  p.lse = lse;
  p.err = err;
  p.window = (int)(window < kMaxLen ? window : kMaxLen);
  p.sinks = (int)(sinks < kMaxLen ? sinks : kMaxLen);
  p.scale_log2 = log2_scale(scale);
  p.Hq = (int)Hq;
  p.Hkv = (int)Hkv;
  p.o_vec32 = (reinterpret_cast<uintptr_t>(o) & 31u) == 0;
  p.drop_pos = fa::internal_take_inject() ? 1 : -1;
  p.cu_q = cu_q;
  p.seq_k = seq_k;
  p.table = block_table;
  p.B = (int)B;
  p.T = (int)T;
  p.max_pages = (int)max_pages;
  p.table_stride = table_stride;
  p.num_pages = (int)cache->num_pages;
  p.page_shift = shift_of(cache->page_size);
  p.mask = mask;
  p.words = (int)words;
  p.positions = positions;
  p.g = (int)g;
  p.tpt = (int)tpt;
  // the line of work: at most this many units, each of at most this many
  // key tiles, two places to a tile
  const int64_t unit_tok = (pair ? 2 : 1) * tpt;
  const int64_t keys = max_pages * cache->page_size < kMaxLen ? max_pages * cache->page_size : kMaxLen;
  int64_t tiles = keys / fa::kBN + 1;
  const int64_t reach = p.window + (int64_t)p.sinks + unit_tok + 32 * words;  // (a tree's units start their windows at its root's)
  if (reach < keys) tiles = reach / fa::kBN + 4;
  const int64_t units = (T / unit_tok + B) * Hkv;
  if (mask) tiles += 2;  // (the places behind a tree unit's: end_places)
  if (units >= (int64_t)0x7fffffff / (2 * (tiles + 1))) return FA_ERR_UNSUPPORTED;
  p.max_places = (uint32_t)(units * 2 * (tiles + 1));
  uint8_t* w = static_cast<uint8_t*>(workspace);
  p.o_part = reinterpret_cast<float*>(w);
  p.lse_part = reinterpret_cast<float*>(w + ws.lse_at);
  p.desc = reinterpret_cast<int4*>(w + ws.desc_at);
  L.grid = ctas;
  L.stream = stream;
  if (mask)
    st = cache->dtype == FA_DTYPE_BF16 ? launch_paged<fa::kBF16, true>(L, d, form) : launch_paged<fa::kFP16, true>(L, d, form);
  else
    st = cache->dtype == FA_DTYPE_BF16 ? launch_paged<fa::kBF16, false>(L, d, form) : launch_paged<fa::kFP16, false>(L, d, form);
  if (st != FA_OK) return st;
  const int64_t most = (max_q > 0 && max_q < unit_tok ? max_q : unit_tok) * g;
  return fa::launch_paged_combine(p.o_part, p.lse_part, p.desc, o, lse, sms, ctas, (int)units, slot_rows, (int)most,
                                  (int)g, (int)Hq, (int)d, cache->dtype == FA_DTYPE_FP16, stream) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // namespace

namespace fa {
fa_status internal_check_cache(const fa_kv_cache* cache) { return check_cache(cache); }
int internal_shift_of(int64_t page_size) { return shift_of(page_size); }
}  // namespace fa

extern "C" {

fa_status fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t Hq,
                        int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d, int64_t window, int64_t sinks, float scale,
                        int dtype, cudaStream_t stream) {
  if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP16) return FA_ERR_INVALID_ARG;
  if (window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
  bool empty = false;
  fa_status st = fa::internal_check_common(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, &empty);
  if (st != FA_OK || empty) return st;
  if (Nq > kMaxLen || Nk > kMaxLen) return FA_ERR_UNSUPPORTED;
  int dev = 0;
  int* err = nullptr;
  if ((st = fa::internal_device_setup(&dev, &err)) != FA_OK) return st;
  fa::WinLaunch L;
  std::memset(&L, 0, sizeof(L));
  const CUtensorMapDataType dt = map_type(dtype);
  if ((st = fa::internal_encode_map(&L.q, q, dt, 2, B * Hq, Nq, d, 128)) != FA_OK) return st;
  if ((st = fa::internal_encode_map(&L.k, k, dt, 2, B * Hkv, Nk, d, 128)) != FA_OK) return st;
  if ((st = fa::internal_encode_map(&L.v, v, dt, 2, B * Hkv, Nk, d, 128)) != FA_OK) return st;
  if ((st = fa::internal_encode_map(&L.o, o, dt, 2, B * Hq, Nq, d, 32)) != FA_OK) return st;
  L.prm.o = o;
  L.prm.lse = lse;
  L.prm.err = err;
  L.prm.window = (int)(window < kMaxLen ? window : kMaxLen);
  L.prm.sinks = (int)(sinks < kMaxLen ? sinks : kMaxLen);
  L.prm.scale_log2 = log2_scale(scale);
  L.prm.Hq = (int)Hq;
  L.prm.Hkv = (int)Hkv;
  L.prm.o_vec32 = (reinterpret_cast<uintptr_t>(o) & 31u) == 0;
  L.prm.drop_pos = fa::internal_take_inject() ? 1 : -1;  // (a slot that any unit with a key uses)
  L.prm.N = (int)Nq;
  L.prm.Nk = (int)Nk;
  L.prm.BH = (int)(B * Hq);
  L.stream = stream;
  // few query tiles over some key tiles: a cluster for each, as large as all run
  // at once, a key tile and more per CTA (see WinForm; below 512 keys the join
  // takes what the split gives)
  const int64_t tiles = B * Hq * ((Nq + fa::kBM - 1) / fa::kBM);
  int64_t reach = L.prm.window + (int64_t)L.prm.sinks + fa::kBM;  // keys a query tile sees, and what its edges add
  if (reach > Nk) reach = Nk;
  for (int c = 8; c > 1 && L.cluster == 0; c /= 2)
    if (reach >= 512 && reach >= c * fa::kBN && tiles <= fa::window_clusters(dev, c)) L.cluster = c;
  int form = d == 256 ? fa::WIN_ONE : fa::WIN_PAIR;
  if (d == 64 && reach <= 6 * fa::kBN && tiles > fa::internal_sm_count(dev)) form = fa::WIN_TWO;
  if (L.cluster > 0) form = fa::WIN_SPLIT;
  return dtype == FA_DTYPE_BF16 ? launch_dense<fa::kBF16>(L, d, form) : launch_dense<fa::kFP16>(L, d, form);
}

fa_status fa_paged_workspace_bytes(int64_t d, size_t* bytes) {
  if (!bytes) return FA_ERR_INVALID_ARG;
  *bytes = 0;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  *bytes = paged_workspace(fa::internal_sm_count(dev), d).bytes;
  return FA_OK;
}

fa_status fa_fwd_paged(const void* q, const fa_kv_cache* cache, void* o, float* lse, const int32_t* block_table,
                       int64_t table_stride, int64_t max_pages, const int32_t* cu_q, const int32_t* seq_k, int64_t B,
                       int64_t T, int64_t Hq, int64_t q_stride, int64_t max_q, int64_t window, int64_t sinks,
                       float scale, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return fwd_paged(q, cache, o, lse, block_table, table_stride, max_pages, cu_q, seq_k, nullptr, 0, nullptr, B, T, Hq, q_stride,
                   max_q, window, sinks, scale, workspace, workspace_bytes, stream);
}

fa_status fa_fwd_tree(const void* q, const fa_kv_cache* cache, void* o, float* lse, const int32_t* block_table,
                      int64_t table_stride, int64_t max_pages, const int32_t* cu_q, const int32_t* seq_k,
                      const uint32_t* mask, int64_t words, const int32_t* positions, int64_t B, int64_t T, int64_t Hq,
                      int64_t q_stride, int64_t max_q, int64_t window, int64_t sinks, float scale, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
  if (words < 1) return FA_ERR_INVALID_ARG;
  if (words > kMaxWords) return FA_ERR_UNSUPPORTED;
  if (B > 0 && T > 0 && Hq > 0 && (!mask || !aligned4(mask) || (positions && !aligned4(positions)))) return FA_ERR_INVALID_ARG;
  return fwd_paged(q, cache, o, lse, block_table, table_stride, max_pages, cu_q, seq_k, mask, words, positions, B, T, Hq, q_stride,
                   max_q, window, sinks, scale, workspace, workspace_bytes, stream);
}

fa_status fa_tree_plan(const int32_t* parents, const int32_t* cu_q, const int32_t* seq_k, int64_t B, int64_t T,
                       uint32_t* mask, int64_t words, int32_t* positions, cudaStream_t stream) {
  return fa_tree_plan_window(parents, cu_q, seq_k, B, T, mask, words, positions, kMaxLen, 0, stream);
}

fa_status fa_tree_plan_window(const int32_t* parents, const int32_t* cu_q, const int32_t* seq_k, int64_t B, int64_t T,
                              uint32_t* mask, int64_t words, int32_t* positions, int64_t window, int64_t sinks,
                              cudaStream_t stream) {
  if (B < 0 || T < 0 || words < 1 || window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (words > kMaxWords || B > (1 << 24) || T > kMaxLen) return FA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return FA_OK;
  if (!parents || !cu_q || !seq_k || !mask || !positions) return FA_ERR_INVALID_ARG;
  if (!aligned4(parents) || !aligned4(cu_q) || !aligned4(seq_k) || !aligned4(mask) || !aligned4(positions)) return FA_ERR_INVALID_ARG;
  int dev = 0;
  int* err = nullptr;
  const fa_status st = fa::internal_device_setup(&dev, &err);
  if (st != FA_OK) return st;
  return fa::launch_tree_plan(parents, cu_q, seq_k, (int)B, (int)T, mask, (int)words, positions,
                              (int)(window < kMaxLen ? window : kMaxLen), (int)(sinks < kMaxLen ? sinks : kMaxLen), err,
                              stream) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status fa_cache_append(const fa_kv_cache* cache, const void* q, const void* k, const void* v, void* q_out,
                          int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t* block_table,
                          int64_t table_stride, int64_t max_pages, const int32_t* cu_q, const int32_t* seq_k,
                          int64_t B, int64_t T, int64_t Hq, const float* rope_cos, const float* rope_sin,
                          int64_t rope_len, int rope_layout, cudaStream_t stream) {
  return fa_cache_append_at(cache, q, k, v, q_out, q_stride, k_stride, v_stride, block_table, table_stride, max_pages, cu_q,
                            seq_k, B, T, Hq, rope_cos, rope_sin, rope_len, cache ? cache->d : 0, rope_layout, nullptr, stream);
}

fa_status fa_cache_append_at(const fa_kv_cache* cache, const void* q, const void* k, const void* v, void* q_out,
                             int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t* block_table,
                             int64_t table_stride, int64_t max_pages, const int32_t* cu_q, const int32_t* seq_k,
                             int64_t B, int64_t T, int64_t Hq, const float* rope_cos, const float* rope_sin,
                             int64_t rope_len, int64_t rope_dim, int rope_layout, const int32_t* positions,
                             cudaStream_t stream) {
  if (B < 0 || T < 0 || Hq < 0 || rope_len < 0) return FA_ERR_INVALID_ARG;
  if (rope_layout != 0 && rope_layout != FA_ROPE_INTERLEAVED && rope_layout != FA_ROPE_HALF) return FA_ERR_INVALID_ARG;
  fa_status st = check_cache(cache);
  if (st != FA_OK) return st;
  if (rope_layout != 0 && (rope_dim < 16 || rope_dim > cache->d || rope_dim % 16 != 0)) return FA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return FA_OK;
  if ((st = check_batch(block_table, table_stride, max_pages, cu_q, seq_k, B, T)) != FA_OK) return st;
  if (rope_layout != 0 && positions && !aligned4(positions)) return FA_ERR_INVALID_ARG;
  const int64_t d = cache->d, Hkv = cache->heads;
  if (rope_layout != 0 && (!rope_cos || !rope_sin || !aligned16(rope_cos) || !aligned16(rope_sin)))
    return FA_ERR_INVALID_ARG;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return FA_ERR_INVALID_ARG;
  if (Hq > 0 && (!q || !q_out || !aligned16(q) || !aligned16(q_out))) return FA_ERR_INVALID_ARG;
  if (T > 1) {
    if (k_stride < Hkv * d || k_stride % 8 != 0 || v_stride < Hkv * d || v_stride % 8 != 0) return FA_ERR_INVALID_ARG;
    if (Hq > 0 && (q_stride < Hq * d || q_stride % 8 != 0)) return FA_ERR_INVALID_ARG;
  }
  if (Hq > (1 << 20)) return FA_ERR_UNSUPPORTED;
  int dev = 0;
  int* err = nullptr;
  if ((st = fa::internal_device_setup(&dev, &err)) != FA_OK) return st;
  fa::AppendParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_pages = static_cast<uint16_t*>(cache->k);
  p.v_pages = static_cast<uint16_t*>(cache->v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.page_stride = cache->page_stride;
  p.head_stride = cache->head_stride;
  p.token_stride = cache->token_stride;
  p.table = block_table;
  p.cu_q = cu_q;
  p.seq_k = seq_k;
  p.table_stride = table_stride;
  p.max_pages = (int)max_pages;
  p.num_pages = (int)cache->num_pages;
  p.page_shift = shift_of(cache->page_size);
  p.B = (int)B;
  p.T = (int)T;
  p.Hq = (int)Hq;
  p.Hkv = (int)Hkv;
  p.cos = rope_cos;
  p.sin = rope_sin;
  p.rope_len = (int)(rope_len < kMaxLen ? rope_len : kMaxLen);
  p.rope_dim = (int)(rope_layout != 0 ? rope_dim : 0);
  p.positions = positions;
  p.err = err;
  return fa::launch_cache_append(p, (int)d, cache->dtype == FA_DTYPE_FP16, rope_layout, stream) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // extern "C"
