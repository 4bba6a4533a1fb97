// pages_api.cu -- the C ABI of the operators on a cache's pages (declared in
// include/fa.h): argument checks and launch on the caller's stream.
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "fa.h"
#include "api_internal.h"
#include "pages.h"

namespace {

constexpr int64_t kMaxLen = (int64_t)1 << 30;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A cache of `layers` layers, layer_stride elements apart.
fa_status check_layers(const fa_kv_cache* c, int64_t layers, int64_t layer_stride, fa::PageRows* r) {
  if (layers < 0) return FA_ERR_INVALID_ARG;
  const fa_status st = fa::internal_check_cache(c);
  if (st != FA_OK) return st;
  if (layers > 1 && (layer_stride < c->d || layer_stride % 8 != 0)) return FA_ERR_INVALID_ARG;
  if (layers > 32767 || (layers > 1 && layer_stride >= (int64_t)1 << 44)) return FA_ERR_UNSUPPORTED;
  if (c->heads * c->page_size * (c->d / 8) > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;  // (pieces of a page's plane)
  std::memset(r, 0, sizeof(*r));
  r->k = static_cast<uint16_t*>(c->k);
  r->v = static_cast<uint16_t*>(c->v);
  // a stride that is never stepped over counts for nothing
  r->layer_stride = layers > 1 ? layer_stride : 0;
  r->page_stride = c->num_pages > 1 ? c->page_stride : 0;
  r->head_stride = c->heads > 1 ? c->head_stride : 0;
  r->token_stride = c->token_stride;
  r->layers = (int)layers;
  r->heads = (int)c->heads;
  r->num_pages = (int)c->num_pages;
  r->page_shift = fa::internal_shift_of(c->page_size);
  return FA_OK;
}

fa_status check_table(const int32_t* block_table, int64_t table_stride, int64_t max_pages, int64_t rows) {
  if (max_pages < 1 || (rows > 1 && table_stride < max_pages)) return FA_ERR_INVALID_ARG;
  if (!aligned4(block_table)) return FA_ERR_INVALID_ARG;
  return max_pages > kMaxLen ? FA_ERR_UNSUPPORTED : FA_OK;
}

fa::PoolParams pool_of(int32_t* refs, int64_t num_pages, int shift, int32_t* block_table, int64_t table_stride, int64_t max_pages,
                       int32_t* seq_k, int64_t rows) {
  fa::PoolParams p;
  std::memset(&p, 0, sizeof(p));
  p.refs = refs;
  p.table = block_table;
  p.table_stride = rows > 1 ? table_stride : max_pages;
  p.max_pages = (int)max_pages;
  p.num_pages = (int)num_pages;
  p.page_shift = shift;
  p.rows = (int)rows;
  p.seq_k = seq_k;
  return p;
}

}  // namespace

extern "C" {

fa_status fa_pages_resize(int32_t* refs, int64_t num_pages, int64_t page_size, int32_t* block_table, int64_t table_stride,
                          int64_t max_pages, int32_t* seq_k, const int32_t* want, int64_t B, cudaStream_t stream) {
  if (B < 0 || num_pages < 1) return FA_ERR_INVALID_ARG;
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0 || num_pages > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (B > fa::kMaxResizeRows) return FA_ERR_UNSUPPORTED;
  if (B == 0) return FA_OK;
  fa_status st = check_table(block_table, table_stride, max_pages, B);
  if (st != FA_OK) return st;
  if (!refs || !aligned16(refs) || !aligned4(seq_k) || !aligned4(want)) return FA_ERR_INVALID_ARG;
  int dev = 0;
  int* err = nullptr;
  if ((st = fa::internal_device_setup(&dev, &err)) != FA_OK) return st;
  fa::PoolParams p = pool_of(refs, num_pages, fa::internal_shift_of(page_size), block_table, table_stride, max_pages, seq_k, B);
  p.err = err;
  return fa::launch_pages_resize(p, want, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_pages_fork(const fa_kv_cache* cache, int64_t layers, int64_t layer_stride, int32_t* refs, int32_t* block_table,
                        int64_t table_stride, int64_t max_pages, int32_t* seq_k, int64_t rows, const int32_t* src,
                        const int32_t* dst, int32_t* fresh, int64_t n, cudaStream_t stream) {
  if (n < 0 || rows < 0) return FA_ERR_INVALID_ARG;
  fa::PageRows r;
  fa_status st = check_layers(cache, layers, layer_stride, &r);
  if (st != FA_OK) return st;
  if (rows > fa::kMaxForkRows || n > fa::kMaxForks) return FA_ERR_UNSUPPORTED;
  if (n == 0) return FA_OK;
  if (layers == 0 || rows == 0) return FA_ERR_INVALID_ARG;
  if ((st = check_table(block_table, table_stride, max_pages, rows)) != FA_OK) return st;
  if (!refs || !aligned16(refs) || !aligned4(seq_k) || !aligned4(src) || !aligned4(dst) || !aligned4(fresh)) return FA_ERR_INVALID_ARG;
  int dev = 0;
  int* err = nullptr;
  if ((st = fa::internal_device_setup(&dev, &err)) != FA_OK) return st;
  fa::PoolParams p = pool_of(refs, cache->num_pages, r.page_shift, block_table, table_stride, max_pages, seq_k, rows);
  p.err = err;
  return fa::launch_pages_fork(p, r, (int)cache->d, src, dst, fresh, (int)n, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_copy(const fa_kv_cache* cache, int64_t layers, int64_t layer_stride, const int32_t* src, const int32_t* dst,
                        int64_t n, cudaStream_t stream) {
  if (n < 0) return FA_ERR_INVALID_ARG;
  fa::PageRows r;
  fa_status st = check_layers(cache, layers, layer_stride, &r);
  if (st != FA_OK) return st;
  // (a page's blocks times the pairs make a grid)
  if (n > kMaxLen || n * ((cache->heads * cache->page_size * (cache->d / 8) + 2047) / 2048) > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (n == 0 || layers == 0) return FA_OK;
  if (!aligned4(src) || !aligned4(dst)) return FA_ERR_INVALID_ARG;
  int dev = 0;
  int* err = nullptr;
  if ((st = fa::internal_device_setup(&dev, &err)) != FA_OK) return st;
  return fa::launch_cache_copy(r, (int)cache->d, src, dst, (int)n, err, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_compact(const fa_kv_cache* cache, int64_t layers, int64_t layer_stride, const int32_t* block_table,
                           int64_t table_stride, int64_t max_pages, const int32_t* first, const int32_t* keep,
                           int64_t keep_stride, int64_t max_keep, const int32_t* keep_n, int32_t* seq_k_out, int64_t B,
                           cudaStream_t stream) {
  if (B < 0 || max_keep < 0) return FA_ERR_INVALID_ARG;
  fa::CompactParams p;
  std::memset(&p, 0, sizeof(p));
  fa_status st = check_layers(cache, layers, layer_stride, &p.rows);
  if (st != FA_OK) return st;
  if (B > (1 << 24) || max_keep > kMaxLen || B * cache->heads * 4 > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (B == 0) return FA_OK;
  if (layers == 0) return FA_ERR_INVALID_ARG;
  if ((st = check_table(block_table, table_stride, max_pages, B)) != FA_OK) return st;
  if (B > 1 && keep_stride < max_keep) return FA_ERR_INVALID_ARG;
  if (!aligned4(first) || !aligned4(keep_n) || !aligned4(seq_k_out) || (max_keep > 0 && !aligned4(keep))) return FA_ERR_INVALID_ARG;
  int dev = 0;
  int* err = nullptr;
  if ((st = fa::internal_device_setup(&dev, &err)) != FA_OK) return st;
  p.table = block_table;
  p.table_stride = table_stride;
  p.max_pages = (int)max_pages;
  p.first = first;
  p.keep = keep;
  p.keep_stride = keep_stride;
  p.max_keep = (int)max_keep;
  p.keep_n = keep_n;
  p.seq_k_out = seq_k_out;
  p.B = (int)B;
  p.err = err;
  return fa::launch_cache_compact(p, (int)cache->d, fa::internal_sm_count(dev), stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
