// pages.cu -- a paged cache's pages: handed out and taken back, shared by
// sequences that go on from the same tokens, copied, and compacted.
#include <climits>
#include <cstdint>

#include "fa.h"
#include "pages.h"
#include "ptx_window.cuh"

namespace fa {
namespace {

// Tokens as a row of the table can hold them; *bad where they had to be cut.
__device__ __forceinline__ int cut_tokens(int n, const PoolParams& prm, bool& bad) {
  const long long cap = (long long)prm.max_pages << prm.page_shift;
  const int cut = n < 0 ? 0 : n > cap ? (int)cap : n;
  bad |= cut != n;
  return cut;
}
__device__ __forceinline__ int pages_of(int tokens, int shift) {
  return (int)(((long long)tokens + (1 << shift) - 1) >> shift);
}

// Exclusive sum over the block's THREADS threads, and the total.
template <int THREADS>
__device__ __forceinline__ long long block_scan(long long x, long long& total, long long* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  __syncthreads();  // (the sums of the call before have been read)
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  long long w = lane < THREADS / 32 ? sums[lane] : 0;
#pragma unroll
  for (int d = 1; d < THREADS / 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, THREADS / 32 - 1);
  const long long before = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
  return incl - x + (warp == 0 ? 0 : before);
}

// The lowest-numbered free pages: give(rank, page) for the first `need` of
// them in ascending order.  Returns how many there are (at least `need` where
// there are more).  The reference counts are read 16 to a thread and block-wide
// round, the next round's on their way while this one's are counted, and no list of
// free pages has to be kept.
template <int THREADS, typename Give>
__device__ __forceinline__ long long take_free(const int* refs, int num_pages, long long need, long long* sums, Give give) {
  constexpr int PER = 16;
  int4 next[PER / 4];
  auto load = [&](long long base) {
    const long long at = base + threadIdx.x * PER;
#pragma unroll
    for (int i = 0; i < PER / 4; ++i) {
      const long long p = at + 4 * i;
      if (p + 4 <= num_pages) {
        next[i] = __ldcg(reinterpret_cast<const int4*>(refs + p));
      } else {
        next[i].x = p < num_pages ? __ldcg(refs + p) : 1;
        next[i].y = p + 1 < num_pages ? __ldcg(refs + p + 1) : 1;
        next[i].z = p + 2 < num_pages ? __ldcg(refs + p + 2) : 1;
        next[i].w = 1;  // (p + 3 is behind the last page)
      }
    }
  };
  long long found = 0;
  if (need > 0) load(0);
  for (long long base = 0; base < num_pages && found < need; base += THREADS * PER) {
    uint32_t free = 0;
#pragma unroll
    for (int i = 0; i < PER / 4; ++i)
      free |= ((next[i].x == 0 ? 1u : 0u) | (next[i].y == 0 ? 2u : 0u) | (next[i].z == 0 ? 4u : 0u) | (next[i].w == 0 ? 8u : 0u)) << (4 * i);
    load(base + THREADS * PER);
    long long total;
    long long rank = found + block_scan<THREADS>(__popc(free), total, sums);
    for (; free != 0 && rank < need; ++rank, free &= free - 1)
      give(rank, (int)(base + threadIdx.x * PER + (__ffs(free) - 1)));
    found += total;
  }
  return found;
}

// The last of n ascending ranks that is at most `rank`.
__device__ __forceinline__ int owner_of(const int* start, int n, long long rank) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= rank) lo = mid;
    else hi = mid;
  }
  return lo;
}

// -------------------------------------------------------------- resize --
// All latency: a few words per row and page.  A block per row gives back, then one
// block hands out, launched ahead and waiting: of 256 threads, whose barriers take
// less, or of 1024 where many counts or rows are looked over.
//   64 rows that grow by a page each 9.0 us, 10.4 with 1024 threads; with the free
//   ones behind 64000 pages 18.1 and 16.5; 4096 rows 30.7 and 26.4.  256 rows of 1024
//   pages all given back: 6.9 us, and 163 by one block that does both; 16 rows of
//   64: 2.9 and 4.2 (0.7 less where nothing is given back).
constexpr int kReleaseThreads = 128;

__global__ void __launch_bounds__(kReleaseThreads) release_kernel(const PoolParams prm, const int* __restrict__ want) {
  constexpr int AHEAD = 4;  // entries in flight per thread
  pdl_launch();
  const int row = blockIdx.x;
  bool bad = false;
  const int hold = pages_of(cut_tokens(prm.seq_k[row], prm, bad), prm.page_shift);
  const int goal = pages_of(cut_tokens(want[row], prm, bad), prm.page_shift);
  int* entries = prm.table + row * prm.table_stride;
  for (long long j0 = goal + threadIdx.x; j0 < hold; j0 += kReleaseThreads * AHEAD) {
    int page[AHEAD], held[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) page[i] = j0 + i * kReleaseThreads < hold ? entries[j0 + i * kReleaseThreads] : 0;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      held[i] = 1;
      if (j0 + i * kReleaseThreads >= hold) continue;
      entries[j0 + i * kReleaseThreads] = -1;
      held[i] = (unsigned)page[i] < (unsigned)prm.num_pages ? atomicSub(prm.refs + page[i], 1) : -1;
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (held[i] > 0) continue;
      bad = true;
      if ((unsigned)page[i] < (unsigned)prm.num_pages) atomicAdd(prm.refs + page[i], 1);  // nobody held it
    }
  }
  if (bad) report_index(prm.err);
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) resize_kernel(const PoolParams prm, const int* want) {
  extern __shared__ int start[];  // [rows] the rank of a row's first new page
  __shared__ long long sums[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  bool bad = false;  // (cut lengths have been reported by release_kernel)
  auto hold_of = [&](int row) { return pages_of(cut_tokens(prm.seq_k[row], prm, bad), prm.page_shift); };
  auto goal_of = [&](int row) { return pages_of(cut_tokens(want[row], prm, bad), prm.page_shift); };
  long long need = 0;
  for (int base = 0; base < prm.rows; base += THREADS) {
    const int row = base + threadIdx.x;
    long long total;
    const long long before = block_scan<THREADS>(row < prm.rows ? max(0, goal_of(row) - hold_of(row)) : 0, total, sums);
    if (row < prm.rows) start[row] = (int)min(need + before, (long long)INT_MAX);  // (no page has so high a rank)
    need += total;
  }
  __syncthreads();
  const long long found = take_free<THREADS>(prm.refs, prm.num_pages, need, sums, [&](long long rank, int page) {
    const int row = owner_of(start, prm.rows, rank);
    prm.table[row * prm.table_stride + hold_of(row) + (rank - start[row])] = page;
    prm.refs[page] = 1;
  });
  __syncthreads();  // the rows' old lengths have been read
  if (found >= need) {
    for (int row = threadIdx.x; row < prm.rows; row += THREADS) prm.seq_k[row] = cut_tokens(want[row], prm, bad);
    return;
  }
  // the pages ran out: the entries that got none are marked
  for (int row = warp; row < prm.rows; row += THREADS / 32) {
    const int hold = hold_of(row), goal = goal_of(row), tokens = cut_tokens(want[row], prm, bad);
    int room = goal;
    if (goal > hold) {
      room = hold + (int)max(0LL, min((long long)(goal - hold), found - start[row]));
      for (int j = room + lane; j < goal; j += 32) prm.table[row * prm.table_stride + j] = -1;
    }
    __syncwarp();  // every lane has read the row's old length
    if (lane == 0) prm.seq_k[row] = (int)min((long long)tokens, (long long)room << prm.page_shift);
  }
}

// ---------------------------------------------------------------- copy --
// Rows of a page, in 16-byte pieces: those of one plane (a layer's keys or
// values) with `tokens` rows per head, a block's share of them.  All bytes,
// each read once and written once; a thread has eight pieces on their way.
//   160 pages of 64 tokens, 8 layers of 8 heads, d = 128: 671 MB moved in 99.8 us,
//   6.7 TB/s (0.99 of the measured copy rate); call after call 99.5, and 102 where
//   each is launched at the end of the one before.
constexpr int kCopyThreads = 256, kCopyPieces = 8;

template <int D>
__device__ __forceinline__ void copy_rows(const PageRows& r, int plane, int src, int dst, int tokens, int block) {
  constexpr int PV = D / 8;  // pieces of a row
  uint16_t* base = (plane & 1 ? r.v : r.k) + (plane >> 1) * r.layer_stride;
  const uint16_t* from = base + src * r.page_stride;
  uint16_t* to = base + dst * r.page_stride;
  const unsigned n = (unsigned)(r.heads * tokens) * PV;
  const bool tokens_inside = r.token_stride <= r.head_stride;  // the order of addresses
  const unsigned inner = tokens_inside ? tokens : r.heads;
  const long long inner_stride = tokens_inside ? r.token_stride : r.head_stride;
  const long long outer_stride = tokens_inside ? r.head_stride : r.token_stride;
  uint4 x[kCopyPieces];
  long long at[kCopyPieces];
  const unsigned i0 = (unsigned)block * (kCopyThreads * kCopyPieces) + threadIdx.x;
#pragma unroll
  for (int k = 0; k < kCopyPieces; ++k) {
    const unsigned i = i0 + k * kCopyThreads;
    if (i < n) {
      const unsigned row = i / PV, o = row / inner;
      at[k] = o * outer_stride + (row - o * inner) * inner_stride + (i % PV) * 8;
      x[k] = __ldcs(reinterpret_cast<const uint4*>(from + at[k]));
    }
  }
#pragma unroll
  for (int k = 0; k < kCopyPieces; ++k)
    if (i0 + k * kCopyThreads < n) *reinterpret_cast<uint4*>(to + at[k]) = x[k];
}
// Blocks of a plane's page.
template <int D>
unsigned page_blocks(const PageRows& r) {
  const int64_t pieces = ((int64_t)r.heads << r.page_shift) * (D / 8);
  return (unsigned)((pieces + kCopyThreads * kCopyPieces - 1) / (kCopyThreads * kCopyPieces));
}

template <int D>
__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(const PageRows r, const int* src, const int* dst, int blocks, int* err) {
  pdl_launch();
  pdl_wait();
  const int pair = blockIdx.x / blocks, block = blockIdx.x - pair * blocks;
  const int a = src[pair], b = dst[pair];
  if ((unsigned)a >= (unsigned)r.num_pages || (unsigned)b >= (unsigned)r.num_pages) {
    if (threadIdx.x == 0) report_index(err);
    return;
  }
  if (a != b) copy_rows<D>(r, blockIdx.y, a, b, 1 << r.page_shift, block);
}

// ---------------------------------------------------------------- fork --
// First which forks can be done and the pages for what a source's last, partly
// filled page holds, by one block (as resize); then the table's rows, the
// reference counts and the copies, by a block for each share of them.  The two
// meet in fresh[f]: the page, kWhole (all pages full and shared), kRefused or kNoPage
// (there was none left).
constexpr int kWhole = -1, kRefused = -2, kNoPage = -3;

template <int THREADS>
__global__ void __launch_bounds__(THREADS) fork_plan_kernel(const PoolParams prm, const int* src, const int* dst, int* fresh, int n) {
  extern __shared__ int smem[];
  __shared__ long long sums[32];
  pdl_launch();
  int* start = smem;  // [n]
  const int words = (prm.rows + 31) / 32;
  uint32_t* is_src = reinterpret_cast<uint32_t*>(smem + n);
  uint32_t *is_dst = is_src + words, *twice = is_dst + words;
  for (int i = threadIdx.x; i < 3 * words; i += THREADS) is_src[i] = 0;
  __syncthreads();
  for (int f = threadIdx.x; f < n; f += THREADS) {
    const int a = src[f], b = dst[f];
    if ((unsigned)a < (unsigned)prm.rows) atomicOr(is_src + (a >> 5), 1u << (a & 31));
    if ((unsigned)b < (unsigned)prm.rows && (atomicOr(is_dst + (b >> 5), 1u << (b & 31)) >> (b & 31) & 1))
      atomicOr(twice + (b >> 5), 1u << (b & 31));
  }
  __syncthreads();
  bool bad = false;
  // what fork f needs: kWhole nothing, 0 a page, kRefused it cannot be done
  auto need_of = [&](int f) -> int {
    const int a = src[f], b = dst[f];
    if ((unsigned)a >= (unsigned)prm.rows || (unsigned)b >= (unsigned)prm.rows) return kRefused;
    if ((is_src[b >> 5] | twice[b >> 5]) >> (b & 31) & 1) return kRefused;
    bool cut = false;
    const int tokens = cut_tokens(prm.seq_k[a], prm, cut);
    if (cut || prm.seq_k[b] != 0) return kRefused;
    if ((tokens & ((1 << prm.page_shift) - 1)) == 0) return kWhole;
    return (unsigned)prm.table[a * prm.table_stride + (tokens >> prm.page_shift)] < (unsigned)prm.num_pages ? 0 : kRefused;
  };
  const int share = (n + THREADS - 1) / THREADS;
  const int f0 = min(n, (int)threadIdx.x * share), f1 = min(n, f0 + share);
  long long mine = 0, need;
  for (int f = f0; f < f1; ++f) {
    const int what = need_of(f);
    bad |= what == kRefused;
    fresh[f] = what == 0 ? kNoPage : what;
    mine += what == 0;
    start[f] = what == 0;
  }
  long long at = block_scan<THREADS>(mine, need, sums);
  for (int f = f0; f < f1; ++f) {
    const int one = start[f];
    start[f] = (int)at;
    at += one;
  }
  __syncthreads();
  take_free<THREADS>(prm.refs, prm.num_pages, need, sums, [&](long long rank, int page) {
    fresh[owner_of(start, n, rank)] = page;
    prm.refs[page] = 1;
  });
  if (bad) report_index(prm.err);
}

// (fresh is volatile: the compiler may read what is const and __restrict__ ahead of
// pdl_wait.)
template <int D>
__global__ void __launch_bounds__(kCopyThreads) fork_kernel(const PoolParams prm, const PageRows r, const int* src, const int* dst,
                                                            const volatile int* fresh) {
  pdl_wait();
  const int f = blockIdx.z, page = fresh[f];
  if (page < kWhole) return;
  const int a = src[f], b = dst[f];
  const int tokens = prm.seq_k[a], full = tokens >> prm.page_shift, rest = tokens & ((1 << prm.page_shift) - 1);
  const int* old = prm.table + a * prm.table_stride;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    int* entries = prm.table + b * prm.table_stride;
    bool bad = false;
    for (int j = threadIdx.x; j < full; j += kCopyThreads) {
      int p = old[j];
      if ((unsigned)p < (unsigned)prm.num_pages) {
        atomicAdd(prm.refs + p, 1);
      } else {
        p = -1;
        bad = true;
      }
      entries[j] = p;
    }
    if (threadIdx.x == 0) {
      if (rest > 0) entries[full] = page;
      prm.seq_k[b] = tokens;
    }
    if (bad) report_index(prm.err);
  }
  if (rest > 0) copy_rows<D>(r, blockIdx.y, old[full], page, rest, blockIdx.x);
}

// ------------------------------------------------------------- compact --
// Row i of the kept ones moves from slot keep[i] to slot first + i, keep[i] >=
// first + i.  All bytes; what has to be right is the order, since slots are both
// read and written: slot first + i is read by rows up to i alone.  So a block
// takes the rows in rounds, in order, and has read a round (RS * MOVES rows, in
// registers) before it writes it: no row behind the round reads what the round
// writes.  Between blocks there is nothing to order, as each has planes, heads and
// columns of its own.  A block's threads are PV pieces of a row (a part of the head),
// RS rows and HS heads; rows' places (three dependent look-ups) are worked out for
// kTile rows at once, into shared memory.
//   8 sequences of 12000 to 16000 tokens, 2 layers of 8 heads, 4000 of each kept:
//   344 MB in 65 us, 5.3 TB/s (a row's columns shared by two blocks; whole 74, by
//   four 71).  8 of the last 60 tokens of 32 sequences, 8 layers: 6.3 us, four
//   dependent look-ups and a round.  One sequence makes few blocks, each of which
//   waits for its own reads round after round: 4000 of 16000 tokens of 8 heads, one
//   layer 28.6 us (floor 4.8), 8 layers in one call 58 (39), 32 layers 179 (154).
// Rows in flight per thread: two where there are at most four to a thread in all (up
// to 8, 24, 64 tokens kept of 32 sequences, 8 layers: 6.3, 10.5, 16.4 us; with eight,
// which leave fewer blocks to an SM, 8.5, 14.7, 19.5), else eight (300 tokens 68.6,
// with two 70.7; the 4000 above 60.8 and 73.8, on one box).
constexpr int kCompactThreads = 256, kTile = 1024;

template <int MOVES>
__global__ void __launch_bounds__(kCompactThreads) cache_compact_kernel(const __grid_constant__ CompactParams prm, int lg_pv, int parts,
                                                                        int lg_rs, int head_groups) {
  __shared__ long long from[kTile], to[kTile];
  const int pv = threadIdx.x & ((1 << lg_pv) - 1);
  const int rs = (threadIdx.x >> lg_pv) & ((1 << lg_rs) - 1);
  const int hs = threadIdx.x >> (lg_pv + lg_rs);
  const int heads_at_once = kCompactThreads >> (lg_pv + lg_rs);
  int x = blockIdx.x;
  const int part = x % parts;
  x /= parts;
  const int group = x % head_groups, b = x / head_groups;
  const PageRows& r = prm.rows;
  const int first = prm.first[b], asked = prm.keep_n[b];
  const int n = min(max(asked, 0), prm.max_keep);
  const long long cap = (long long)prm.max_pages << r.page_shift;
  const bool teller = part == 0 && group == 0 && blockIdx.y == 0;  // speaks for the sequence
  bool bad = asked != n || first < 0 || (long long)first + n > cap;
  if (teller && threadIdx.x == 0) prm.seq_k_out[b] = (int)min(max((long long)first + n, 0LL), cap);
  const int head = group * heads_at_once + hs;
  const bool mine = head < r.heads;
  uint16_t* base = (blockIdx.y & 1 ? r.v : r.k) + (blockIdx.y >> 1) * r.layer_stride + head * r.head_stride +
                   ((part << lg_pv) + pv) * 8;
  const int* table = prm.table + b * prm.table_stride;
  auto place = [&](long long slot) -> long long {  // the row at a slot, or -1
    if (slot < 0 || slot >= cap) return -1;
    const int page = table[slot >> r.page_shift];
    if ((unsigned)page >= (unsigned)r.num_pages) return -1;
    return page * r.page_stride + (slot & ((1 << r.page_shift) - 1)) * r.token_stride;
  };
  for (int t0 = 0; t0 < n; t0 += kTile) {
    __syncthreads();  // the places of the tile before have been read
    const int rows = min(kTile, n - t0);
    for (int i = threadIdx.x; i < rows; i += kCompactThreads) {
      const long long a = prm.keep[b * prm.keep_stride + t0 + i], z = (long long)first + t0 + i;
      long long p = -1, q = -1;
      if (a != z) {
        p = place(a);
        q = place(z);
        if (a < z || p < 0 || q < 0) {
          bad = true;
          p = -1;
        }
      }
      from[i] = p;
      to[i] = q;
    }
    __syncthreads();
    for (int i0 = 0; i0 < rows; i0 += MOVES << lg_rs) {
      uint4 u[MOVES];
#pragma unroll
      for (int k = 0; k < MOVES; ++k) {
        const int i = i0 + (k << lg_rs) + rs;
        if (mine && i < rows && from[i] >= 0) u[k] = *reinterpret_cast<const uint4*>(base + from[i]);
      }
      __syncthreads();  // the round has been read
#pragma unroll
      for (int k = 0; k < MOVES; ++k) {
        const int i = i0 + (k << lg_rs) + rs;
        if (mine && i < rows && from[i] >= 0) *reinterpret_cast<uint4*>(base + to[i]) = u[k];
      }
    }
  }
  if (bad && teller) report_index(prm.err);
}

// A launch that may begin while the kernel before it in the stream still runs
// (what that one is: its blocks then wait for its end, and the next launch need not).
void dependent_launch(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, dim3 grid, unsigned threads, size_t smem, cudaStream_t stream) {
  cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

// Lets a kernel take `bytes` of dynamic shared memory, at most `most` in any call.
// (48 KB, its static part included, need no asking.)  The limit belongs to the kernel,
// not to a launch: what is asked for is always the most, so that no call lowers the
// limit between another thread's asking and its launch.
template <typename K>
cudaError_t allow_smem(K kern, size_t bytes, size_t most) {
  return bytes <= 40 * 1024 ? cudaSuccess : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}
constexpr size_t resize_smem(size_t rows) { return rows * sizeof(int); }
constexpr size_t fork_smem(size_t n, size_t rows) { return (n + 3 * ((rows + 31) / 32)) * sizeof(int); }
static_assert(resize_smem(kMaxResizeRows) <= 226 * 1024 && fork_smem(kMaxForks, kMaxForkRows) <= 226 * 1024,
              "a block's dynamic shared memory, beside the static");

}  // namespace

// Whether a pool's block has 1024 threads: see release_kernel.
static bool large_pool(int num_pages, int rows) { return num_pages > 16384 || rows > 1024; }

cudaError_t launch_pages_resize(const PoolParams& prm, const int* want, cudaStream_t stream) {
  const size_t smem = resize_smem(prm.rows);
  auto go = [&](auto kern, unsigned threads) {
    cudaError_t e = allow_smem(kern, smem, resize_smem(kMaxResizeRows));
    if (e != cudaSuccess) return e;
    release_kernel<<<(unsigned)prm.rows, kReleaseThreads, 0, stream>>>(prm, want);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    dependent_launch(cfg, attr, dim3(1, 1, 1), threads, smem, stream);
    return cudaLaunchKernelEx(&cfg, kern, prm, want);
  };
  return large_pool(prm.num_pages, prm.rows) ? go(resize_kernel<1024>, 1024) : go(resize_kernel<256>, 256);
}

cudaError_t launch_pages_fork(const PoolParams& prm, const PageRows& rows, int d, const int* src, const int* dst, int* fresh, int n,
                              cudaStream_t stream) {
  const size_t smem = fork_smem(n, prm.rows);
  auto plan = [&](auto kern, int threads) {
    const cudaError_t e = allow_smem(kern, smem, fork_smem(kMaxForks, kMaxForkRows));
    if (e != cudaSuccess) return e;
    kern<<<1, threads, smem, stream>>>(prm, src, dst, fresh, n);
    return cudaGetLastError();
  };
  const cudaError_t e = large_pool(prm.num_pages, n) ? plan(fork_plan_kernel<1024>, 1024) : plan(fork_plan_kernel<256>, 256);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  auto go = [&](auto kern, unsigned blocks) {
    dependent_launch(cfg, attr, dim3(blocks, 2u * rows.layers, (unsigned)n), kCopyThreads, 0, stream);
    return cudaLaunchKernelEx(&cfg, kern, prm, rows, src, dst, (const volatile int*)fresh);
  };
  switch (d) {
    case 64: return go(fork_kernel<64>, page_blocks<64>(rows));
    case 128: return go(fork_kernel<128>, page_blocks<128>(rows));
    case 256: return go(fork_kernel<256>, page_blocks<256>(rows));
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_cache_copy(const PageRows& rows, int d, const int* src, const int* dst, int n, int* err, cudaStream_t stream) {
  auto go = [&](auto kern, unsigned blocks) {
    if ((int64_t)blocks * n > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    dependent_launch(cfg, attr, dim3(blocks * (unsigned)n, 2u * rows.layers, 1), kCopyThreads, 0, stream);
    return cudaLaunchKernelEx(&cfg, kern, rows, src, dst, (int)blocks, err);
  };
  switch (d) {
    case 64: return go(cache_copy_kernel<64>, page_blocks<64>(rows));
    case 128: return go(cache_copy_kernel<128>, page_blocks<128>(rows));
    case 256: return go(cache_copy_kernel<256>, page_blocks<256>(rows));
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_cache_compact(const CompactParams& prm, int d, int sms, cudaStream_t stream) {
  auto log2_up = [](int64_t n) {
    int l = 0;
    while (((int64_t)1 << l) < n) ++l;
    return l;
  };
  // Rows at once: all that there can be, up to what a block's threads hold, and
  // the threads left over for more heads.  Where that makes too few blocks to
  // fill the GPU, a row's columns are shared out, down to 64 bytes.
  int lg_pv = log2_up(d / 8), parts = 1, lg_rs, groups;
  for (;;) {
    lg_rs = log2_up(prm.max_keep);
    if (lg_rs > 8 - lg_pv) lg_rs = 8 - lg_pv;
    const int at_once = kCompactThreads >> (lg_pv + lg_rs);
    groups = (prm.rows.heads + at_once - 1) / at_once;
    const int64_t blocks = (int64_t)prm.B * groups * parts * 2 * prm.rows.layers;
    if (blocks >= 2 * sms || lg_pv <= 2) break;
    --lg_pv;
    parts *= 2;
  }
  const int64_t x = (int64_t)prm.B * groups * parts;
  if (x > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto go = [&](auto kern) {
    kern<<<dim3((unsigned)x, 2u * prm.rows.layers, 1), kCompactThreads, 0, stream>>>(prm, lg_pv, parts, lg_rs, groups);
    return cudaGetLastError();
  };
  return prm.max_keep <= 4 << lg_rs ? go(cache_compact_kernel<2>) : go(cache_compact_kernel<8>);
}

}  // namespace fa
