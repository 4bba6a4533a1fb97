// tree.cu -- the layout of trees of drafted tokens: which nodes a node descends
// from, and the position that its depth gives it.
#include <cstdint>

#include "paged_search.cuh"
#include "ptx_window.cuh"
#include "tree.h"

namespace fa {
namespace {

// One warp per node climbs from it to its root; lane l keeps word l of the mask
// row.  All latency: a step would be a dependent load, so the warp loads the 32
// parents around the node it has come to at once and climbs by shuffles until it
// leaves them (parents lie before their nodes, so a tree of n nodes takes at most
// n / 32 + 1 loads, whatever its depth).  Under a window that the path is longer
// than, sinks among the nodes are known once its length is: it is climbed again.
constexpr int kPlanThreads = 128;

template <bool WINDOW>  // whether a tree can be deeper than the window
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(const int* __restrict__ parents, const int* __restrict__ cu_q,
                                                                 const int* __restrict__ seq_k, int B, int T,
                                                                 uint32_t* __restrict__ mask, int words,
                                                                 int* __restrict__ positions, int window, int sinks, int* err) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kPlanThreads / 32) + (threadIdx.x >> 5);
  if (t >= T) return;
  const int b = find_sequence(cu_q, B, t, lane);
  const int q0 = max(0, cu_q[b]), q1 = min(T, cu_q[b + 1]);  // (cut as the other calls cut them)
  if (t < q0 || t >= q1) return;  // a row that belongs to no sequence
  const int n = q1 - q0, self = t - q0, first = seq_k[b] - n;
  uint32_t word = 0;
  int depth = 0;
  bool bad = false;
  if (n > 32 * words) {
    // a chunk of a prompt: each token follows the one before
    const int left = self + 1 - 32 * lane;
    word = left <= 0 ? 0u : left >= 32 ? 0xffffffffu : (1u << left) - 1;
    depth = self;
    bad = parents[t] != self - 1;
  } else {
    int have = -1, mine = -1;
    // of the nodes above, those less than `window` steps up are seen, and those more
    // than `beyond`: there the positions are the sinks'
    long long beyond = n;
    for (;;) {
      int at = self, steps = 0;
      for (;;) {
        if (lane == at >> 5 && (!WINDOW || steps < window || steps > beyond)) word |= 1u << (at & 31);
        if (at >> 5 != have) {
          have = at >> 5;
          mine = 32 * have + lane < n ? parents[q0 + 32 * have + lane] : -1;
        }
        const int up = __shfl_sync(0xffffffffu, mine, at & 31);
        bad |= up < -1 || up >= at;  // (such a node counts as a root, so the climb ends)
        if (up < 0 || up >= at) break;
        at = up;
        ++steps;
      }
      depth = steps;
      if (!WINDOW || beyond < n || depth < window || first >= sinks) break;
      beyond = max(-1LL, (long long)first + depth - sinks);  // (below depth)
    }
  }
  if (lane < words) mask[(long long)t * words + lane] = word;
  if (lane == 0) {
    positions[t] = first + depth;
    if (bad) report_index(err);
  }
}

}  // namespace

cudaError_t launch_tree_plan(const int* parents, const int* cu_q, const int* seq_k, int B, int T, uint32_t* mask, int words,
                             int* positions, int window, int sinks, int* err, cudaStream_t stream) {
  const int per = kPlanThreads / 32;
  auto go = [&](auto kern) {
    kern<<<(unsigned)((T + (long long)per - 1) / per), kPlanThreads, 0, stream>>>(parents, cu_q, seq_k, B, T, mask, words, positions,
                                                                                  window, sinks, err);
    return cudaGetLastError();
  };
  // (without the window's steps 60 nodes of 32 trees take 0.9 us less)
  return window < 32 * words ? go(tree_plan_kernel<true>) : go(tree_plan_kernel<false>);
}

}  // namespace fa
