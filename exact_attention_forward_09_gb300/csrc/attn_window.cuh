// attn_window.cuh -- attention forward under a sliding window with sinks, on
// dense tensors and over a paged key/value cache, for sm_103a (tcgen05 + TMEM
// + TMA).
//
// What it computes, for a query at position p of its sequence:
//   O = sum_j softmax_j(scale q . k_j) v_j,   LSE = ln sum_j exp(scale q . k_j)
// over the visible keys: j <= p and (j > p - window or j < sinks).  A window
// of at least the sequence length makes it plain causal attention.
//
// Key tiles.  A query tile visits the 128-key tiles that hold a sink (first
// `ns` tiles) and those from its first row's window start to its last row's
// position; the tiles between the two are skipped (never loaded nor
// multiplied).  The visited tiles are numbered 0 .. L-1 without the gap
// ("list index"); with two query tiles per CTA the list is the union of both
// tiles' ranges and each tile takes part in its own list indices only.
//
// The CTA is organised as the full-mask kernel of attn_fwd.cuh: a load warp
// (TMA through an NS-slot ring), an MMA warp that issues S = Q K^T and
// O += P V with P in TMEM, and one softmax warpgroup per query tile with one
// thread per row and a lazily rescaled O.  What differs is described where it
// happens: visibility as four 32-bit words per row and tile, and, for PAGED:
//   * rows: the g query heads of a key/value head are packed, row = token * g
//     + head, so that each key/value byte is read once per group;
//   * pages: a key tile is gathered by one TMA box per page (4-D map: column,
//     row in page, head, page); pages without a visible key are not read;
//   * work: the (sequence, query group, head) units of the ragged batch are
//     laid end to end in units of key tiles and every CTA takes an equal run
//     of that line, so that one long sequence, or a few, fill the GPU as well
//     as many; a unit that is cut leaves fp32 partial results (O normalised
//     over its run and the run's LSE), which a second kernel joins by LSE
//     weights.  Every CTA derives the line from cu_q and seq_k itself, so a
//     captured graph follows lengths that change on the device;
//   * what no query may see but a key tile holds all the same (rows behind
//     the sequence's end in its last page, pages that left the window) may be
//     anything, NaN included: its scores are replaced, and its V rows are
//     zeroed in shared memory before P V.
// and for TREE (of PAGED), where a sequence's new tokens are the nodes of a tree:
//   * a node's row sees the cached keys by its own position (the window's start)
//     and the new keys by the bits of its mask row.  Only the tiles that hold a new
//     key are masked so (one or two at the end of a context), out of line;
//   * every unit of a sequence starts its window at the first position that a
//     node can have, the cached tokens' end, as a node's position is known to its own
//     row alone; nodes lie one behind the other up to their own slot, as tokens do;
//   * sequences of more tokens than a mask row has bits are plain chunks.
//
// Roundings.  Scores, maxima, sums, O and the parts that are joined are fp32.  P
// is rounded to the element type: both operands of a 16-bit MMA have one type, and
// P in two 16-bit pieces would double P V.  It is rounded before its division by
// the row's sum, which is taken of the unrounded P.  With O's own rounding that
// makes a relative error against 64 bits of 2.0 to 2.4e-3 in bf16 and 2.5 to 2.9e-4
// in fp16, where rounding O alone gives 1.6e-3 and 2.1e-4.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_fwd.cuh"
#include "ptx_window.cuh"

namespace fa {

// The kernel's forms.
// WIN_PAIR (d <= 128): two query tiles per CTA.  On long chunks and dense calls
// the fastest: it reads each key tile once for two query tiles (500 against 566
// us for 4 x 2048 tokens over 4000 to 10000 keys, d = 64).
// WIN_ONE: one query tile per CTA; all of d = 256, and paged batches whose
// sequences mostly bring few rows.  There one query tile of a pair would be in
// use, and a key tile's chain (S, softmax, P V) be all that runs in its CTA.
// So d = 128 takes the room of the second query tile for a second S buffer, as
// d = 256 does (one token each, 32/8 heads: 256 sequences under a window of
// 1024 278 -> 227 us, one of 131000 keys 36.0 -> 32.9), and d = 64 runs two
// CTAs per SM: two chains (64 sequences of 2000 to 16000 keys 310 -> 220 us).
// WIN_FEW: as WIN_ONE, for units of at most FEW_ROWS rows (a token's g heads,
// or a few tokens').  One softmax warp would do the work of a whole key tile
// for a few rows while three work on rows that do not exist.  So the rows lie
// four times in the query tile, at rows 0, 32, 64 and 96, and with that in the
// TMEM lanes of each warp; warp w exponentiates columns 32 w .. 32 w + 31 alone,
// for its copy, and hands over zeros for the others.  The four copies are
// attention over disjoint keys, joined by their maxima and sums when the unit
// ends.  (One token each, 32/8 heads, against WIN_ONE: 256 sequences under a
// window of 1024 at d = 64, 128, 256: 149 -> 107, 224 -> 186, 430 -> 367 us; of
// 50 to 600 keys 78 -> 62, 125 -> 115, 190 -> 168; 64 of 2000 to 16000 at d = 64
// 224 -> 195, 6.5 TB/s.)  An infinite value in a row of V that is seen gives
// NaN, as the copies that do not take its key weigh it with 0; the other forms
// give infinity unless a row of the tile weighs it with 0.
// WIN_FEW2 (d <= 128): the same with two CTAs per SM, where a unit's start and
// end pass while the other CTA works.  At d = 128 it takes units of up to 8 rows
// and half the tiles in flight, and pays where units are many (256 of 50 to 600
// keys 116 -> 96 us, 64 of 2000 to 16000 373 -> 360; under the window of 1024
// 185 -> 194) and not where few are cut in many parts (one of 131000 keys, 16/2
// heads, 32.2 against 34.8).
// WIN_SPLIT (dense): one query tile per cluster, whose CTAs take runs of its key
// tiles and join their results through each other's shared memory, for calls
// of so few query tiles that most SMs would idle.  (d = 128, 8/2 heads over 8000
// keys without a window: 1 query 81.4 -> 14.5 us, 100 82.0 -> 16.5, 1000 82.0 ->
// 38.7; 12 heads, window 500, 1 and 100 queries: 13.4 -> 9.4, 15.4 -> 10.8.)
// WIN_TWO (dense, d = 64): two CTAs of one query tile per SM, for short windows,
// whose units' starts and ends pass while the other CTA works (2 x 4096 tokens,
// 16/4 heads, window 128, 256, 512, 1024: 32.2 -> 28.0, 37.5 -> 33.0, 42.7 ->
// 41.3, 56.3 -> 56.6 us; 64 x 128 tokens, 8 heads 16.1 -> 11.0), where there is
// more than one query tile per SM (72 tiles of 1025 tokens: +1 us of 9).  At d =
// 128 it costs 5 to 25%: twice the key tiles from L2, and half the ring each.
enum WinForm { WIN_FEW, WIN_FEW2, WIN_ONE, WIN_PAIR, WIN_SPLIT, WIN_TWO };
constexpr int few_rows(int d, int form) { return form == WIN_FEW2 && d == 128 ? 8 : 16; }

template <int ELEM, int D, bool PAGED, int FORM = (D <= 128 ? WIN_PAIR : WIN_ONE)>
struct WinCfg {
  static constexpr bool PAIR = FORM == WIN_PAIR, FEW = FORM == WIN_FEW || FORM == WIN_FEW2,
                        SPLIT = FORM == WIN_SPLIT;
  static_assert(ELEM == kBF16 || ELEM == kFP16, "16-bit operands");
  static constexpr int D_ = D, ELEM_ = ELEM;
  static constexpr int ROW_BYTES = D * 2;
  static constexpr int CH_ELEMS = 64;                      // elements per 128-byte chunk
  static constexpr int NCH = D / CH_ELEMS;
  static constexpr int CHUNK_BYTES = 128 * 128;            // 128 rows x 128 bytes
  static constexpr int NQT = PAIR ? 2 : 1;                 // query tiles per CTA
  static constexpr bool ALT = PAIR || FORM == WIN_FEW2 || (D == 64 && !SPLIT);             // one S buffer per query tile; ring K0 V0 K1 V1 ...
  static constexpr int OCC = ALT && !PAIR ? 2 : 1;         // CTAs per SM
  static_assert(!PAIR || D <= 128, "two query tiles of d = 256 exceed tensor memory");
  static_assert((OCC == 1 && !FEW) || PAGED || FORM == WIN_TWO, "a paged form");
  static_assert(FORM != WIN_TWO || (!PAGED && D == 64), "dense calls at d = 64");
  static_assert(!SPLIT || !PAGED, "paged units are cut along the line of work");
  static constexpr int FEW_ROWS = few_rows(D, FORM);
  static constexpr int ML_BYTES = FEW ? 4 * FEW_ROWS * 8 : (SPLIT ? kBM * 8 : 0);
  // WIN_FEW2, d = 128: the column chunks of the query tile lie in each other's unused rows
  static constexpr bool Q_PACKED = FEW && FEW_ROWS == 8;
  // shared memory of a CTA: what two per SM leave beside their reserves
  static constexpr int SMEM_LIMIT = OCC == 2 ? 115712 : kSmemLimit;
  static constexpr int TILE_BYTES = kBN * ROW_BYTES;
  static constexpr int SLOT_BYTES = TILE_BYTES < 32768 ? TILE_BYTES : (OCC == 2 ? 16384 : 32768);
  static constexpr int SPT = TILE_BYTES / SLOT_BYTES;      // ring slots per tile
  static constexpr int SLOT_CH = SLOT_BYTES / CHUNK_BYTES;
  static constexpr int SLOT_D = SLOT_CH * CH_ELEMS;
  static constexpr int Q_CHUNK = Q_PACKED ? FEW_ROWS * 128 : CHUNK_BYTES;
  static constexpr int Q_BYTES = Q_PACKED ? CHUNK_BYTES + Q_CHUNK : NQT * kBM * ROW_BYTES;
  // dense d <= 128: O goes out through per-warp staging boxes and bulk tensor
  // copies (as attn_fwd.cuh); a paged row tile ends inside its neighbours'
  // rows, so there every thread stores its own row
  static constexpr bool EPI_TMA = !PAGED && D <= 128 && !SPLIT;
  static constexpr int EPI_WARP_BYTES = 32 * 64 * 2;
  static constexpr int EPI_BYTES = EPI_TMA ? 4 * NQT * EPI_WARP_BYTES : 0;
  static constexpr int NS_MAX = (SMEM_LIMIT - 2048 - ML_BYTES - EPI_BYTES - Q_BYTES) / SLOT_BYTES;
  static constexpr int NS = NS_MAX > 8 ? 8 : NS_MAX;
  static_assert(NS >= 2 * SPT, "ring too shallow");
  static constexpr int P_COLS = kBN / 2;
  static constexpr uint32_t TMEM_COLS = 512 / OCC;
  static constexpr uint32_t O_COL0 = OCC == 2 ? 128 : 256;  // behind the S / P buffers at 0 and (but for OCC 2) 128
  static_assert(O_COL0 + NQT * D <= TMEM_COLS, "TMEM budget");
  static constexpr int SOFTMAX_WARPS = 4 * NQT;
  static constexpr int MMA_WARP = SOFTMAX_WARPS;
  static constexpr int LOAD_WARP = SOFTMAX_WARPS + 1;
  // paged: a second load warp takes the V tiles.  A box is one page's rows of
  // one 128-byte column chunk, and a warp issues one about every 80 clocks: at
  // 16-token pages a K and a V tile of d = 128 are 32 boxes, as long to issue
  // as the tiles' arithmetic takes (chunks over 16-token pages: 652 -> 590 us
  // for 4 x 2048 new tokens over 4000 to 10000 keys).  Two CTAs per SM at d = 64
  // do without: half the boxes, and registers for no more warps.
  static constexpr bool V_WARP = PAGED && (OCC == 1 || D == 128);
  static constexpr int LOADV_WARP = V_WARP ? LOAD_WARP + 1 : -1;
  static constexpr int UNIT_READERS = SOFTMAX_WARPS + 1 + (V_WARP ? 1 : 0);  // warps that release a unit's slot
  // two query tiles: a third, control warpgroup gives registers to the
  // softmax warpgroups (the split of attn_fwd.cuh)
  static constexpr bool REALLOC = PAIR;
  static constexpr int THREADS = REALLOC ? 32 * (SOFTMAX_WARPS + 4) : 32 * (SOFTMAX_WARPS + (V_WARP ? 3 : 2));
  static constexpr int CTRL_REGS = 104;
  static constexpr int SOFTMAX_REGS = 200;
  // A few sinks are usually all that is seen of tile 0: then only its first
  // NARROW keys are multiplied and exponentiated (an MMA with N = 32 runs at
  // 40% of the N = 128 rate, so the tile costs a third of a full one).
  static constexpr int NARROW = 32;
  static constexpr uint32_t IDESC_QK_NARROW = instr_desc(ELEM == kBF16 ? 1u : 0u, ELEM == kBF16 ? 1u : 0u, 0, 0, 128, NARROW);
  static constexpr float TAU = 8.0f;                       // lazy-rescale threshold, log2 units
  static constexpr uint32_t FMT = ELEM == kBF16 ? 1u : 0u;
  static constexpr uint32_t IDESC_QK = instr_desc(FMT, FMT, 0, 0, 128, kBN);
  static constexpr uint32_t IDESC_PV = instr_desc(FMT, FMT, 0, 1, 128, SLOT_D);
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = Q_BYTES;
  static constexpr int OFF_EPI = OFF_RING + NS * SLOT_BYTES;
  static constexpr int OFF_BAR = OFF_EPI + EPI_BYTES;
  static_assert(OFF_EPI % 1024 == 0 && OFF_BAR % 1024 == 0, "1024-byte swizzle atoms");
  static constexpr int OFF_ML = OFF_BAR + 1024;                // WIN_FEW: maxima and sums, [row][warp]; WIN_SPLIT: [row]
  static constexpr int OFF_WEIGHT = OFF_Q;                     // WIN_SPLIT: [row][CTA], over Q, which is done with
  static constexpr int SMEM_BYTES = OFF_ML + ML_BYTES + 1024;  // + alignment slack
  static_assert(SMEM_BYTES <= SMEM_LIMIT, "shared memory budget");
  static_assert(!SPLIT || NS * SLOT_BYTES >= kBM * D * 4, "WIN_SPLIT leaves its part of O in the ring");
};

struct WinParams {
  void* o;            // dense [BH, N, D]; paged [T, Hq, D]
  float* lse;         // dense [BH, N]; paged [T, Hq]
  int* err;           // device error word
  int window, sinks;  // both at most 2^30
  float scale_log2;   // scale * log2(e), never zero
  int Hq, Hkv;
  int o_vec32;        // o is 32-byte aligned
  int drop_pos;       // test hook: ring position CTA 0 never fills (-1: none)
  // dense
  int N, Nk;          // query rows / keys per head
  int BH;             // batch x query heads
  int head_chunk;     // heads taken together, heaviest units first (see attn_fwd.cuh)
  int pair_units;     // units that hold two query tiles; the groups behind them run as units of one
  // paged
  const int* cu_q;    // [B + 1] first token of each sequence in q
  const int* seq_k;   // [B] keys per sequence, the new tokens' included
  const int* table;   // [B, table_stride] page of each run of page_size keys
  int B, T;
  int max_pages;      // table entries per sequence
  long long table_stride;
  int num_pages, page_shift;
  int g;              // query heads per key/value head
  int tpt;            // tokens per query tile (tpt * g <= 128)
  uint32_t max_places;  // the longest line of work of token ranges that do not overlap, below 2^31
  float* o_part;      // [2 * grid][slot rows][D] partial results of cut units
  float* lse_part;    // [2 * grid][slot rows], NQT * 128 of them
  int4* desc;         // [grid] cut units: {parts, first token, kv head, rows}
  // trees
  const uint32_t* mask;  // [T, words] which new tokens of its sequence a token sees
  const int* positions;  // [T] positions of the tokens in their sequence; null: where they lie
  int words;             // 32 words is at most 2^30
};

// The key tiles that a unit of up to two query tiles visits.
struct WinTiles {
  int ns, skip;       // list index l is tile l (l < ns) or l + skip
  int len;            // list length
  int sa[2], la[2], lb[2];  // query tile t takes part in l < sa[t] and in la[t] <= l < lb[t]
};

// Visited tiles of a query tile whose valid rows sit at positions first ..
// last (last <= nk - 1): window tiles [w0, w1), sink tiles [0, sk).
__host__ __device__ __forceinline__ void win_range(int first, int last, int window, int sinks, int& w0, int& w1,
                                                   int& sk) {
  w1 = last < 0 ? 0 : last / kBN + 1;
  const int lo = first - window + 1;
  w0 = lo > 0 ? lo / kBN : 0;
  if (w0 > w1) w0 = w1;
  sk = (sinks + kBN - 1) / kBN;
  if (sk > w1) sk = w1;
}

// p0: position of the unit's first token; ntok: its valid tokens, tpt to a query tile;
// base: a position at which any of them may sit (trees).
__host__ __device__ __forceinline__ WinTiles win_tiles(int p0, int ntok, int tpt, int nqt, int window, int sinks,
                                                       int base = 0x7fffffff) {
  WinTiles u;
  int w0[2] = {0, 0}, w1[2] = {0, 0}, sk[2] = {0, 0};
  const int n0 = ntok < tpt ? ntok : tpt;
  auto from = [&](int first) { return first < base ? first : base; };
  win_range(from(p0), p0 + n0 - 1, window, sinks, w0[0], w1[0], sk[0]);
  const bool two = nqt == 2 && ntok > tpt;
  if (two) win_range(from(p0 + tpt), p0 + ntok - 1, window, sinks, w0[1], w1[1], sk[1]);
  const int top = two ? w1[1] : w1[0];
  u.ns = two ? sk[1] : sk[0];
  u.skip = w0[0] > u.ns ? w0[0] - u.ns : 0;
  u.len = top - u.skip;
  for (int t = 0; t < 2; ++t) {
    auto index = [&](int x) { return x <= u.ns ? x : (x - u.skip > u.ns ? x - u.skip : u.ns); };
    u.sa[t] = sk[t];
    u.la[t] = index(w0[t]) > sk[t] ? index(w0[t]) : sk[t];
    u.lb[t] = index(w1[t]) > u.la[t] ? index(w1[t]) : u.la[t];
  }
  return u;
}

// One unit as the load warp hands it to the other roles.
struct alignas(16) WinUnit {
  int kz;       // key/value coordinate (dense: batch * Hkv + head; paged: head); -1: no more units
  int qz;       // query coordinate (dense: batch * Hq + head; paged: first token in q)
  int q_row;    // dense: first row
  int p0;       // position of the first token
  int ntok;     // valid tokens (dense: rows) of the unit
  int nk;       // keys of the sequence
  int ns, skip;
  int r0, r1;   // the run of list indices to do
  int sa[2], la[2], lb[2];
  int part;     // -1: whole unit, written to o; else the partial slot
  int lo;       // keys in [sinks, lo) are visible to no query of the unit
  int seq;      // paged: sequence
  int narrow;   // tile 0 is visited for its sinks alone, which lie in its first NARROW columns
};
static_assert(sizeof(WinUnit) == 80, "WinUnit is copied in 16-byte pieces");

// The list indices of one query tile.  (Selected rather than indexed: t is a
// run-time value in the softmax warps, and the unit stays in registers.)
struct WinPart {
  int sa, la, lb;
  __device__ __forceinline__ WinPart(const WinUnit& w, int t)
      : sa(t ? w.sa[1] : w.sa[0]), la(t ? w.la[1] : w.la[0]), lb(t ? w.lb[1] : w.lb[0]) {}
  __device__ __forceinline__ int count(int r0, int r1) const {  // of [r0, r1)
    return max(0, min(r1, sa) - r0) + max(0, min(r1, lb) - max(r0, la));
  }
  // the first of them at or behind l, where there is one
  __device__ __forceinline__ int from(int l) const { return l < sa || l >= la ? l : la; }
};
__device__ __forceinline__ int win_count(const WinUnit& w, int t) { return WinPart(w, t).count(w.r0, w.r1); }

template <int NS>
struct WinBars {
  uint64_t q_full, q_empty;
  uint64_t full[NS], empty[NS];
  uint64_t s_full[2];
  uint64_t p_full[2][2];   // [S/P buffer][half of the key tile]
  uint64_t o_ready[2];
  uint64_t o_full[2];
  uint64_t drain, clc_bar;
  uint64_t unit_full[2], unit_empty[2];
  alignas(16) uint32_t clc_resp[4];
  WinUnit unit[2];
  // the line of work (paged): per-warp sums, then the unit this CTA's run starts in
  uint32_t warp_sum[12];
  int start_b, start_tok0, start_nq, start_nk, start_group, start_len, start_at;
  uint32_t start_off;
  uint32_t tmem_base;
  int abort_flag;
};

// One sequence of the ragged batch.  Values that would lead out of range
// (they are device data, so the host cannot refuse them) are cut to what
// exists; *bad is then set.
struct WinSeq {
  int tok0, nq, nk;
};
__device__ __forceinline__ WinSeq win_seq(const WinParams& prm, int a, int e, int n, bool* bad) {
  WinSeq s;
  s.tok0 = min(max(a, 0), prm.T);
  const int end = min(max(e, s.tok0), prm.T);
  s.nq = end - s.tok0;
  const long long cap = (long long)prm.max_pages << prm.page_shift;
  s.nk = (long long)n > cap ? (int)cap : (n < 0 ? 0 : n);
  if (s.nk > (1 << 30)) s.nk = 1 << 30;
  if (s.tok0 != a || end != e || s.nk != n) *bad = true;
  return s;
}
// Whether a sequence's nq new tokens are a tree's nodes (else a plain chunk).
__device__ __forceinline__ bool win_is_tree(const WinParams& prm, int nq) { return nq <= 32 * prm.words; }
// Key tiles of query group i (at least 1, so that a group without visible
// keys still has its place on the line and gets its zero rows written).
template <bool TREE>
__device__ __forceinline__ int win_group_len(const WinParams& prm, const WinSeq& s, int tpg, int i) {
  const int first = s.nk - s.nq + i * tpg;
  const int last = min(first + tpg, s.nk) - 1;
  int w0, w1, sk;
  win_range(TREE && win_is_tree(prm, s.nq) ? s.nk - s.nq : first, last, prm.window, prm.sinks, w0, w1, sk);
  const int len = w1 - max(0, w0 - sk);
  return len > 0 ? len : 1;
}
// Places on the line of a unit of `len` key tiles: two to a tile when both
// query tiles are in use (such a step takes 1.8 times a single one's time),
// one otherwise, rounded up to even, so that CTAs, which start at even
// places, start at whole tiles.  (Forms with one query tile per CTA: one each.)
// A unit's start and end are not counted, so runs that hold many short units
// take longer than others.
// Trees, whose sequences seldom fill their query tiles evenly, are counted closer to
// what they take: two tiles' places more for each unit, behind its tiles' own
// (32 x 60 nodes over 1000 to 8000 keys 152.7 -> 142.2 us, 200 x 20 to 60 over 100 to 600
// 182 -> 156; with one tile's places 146.8 and 165; with three 141.6 and 158, but 32 x
// 16 nodes 111.5 -> 113.6), and as much for a step of one query tile as for one of two,
// since its chain takes nearly as long (8 chunks of 1000 tokens beside 25 trees of 1 to
// 40 nodes, over 5000 to 8000 keys 504 -> 349 us, 8 x 200 nodes 105 -> 80; 30 trees of 1
// to 40 under a window of 1000 26.3 -> 29.8, which now take the form with one query
// tile, 25.1).  A run that begins behind a unit's tiles has none of it.
template <int NQT, bool TREE>
__device__ __forceinline__ uint32_t win_places(int len, int ntok, int tpt) {
  if (NQT == 1 || TREE) return (uint32_t)(NQT * len);
  return ntok > tpt ? 2u * (uint32_t)len : ((uint32_t)len + 1u) & ~1u;
}
template <int NQT, bool TREE>
constexpr uint32_t end_places() { return TREE ? 2u * NQT : 0u; }

// bits [0, n) of a 32-bit word, n clamped to 0..32
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : (0xffffffffu >> (32 - (n < 32 ? n : 32)));
}

// Which of the 32 keys from c0 on the query at position p sees: those up to
// its own, and from its window's first on or below `sinks`.
__device__ __forceinline__ uint32_t win_visible(int p, int window, int sinks, int c0) {
  return low_bits(p + 1 - c0) & (~low_bits(p - window + 1 - c0) | low_bits(sinks - c0));
}

// Which of the 32 keys from c0 on a tree's node sees that sits at position p and
// lies at `slot`: the cached keys (below ctx) as above, and the new ones up to
// its own that `bits`, the part of its mask row, has.
__device__ __forceinline__ uint32_t tree_visible(uint32_t bits, int ctx, int slot, int p, int window, int sinks, int c0) {
  const uint32_t cached = low_bits(ctx - c0);
  return (cached & (~low_bits(p - window + 1 - c0) | low_bits(sinks - c0))) | (bits & low_bits(slot + 1 - c0) & ~cached);
}

// The softmax of a narrow tile, the first one of its rows: 32 columns of S at
// s_addr, of which `see` are visible; P is written back over them.  Returns
// the row's maximum (log2 units) and sum.  Out of line, so that the full
// tile's loop keeps its registers.
template <int ELEM>
__device__ __noinline__ float2 narrow_softmax(uint32_t s_addr, uint32_t see, float cj) {
  const float mask_val = cj < 0.0f ? INFINITY : -INFINITY;
  uint32_t u[32];
  tmem_ld32(s_addr, u);
  tmem_wait_ld();
  float mx = mask_val;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float x = (see & (1u << i)) ? __uint_as_float(u[i]) : mask_val;
    u[i] = __float_as_uint(x);
    mx = cj < 0.0f ? fminf(mx, x) : fmaxf(mx, x);
  }
  const float m = mx * cj;
  const float nm = m == -INFINITY ? 0.0f : -m;
  float l = 0.0f;
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float a = ex2(fmaf(__uint_as_float(u[2 * i]), cj, nm)), b = ex2(fmaf(__uint_as_float(u[2 * i + 1]), cj, nm));
    l += a + b;
    pk[i] = ELEM == kBF16 ? pack_bf16x2(a, b) : pack_f16x2(a, b);
  }
  tmem_st16(s_addr, pk);
  tmem_wait_st();
  return make_float2(m, l);
}

// What a row of a unit needs to know which keys it sees, in a batch of trees.
// tok: its token in the unit; real: whether the row exists (others see the cached
// keys).  A plain chunk's token takes all keys up to its own as cached ones.
template <bool TREE>
struct WinTreeRow {
  int ctx, slot, pos;
  const uint32_t* row;
  __device__ __forceinline__ WinTreeRow(const WinParams& prm, const WinUnit& w, int tok, bool real) {
    if constexpr (TREE) {
      ctx = w.p0 - w.q_row;
      pos = slot = w.p0 + tok;
      row = nullptr;
      if (!win_is_tree(prm, w.nk - ctx)) {
        ctx = slot + 1;
      } else if (real) {
        row = prm.mask + (long long)(w.qz + tok) * prm.words;
        if (prm.positions && prm.window < w.nk) {  // (else the window reaches over the whole sequence)
          const int p = prm.positions[w.qz + tok];
          pos = min(max(p, ctx), slot);  // (a node has as many nodes above it as lie before it at most)
          if (p != pos) report_index(prm.err);
        }
      }
    }
  }
  __device__ __forceinline__ uint32_t see(const WinParams& prm, int c0) const {
    const int at = (c0 - ctx) >> 5;  // (the word of the first key; below 0: the nodes begin behind it)
    const uint32_t lo = row && (unsigned)at < (unsigned)prm.words ? row[at] : 0u;
    const uint32_t hi = row && (unsigned)(at + 1) < (unsigned)prm.words ? row[at + 1] : 0u;
    return tree_visible(__funnelshift_r(lo, hi, (c0 - ctx) & 31), ctx, slot, pos, prm.window, prm.sinks, c0);
  }
};

// Replaces the scores that a row does not see, in a batch of trees: 128 of them at
// s_addr, of the keys from c0 on.  Out of line, and a loop: it runs once or twice
// per unit, and straight code would be fetched from memory line by line (unrolled
// in the tile loop it took 4 us of a call's last tile, and 2 us of each short
// unit; looked up ahead of the scores, with more code, 1 us).
static __device__ __noinline__ void tree_mask_scores(uint32_t s_addr, int c0, const uint32_t* row, int words, int ctx, int slot,
                                                     int pos, int window, int sinks, float mask_val) {
  int at = (c0 - ctx) >> 5;  // the word that holds the first key's bit (below 0: the nodes begin behind it)
  const int shift = (c0 - ctx) & 31;
  auto word = [&](int i) { return (unsigned)i < (unsigned)words ? row[i] : 0u; };
  if (row == nullptr) words = 0;
  uint32_t lo = word(at);
#pragma unroll 1
  for (int q = 0; q < 4; ++q, c0 += 32, s_addr += 32) {
    const uint32_t hi = word(++at);
    const uint32_t see = tree_visible(__funnelshift_r(lo, hi, shift), ctx, slot, pos, window, sinks, c0);
    lo = hi;
    if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
    uint32_t u[32];
    tmem_ld32(s_addr, u);
    tmem_wait_ld();
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      uint32_t x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = (see & (1u << (h + i))) ? u[h + i] : __float_as_uint(mask_val);
      tmem_st16(s_addr + h, x);
    }
  }
  tmem_wait_st();
}

// Waits for the V tile at ring position pv and, where `dead`, zeroes this
// thread's row of it (row: its shared-memory address in slot 0); made visible
// to the tensor core.  Neighbouring threads start at different 16-byte pieces,
// as equal ones share their banks.  Out of line: it runs once or twice per unit.
template <typename C, typename Bars>
__device__ __noinline__ bool clear_v_row(Bars* bars, uint32_t row, int pv, bool dead, int* err) {
  for (int sp = 0; sp < C::SPT; ++sp)
    if (!__all_sync(0xffffffffu, mbar_wait(&bars->full[(pv + sp) % C::NS], (uint32_t)(((pv + sp) / C::NS) & 1),
                                           &bars->abort_flag, err)))
      return false;
  if (dead) {
#pragma unroll 1
    for (int ch = 0; ch < C::NCH; ++ch) {
      const uint32_t at = row + ((pv + ch / C::SLOT_CH) % C::NS) * C::SLOT_BYTES + (ch % C::SLOT_CH) * C::CHUNK_BYTES;
#pragma unroll
      for (int i = 0; i < 8; ++i) st_shared_v4(at + 16 * ((i + threadIdx.x) & 7), 0u, 0u, 0u, 0u);
    }
  }
  fence_proxy_async_smem();
  return true;
}

// WIN_SPLIT: the join over the cluster's N CTAs of the query tile `w`.  Every
// CTA takes a share of the (row, 4 columns) items; first each row's weight of
// each run.
template <typename C, int N>
__device__ __forceinline__ void cluster_join(uint8_t* smem, const WinUnit& w, const WinParams& prm) {
  constexpr int D = C::D_;
  const int rank = (int)blockIdx.x % N;
  const uint32_t ml_at = smem_u32(smem + C::OFF_ML), o_at = smem_u32(smem + C::OFF_RING);
  float* weight = reinterpret_cast<float*>(smem + C::OFF_WEIGHT);  // [row][N], -1: the row sees no key of the run
  for (int row = threadIdx.x; row < w.ntok; row += C::THREADS) {
    float2 v[N];
    float m_all = -INFINITY, l_all = 0.0f;
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = ld_cluster_f2(cluster_addr(ml_at + row * 8, q));
#pragma unroll
    for (int q = 0; q < N; ++q) m_all = fmaxf(m_all, v[q].x);
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const float f = v[q].x == -INFINITY ? 1.0f : ex2(v[q].x - m_all);  // (-inf and a sum: NaN scores)
      l_all = fmaf(f, v[q].y, l_all);
      v[q].y = v[q].x == -INFINITY && v[q].y == 0.0f ? -1.0f : f;
    }
    const float inv = l_all == 0.0f ? 0.0f : 1.0f / l_all;
#pragma unroll
    for (int q = 0; q < N; ++q) weight[row * N + q] = v[q].y < 0.0f ? -1.0f : v[q].y * inv;
    if (rank == 0)
      prm.lse[(size_t)w.qz * prm.N + w.q_row + row] = (m_all + lg2(l_all)) * 0.69314718055994530942f;
  }
  __syncthreads();
  for (int i = rank * C::THREADS + threadIdx.x; i < w.ntok * (D / 4); i += N * C::THREADS) {
    const int row = i / (D / 4), c = i % (D / 4);
    float4 b[N], a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int q = 0; q < N; ++q)
      b[q] = ld_cluster_f4(cluster_addr(o_at + row * (D * 4) + (((c & ~7) + ((c & 7) ^ (row & 7))) << 4), q));
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const float f = weight[row * N + q];
      if (f < 0.0f) continue;
      a.x = fmaf(f, b[q].x, a.x);
      a.y = fmaf(f, b[q].y, a.y);
      a.z = fmaf(f, b[q].z, a.z);
      a.w = fmaf(f, b[q].w, a.w);
    }
    const uint2 pk = C::ELEM_ == kFP16 ? make_uint2(pack_f16x2(a.x, a.y), pack_f16x2(a.z, a.w))
                                       : make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(prm.o) +
                              ((size_t)w.qz * prm.N + w.q_row + row) * D + 4 * c) = pk;
  }
}

template <int ELEM, int D, bool PAGED, int FORM, bool TREE>
__global__ void __launch_bounds__(WinCfg<ELEM, D, PAGED, FORM>::THREADS, WinCfg<ELEM, D, PAGED, FORM>::OCC)
    attn_window_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                       const WinParams prm) {
  using C = WinCfg<ELEM, D, PAGED, FORM>;
  using Bars = WinBars<C::NS>;
  using TreeRow = WinTreeRow<TREE>;
  constexpr uint32_t END = end_places<C::NQT, TREE>();  // of a unit's places, those behind its tiles'
  static_assert(sizeof(Bars) <= 1024, "barrier area");
  static_assert(!TREE || PAGED, "trees lie in a paged cache");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  volatile int* abort_flag = &bars->abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = PAGED ? prm.g : 1;
  const int tpt = PAGED ? prm.tpt : kBM;   // tokens per query tile
  const int rpt = tpt * g;                 // rows per query tile
  const int tpg = C::NQT * tpt;            // tokens per unit

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t][0], 128);
      mbar_init(&bars->p_full[t][1], 128);
      mbar_init(&bars->o_ready[t], 1);
      mbar_init(&bars->o_full[t], 1);
      mbar_init(&bars->unit_full[t], 1);
      mbar_init(&bars->unit_empty[t], C::UNIT_READERS);
    }
    mbar_init(&bars->drain, 1);
    mbar_init(&bars->clc_bar, 1);
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(&bars->tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }

  if (warp == C::LOAD_WARP && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }

  // launched while the kernel before it ends; nothing above touched global memory
  if constexpr (PAGED) pdl_wait();
  // paged: the lengths of this thread's first sequence
  int seq_a = 0, seq_e = 0, seq_n = 0;
  const int seq_share = PAGED ? (prm.B + C::THREADS - 1) / C::THREADS : 0;  // sequences per thread
  const int seq_b0 = PAGED ? min(prm.B, (int)threadIdx.x * seq_share) : 0;
  if (PAGED && seq_b0 < prm.B) {
    seq_a = prm.cu_q[seq_b0];
    seq_e = prm.cu_q[seq_b0 + 1];
    seq_n = prm.seq_k[seq_b0];
  }
  // paged: this CTA's run [line0, line0 + line_n) of the line of work.  The
  // host refuses batches whose line could pass 2^31 places.  Token ranges that
  // overlap, against the contract, can make it longer than that: the sums stop
  // one behind the most that others can have, and nothing of such a line is run.
  uint32_t line_per = 0, line0 = 0, line_n = 0;
  if constexpr (PAGED) {
    pdl_launch();  // the join can be launched; it waits for this kernel's end
    // rows of a query tile that no TMA box covers (128 % g != 0) are zeros
    if (!C::FEW && rpt < kBM) {
      for (int i = threadIdx.x; i < C::NQT * C::NCH * (kBM - rpt) * 8; i += C::THREADS) {
        const int c = i / ((kBM - rpt) * 8), x = i % ((kBM - rpt) * 8);
        *reinterpret_cast<uint4*>(smem + C::OFF_Q + c * C::CHUNK_BYTES + rpt * 128 + x * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
    }
    if (threadIdx.x == 0) prm.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    // each thread sums the places of a contiguous share of the sequences
    bool bad = false;
    const int b1 = min(prm.B, seq_b0 + seq_share);
    auto seq_of = [&](int b) -> WinSeq {
      if (b == seq_b0) return win_seq(prm, seq_a, seq_e, seq_n, &bad);
      return win_seq(prm, prm.cu_q[b], prm.cu_q[b + 1], prm.seq_k[b], &bad);
    };
    auto group_places = [&](const WinSeq& q, int i) -> uint32_t {
      return (win_places<C::NQT, TREE>(win_group_len<TREE>(prm, q, tpg, i), min(tpg, q.nq - i * tpg), tpt) + END) * (uint32_t)prm.Hkv;
    };
    auto add = [&](uint32_t a, uint32_t b) -> uint32_t { return min(a + b, prm.max_places + 1); };  // (both at most that)
    auto seq_places = [&](const WinSeq& q) -> uint32_t {
      uint32_t n = 0;
      for (int i = 0; i * tpg < q.nq && n <= prm.max_places; ++i) n = add(n, group_places(q, i));
      return n;
    };
    uint32_t mine = 0;
    for (int b = seq_b0; b < b1 && mine <= prm.max_places; ++b) mine = add(mine, seq_places(seq_of(b)));
    uint32_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl = add(incl, x);
    }
    if (lane == 31) bars->warp_sum[warp] = incl;
    __syncthreads();
    uint32_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < C::THREADS / 32; ++w) {
      const uint32_t x = bars->warp_sum[w];
      if (w < warp) before = add(before, x);
      total = add(total, x);
    }
    if (total > prm.max_places) {
      total = 0;
      bad = true;
    }
    line_per = max((total + gridDim.x - 1) / gridDim.x, 1u);
    if (C::NQT == 2) line_per = (line_per + 1) & ~1u;
    line0 = line_per * blockIdx.x;
    line_n = line0 >= total ? 0u : min(line_per, total - line0);
    uint32_t at = before + incl - mine;
    if (line_n > 0 && line0 >= at && line0 - at < mine) {
      // this thread's sequences hold the start of the run: find the unit
      WinSeq q = seq_of(seq_b0);
      int b = seq_b0;
      for (;;) {
        const uint32_t n = b1 - seq_b0 == 1 ? mine : seq_places(q);
        if (line0 - at < n || b + 1 >= b1) break;
        at += n;
        q = seq_of(++b);
      }
      int i = 0;
      while ((i + 1) * tpg < q.nq) {
        const uint32_t n = group_places(q, i);
        if (line0 - at < n) break;
        at += n;
        ++i;
      }
      bars->start_b = b;
      bars->start_tok0 = q.tok0;
      bars->start_nq = q.nq;
      bars->start_nk = q.nk;
      bars->start_group = i;
      bars->start_len = win_group_len<TREE>(prm, q, tpg, i);
      bars->start_off = line0 - at;
    }
    if (bad && blockIdx.x == 0) report_index(prm.err);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // The two load warps' common parts.  Page numbers of list index l: lane i
  // holds that of box i (-1: no visible key, or out of range: reads as zeros).
  auto pages_of = [&](const WinUnit& w, int l) -> int {
    int id = -1;
    const int box_shift = prm.page_shift < 7 ? prm.page_shift : 7;  // rows of a box: a page's, at most a tile's
    if (PAGED && lane < (kBN >> box_shift) && l < w.r1) {
      const int box_rows = 1 << box_shift;
      const int tile = l < w.ns ? l : l + w.skip;
      const int key = tile * kBN + lane * box_rows;
      if (key < w.nk && (key < prm.sinks || key + box_rows > w.lo)) {
        id = prm.table[(long long)w.seq * prm.table_stride + (key >> prm.page_shift)];
        if ((unsigned)id >= (unsigned)prm.num_pages) {
          report_index(prm.err);
          id = -1;
        }
      }
    }
    return id;
  };
  // One K or V tile into the ring from position pos on (SPT slots).
  auto load_tile = [&](const WinUnit& w, const CUtensorMap* map, int pos, int l, int ids, uint64_t policy) -> bool {
    const int key0 = (l < w.ns ? l : l + w.skip) * kBN;
    for (int sp = 0; sp < C::SPT; ++sp, ++pos) {
      const int slot = pos % C::NS;
      const uint32_t ph = (uint32_t)((pos / C::NS) & 1);
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->empty[slot], ph ^ 1u, abort_flag, prm.err))) return false;
      // failure-injection hook (tests only): this slot is never filled, so
      // the MMA warp's wait on it runs out and the kernel aborts
      if (pos == prm.drop_pos && blockIdx.x == 0) continue;
      uint8_t* dst = smem + C::OFF_RING + slot * C::SLOT_BYTES;
      if (lane == 0) mbar_arrive_expect_tx(&bars->full[slot], C::SLOT_BYTES);
      __syncwarp();
      if constexpr (PAGED) {
        // one box per lane
        const int box_shift = prm.page_shift < 7 ? prm.page_shift : 7;
        const int box = lane & ((kBN >> box_shift) - 1), ch = lane >> (7 - box_shift);
        const int id = __shfl_sync(0xffffffffu, ids, box);
        const int row = box << box_shift;
        if (ch < C::SLOT_CH)
          tma_load_4d_hint(dst + ch * C::CHUNK_BYTES + row * 128, map, &bars->full[slot],
                           (sp * C::SLOT_CH + ch) * C::CH_ELEMS, (key0 + row) & ((1 << prm.page_shift) - 1), w.kz, id,
                           policy);
      } else if (lane < C::SLOT_CH) {
        tma_load_3d_hint(dst + lane * C::CHUNK_BYTES, map, &bars->full[slot], (sp * C::SLOT_CH + lane) * C::CH_ELEMS,
                         key0, w.kz, policy);
      }
    }
    return true;
  };
  // Ring positions within a unit of n tiles, in the order in which the MMA
  // warp consumes them: K0 V0 K1 V1 ..., or (S double-buffered) K0 K1 V0 K2 V1 ...
  auto k_at = [&](int j) -> int { return (C::ALT ? 2 * j : (j < 2 ? j : 2 * j - 1)) * C::SPT; };
  auto v_at = [&](int j, int n) -> int { return (C::ALT ? 2 * j + 1 : j + min(j + 2, n)) * C::SPT; };
  // Never leave with copies in flight: the last fills of the slots used (pos
  // positions so far).  After a wait ran out some of them were never issued;
  // those that were land within microseconds.
  auto settle_ring = [&](int pos) {
    const int used = pos < C::NS ? pos : C::NS;
    for (int i = 0; i < used; ++i) {
      const int p_last = pos - 1 - i;
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(&bars->full[p_last % C::NS], (uint32_t)((p_last / C::NS) & 1)) &&
             globaltimer() - t0 < (*abort_flag ? 2000000ull : FA_WAIT_LIMIT_NS)) {
      }
    }
  };

  if (warp >= C::SOFTMAX_WARPS) {
    if constexpr (C::REALLOC) regs_dec<C::CTRL_REGS>();
    // How long a unit's keys and values stay in L2.  Trees bring few units to a sequence
    // as a rule: up to four, its keys and values leave L2 first, for the partial results
    // that the join reads back (32 x 60 nodes over 1000 to 8000 keys 141 -> 138 us, 26 over
    // 131000 44 -> 41).  A longer chunk's stay, read by many units (2 x 1500 tokens over
    // 30000 keys beside 60 single ones 1150, and 1240 where they leave), and those that
    // other rows hold as well, as rows do that fa_pages_fork made (4 x 8 rows over 8000
    // shared keys each, d = 128: one token a row 124 and 146, 16 nodes 131 and 139, 60
    // nodes of 32 rows over 16000 370 and 419; at d = 64 16 nodes 95 and 91).  Looked at
    // are the rows before and behind, at the page where the unit begins: lane 1's row and
    // lane 2's, and the others ask for its own.
    auto near_row = [&](const WinUnit& w) -> int { return min(max(w.seq + (lane == 1) - (lane == 2), 0), prm.B - 1); };
    auto near_page = [&](const WinUnit& w) -> int {
      if (!TREE) return 0;
      const int key = (w.r0 < w.ns ? w.r0 : w.r0 + w.skip) * kBN;
      return prm.table[near_row(w) * prm.table_stride + (key >> prm.page_shift)];
    };
    const uint64_t pol_last = policy_evict_last(), pol_first = policy_evict_first();
    auto kv_policy = [&](const WinUnit& w, int near) -> uint64_t {
      if (!TREE) return pol_last;
      const int own = __shfl_sync(0xffffffffu, near, 0);
      const bool shared = __any_sync(0xffffffffu, near == own && near_row(w) != w.seq);
      return shared || w.nk - w.p0 + w.q_row > 4 * tpg ? pol_last : pol_first;
    };
    if (C::V_WARP && warp == C::LOADV_WARP) {
      // -------------------------------------------------------- load V --
      int pos = 0;
      bool ok = true;
      for (int r = 0; ok; ++r) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->unit_full[r & 1], (uint32_t)((r >> 1) & 1), abort_flag, prm.err));
        if (!ok) break;
        const WinUnit w = bars->unit[r & 1];
        __syncwarp();  // every lane has read the slot before one of them releases it
        if (lane == 0) mbar_arrive(&bars->unit_empty[r & 1]);
        if (w.kz < 0) break;
        const int n = w.r1 - w.r0;
        if (n <= 0) continue;
        const int near = near_page(w);
        int ids = pages_of(w, w.r0), ids1 = pages_of(w, w.r0 + 1);
        const uint64_t pol_kv = kv_policy(w, near);
        for (int j = 0; j < n && ok; ++j) {
          const int ids2 = pages_of(w, w.r0 + j + 2);  // two tiles ahead: its latency hides behind the loads
          ok = load_tile(w, &tm_v, pos + v_at(j, n), w.r0 + j, ids, pol_kv);
          ids = ids1;
          ids1 = ids2;
        }
        pos += 2 * n * C::SPT;
      }
      settle_ring(pos);
      __syncwarp();
    } else if (warp == C::LOAD_WARP) {
      // ---------------------------------------------------------- load --
      // The whole warp runs the loop; lane 0 waits, arms barriers and
      // publishes units; paged boxes are issued one per lane.
      const uint64_t pol_q = pol_first;
      int pos = 0;    // ring position (continues across units)
      int k = 0;      // units with keys loaded by this CTA
      bool ok = true;
      // publish unit r (w.kz < 0: no more units)
      auto publish = [&](int r, const WinUnit& w) -> bool {
        bool good = true;
        if (lane == 0) {
          const int slot = r & 1;
          if (r >= 2) good = mbar_wait(&bars->unit_empty[slot], (uint32_t)(((r - 2) >> 1) & 1), abort_flag, prm.err);
          if (good) {
            bars->unit[slot] = w;
            mbar_arrive(&bars->unit_full[slot]);
          }
        }
        return __shfl_sync(0xffffffffu, (int)good, 0) != 0;
      };
      // Q tiles and every key tile of a unit (and, without a V warp, every value tile)
      auto load_unit = [&](const WinUnit& w) {
        const int n = w.r1 - w.r0;
        if (n <= 0) return;  // no visible key: nothing to load
        const int near = near_page(w);
        int ids = pages_of(w, w.r0), ids1 = pages_of(w, w.r0 + 1);
        const int n0 = win_count(w, 0), n1 = C::NQT == 2 ? win_count(w, 1) : 0;
        // the Q buffer is free once the previous unit's last Q K^T finished
        if (k > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_empty, (uint32_t)((k - 1) & 1), abort_flag, prm.err));
        if (!ok) return;
        if (C::FEW) {
          // the rows' four copies: lane = copy and column chunk
          if (lane == 0) mbar_arrive_expect_tx(&bars->q_full, (uint32_t)(4 * rpt * C::ROW_BYTES));
          __syncwarp();
          const int c = lane / C::NCH, ch = lane % C::NCH;
          if (c < 4)
            tma_load_3d_hint(smem + C::OFF_Q + ch * C::Q_CHUNK + c * 32 * 128, &tm_q, &bars->q_full,
                             ch * C::CH_ELEMS, w.kz * g, w.qz, pol_q);
        } else if (lane == 0) {
          const uint32_t tile = (uint32_t)(rpt * C::ROW_BYTES);
          mbar_arrive_expect_tx(&bars->q_full, (n0 > 0 ? tile : 0u) + (n1 > 0 ? tile : 0u));
          for (int t = 0; t < C::NQT; ++t) {
            if ((t == 0 ? n0 : n1) == 0) continue;
            for (int ch = 0; ch < C::NCH; ++ch) {
              uint8_t* dst = smem + C::OFF_Q + (t * C::NCH + ch) * C::CHUNK_BYTES;
              if constexpr (PAGED)
                tma_load_3d_hint(dst, &tm_q, &bars->q_full, ch * C::CH_ELEMS, w.kz * g, w.qz + t * tpt, pol_q);
              else
                tma_load_3d_hint(dst, &tm_q, &bars->q_full, ch * C::CH_ELEMS, w.q_row + t * kBM, w.qz, pol_q);
            }
          }
        }
        __syncwarp();
        const uint64_t pol_kv = kv_policy(w, near);
        for (int j = 0; j < n && ok; ++j) {
          const int ids2 = pages_of(w, w.r0 + j + 2);
          ok = load_tile(w, &tm_k, pos + k_at(j), w.r0 + j, ids, pol_kv);
          if (!C::V_WARP && ok) {
            // this warp issues V too, in ring order
            if (C::ALT) ok = load_tile(w, &tm_v, pos + v_at(j, n), w.r0 + j, ids, pol_kv);
            else if (j >= 1) ok = load_tile(w, &tm_v, pos + v_at(j - 1, n), w.r0 + j - 1, 0, pol_kv);
          }
          ids = ids1;
          ids1 = ids2;
        }
        if (!C::V_WARP && !C::ALT && ok) ok = load_tile(w, &tm_v, pos + v_at(n - 1, n), w.r0 + n - 1, 0, pol_kv);
        pos += 2 * n * C::SPT;
        ++k;
      };
      // Trees: the softmax warps' first look at their mask rows and positions
      // would be a trip to memory for each unit; this warp, which is ahead of them,
      // has the lines brought into the SM's cache (nothing waits for them here).
      auto warm_rows = [&](const WinUnit& w) {
        const char* rows = reinterpret_cast<const char*>(prm.mask + (long long)w.qz * prm.words);
        const int bytes = w.ntok * prm.words * 4;
        for (int i = lane * 128; i < bytes; i += 32 * 128) prefetch_l1(rows + i);
        if (prm.positions && prm.window < w.nk && lane * 32 < w.ntok) prefetch_l1(prm.positions + w.qz + lane * 32);
      };
      WinUnit w;
      auto take_tiles = [&](const WinTiles& u) {
        w.ns = u.ns;
        w.skip = u.skip;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          w.sa[t] = u.sa[t];
          w.la[t] = u.la[t];
          w.lb[t] = u.lb[t];
        }
        w.narrow = u.skip > 0 && u.ns == 1 && prm.sinks <= C::NARROW ? 1 : 0;
      };
      w.seq = 0;
      if constexpr (PAGED) {
        int r = 0;
        if (line_n > 0) {
          uint32_t rem = line_n, at = line0;
          int b = bars->start_b, i = bars->start_group, len = bars->start_len;
          WinSeq s = {bars->start_tok0, bars->start_nq, bars->start_nk};
          int ntok = min(tpg, s.nq - i * tpg);
          uint32_t places = win_places<C::NQT, TREE>(len, ntok, tpt) + END;
          int head = (int)(bars->start_off / places);
          uint32_t off = bars->start_off % places;
          bool bad = false;
          while (ok) {
            // [off, off + run) of the unit's places are this CTA's
            const uint32_t run = min(rem, places - off);
            const int per_tile = C::NQT == 2 && (TREE || ntok > tpt) ? 2 : 1;
            const bool begins = off == 0, ends = off + run >= places - END;
            const bool none = TREE && off >= places - END;  // of its tiles
            w.kz = head;
            w.seq = b;
            w.q_row = i * tpg;
            w.qz = s.tok0 + w.q_row;
            w.p0 = s.nk - s.nq + w.q_row;
            w.ntok = ntok;
            w.nk = s.nk;
            const int base = TREE && win_is_tree(prm, s.nq) ? s.nk - s.nq : w.p0;
            w.lo = max(0, base - prm.window + 1);
            const WinTiles u = TREE ? win_tiles(w.p0, w.ntok, tpt, C::NQT, prm.window, prm.sinks,
                                                win_is_tree(prm, s.nq) ? base : 0x7fffffff)
                                    : win_tiles(w.p0, w.ntok, tpt, C::NQT, prm.window, prm.sinks);
            take_tiles(u);
            w.r0 = min(u.len, (int)off / per_tile);
            w.r1 = ends ? u.len : min(u.len, (int)(off + run) / per_tile);
            w.part = begins && ends ? -1 : 2 * (int)blockIdx.x + (begins ? 1 : 0);
            if (begins && !ends && lane == 0) {
              // parts: up to the CTA that holds the last place of the unit's tiles
              const uint32_t last = min((at + places - END - 1) / line_per, gridDim.x - 1);
              prm.desc[blockIdx.x] = make_int4((int)(last - blockIdx.x) + 1, w.qz, head, w.ntok * g);
            }
            if (!none) {
              ok = publish(r++, w);
              if constexpr (TREE) warm_rows(w);
              if (ok) load_unit(w);
            }
            rem -= run;
            at += run;
            if (rem == 0) break;
            off = 0;
            if (++head == prm.Hkv) {
              head = 0;
              if (++i * tpg >= s.nq) {
                i = 0;
                do {
                  if (++b >= prm.B) break;
                  s = win_seq(prm, prm.cu_q[b], prm.cu_q[b + 1], prm.seq_k[b], &bad);
                } while (s.nq == 0);
                if (b >= prm.B) break;
              }
              len = win_group_len<TREE>(prm, s, tpg, i);
              ntok = min(tpg, s.nq - i * tpg);
              places = win_places<C::NQT, TREE>(len, ntok, tpt) + END;
            }
          }
        }
        w.kz = -1;
        if (ok) publish(r, w);
      } else {
        // dense: one unit per launched CTA, heaviest first within chunks of
        // heads; a CTA about to finish takes over the next CTA that has not
        // started (cluster launch control), so its loads overlap the tail.
        // Units [0, pair_units) hold both query tiles of a group, the groups
        // behind them run as two units of one query tile each.
        const int n_groups = (prm.N + tpg - 1) / tpg;
        const int units = prm.pair_units + C::NQT * (prm.BH * n_groups - prm.pair_units);
        const int qgroup = prm.Hq / prm.Hkv;
        int n_req = 0;
        bool more = !C::SPLIT;
        auto decode = [&](int x) {
          const bool single = x >= prm.pair_units;
          const int v = single ? prm.pair_units + (x - prm.pair_units) / C::NQT : x;
          const int per_chunk = prm.head_chunk * n_groups;
          const int c = v / per_chunk;
          const int idx = v - c * per_chunk;
          const int heads_here = min(prm.head_chunk, prm.BH - c * prm.head_chunk);
          const int bh = c * prm.head_chunk + idx % heads_here;
          w.q_row = (n_groups - 1 - idx / heads_here) * tpg + (single ? (x - prm.pair_units) % C::NQT * kBM : 0);
          w.qz = bh;
          w.kz = (bh / prm.Hq) * prm.Hkv + (bh % prm.Hq) / qgroup;
          w.p0 = w.q_row + prm.Nk - prm.N;
          w.ntok = max(0, min(single ? kBM : tpg, prm.N - w.q_row));  // (0: a group's missing second tile)
          w.nk = prm.Nk;
          w.lo = max(0, w.p0 - prm.window + 1);
          const WinTiles u = win_tiles(w.p0, w.ntok, tpt, C::NQT, prm.window, prm.sinks);
          take_tiles(u);
          w.r0 = 0;
          w.r1 = w.ntok > 0 ? u.len : 0;
          w.part = -1;
        };
        if constexpr (C::SPLIT) {
          // this CTA's run of the cluster's unit
          const int n_cta = cluster_size(), rank = (int)blockIdx.x % n_cta;
          decode((int)blockIdx.x / n_cta);
          const int len = w.r1;
          w.r0 = (int)((long long)len * rank / n_cta);
          w.r1 = (int)((long long)len * (rank + 1) / n_cta);
        } else {
          decode((int)blockIdx.x);
        }
        ok = publish(0, w);
        for (int r = 0; ok; ++r) {
          load_unit(w);
          if (!ok) break;
          int nu = -1;
          if (more) {
            if (lane == 0) {
              mbar_arrive_expect_tx(&bars->clc_bar, 16);
              clc_try_cancel(bars->clc_resp, &bars->clc_bar);
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->clc_bar, (uint32_t)(n_req & 1), abort_flag, prm.err));
            if (!ok) break;
            ++n_req;
            nu = clc_query_x(bars->clc_resp);
            if (nu < 0 || nu >= units) {
              nu = -1;
              more = false;
            }
            __syncwarp();  // the response is read by every lane before it is asked for again
          }
          if (nu >= 0) decode(nu);
          else w.kz = -1;
          if (!publish(r + 1, w)) ok = false;
          if (nu < 0) break;
        }
      }
      settle_ring(pos);
      if (k > 0) {
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(&bars->q_full, (uint32_t)((k - 1) & 1)) && globaltimer() - t0 < FA_WAIT_LIMIT_NS) {
        }
      }
      __syncwarp();
    } else if (warp == C::MMA_WARP) {
      // ----------------------------------------------------------- MMA --
      // warp-converged issue; elect.sync picks the issuing lane
      const uint32_t q_s = smem_u32(smem + C::OFF_Q);
      const uint32_t ring_s = smem_u32(smem + C::OFF_RING);
      int pos = 0;          // ring position of the next tile to consume
      int k = 0;            // units with keys processed
      int pc[2] = {0, 0};   // P handshakes consumed per query tile
      int it = 0;           // S double-buffered: S/P iterations so far (buffer = it & 1)
      bool ok = true;
      auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, prm.err));
      };
      auto wait_tile = [&](int p) -> bool {
        for (int sp = 0; sp < C::SPT; ++sp)
          if (!warp_wait(&bars->full[(p + sp) % C::NS], (uint32_t)(((p + sp) / C::NS) & 1))) return false;
        tc_fence_after();
        return true;
      };
      auto release_tile = [&](int p) {
        for (int sp = 0; sp < C::SPT; ++sp) mma_commit_elect(&bars->empty[(p + sp) % C::NS]);
      };
      const uint64_t q_desc0 = smem_desc(q_s, 16, 1024, 2);                      // Q tiles, K-major
      const uint64_t ring_k_desc0 = smem_desc(ring_s, 16, 1024, 2);              // K slots, K-major
      const uint64_t ring_v_desc0 = smem_desc(ring_s, C::CHUNK_BYTES, 1024, 2);  // V slots, MN-major
      auto slot_off = [&](int p) -> uint32_t { return (uint32_t)(p % C::NS) * C::SLOT_BYTES; };
      // S_buf = Q_t K^T for the K tile at ring position p
      auto issue_qk_of = [&](int t, int buf, int p, auto idesc) {
        const uint64_t a0 = q_desc0 + (uint64_t)((t * C::NCH * C::CHUNK_BYTES) >> 4);
        uint64_t b0[C::SPT];
#pragma unroll
        for (int sp = 0; sp < C::SPT; ++sp) b0[sp] = ring_k_desc0 + (uint64_t)(slot_off(p + sp) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int ch = ks / 4, in_ch = (ks % 4) * 32;
          const uint64_t a = a0 + (uint64_t)((ch * C::Q_CHUNK + in_ch) >> 4);
          const uint64_t b = b0[ch / C::SLOT_CH] + (uint64_t)(((ch % C::SLOT_CH) * C::CHUNK_BYTES + in_ch) >> 4);
          mma_ss_elect<0>(tmem + buf * kBN, a, b, decltype(idesc)::value, ks > 0 ? 1u : 0u);
        }
      };
      auto issue_qk = [&](int t, int buf, int p) { issue_qk_of(t, buf, p, std::integral_constant<uint32_t, C::IDESC_QK>()); };
      // a narrow tile: S for its first keys, and their P V (all in half 0)
      auto issue_qk_narrow = [&](int t, int buf, int p) {
        issue_qk_of(t, buf, p, std::integral_constant<uint32_t, C::IDESC_QK_NARROW>());
      };
      auto issue_pv_narrow = [&](int t, int buf, int p) {
#pragma unroll
        for (int sp = 0; sp < C::SPT; ++sp)
#pragma unroll
          for (int ks = 0; ks < C::NARROW / 16; ++ks)
            mma_ts_elect<0>(tmem + C::O_COL0 + t * D + sp * C::SLOT_D, tmem + buf * kBN + ks * 8,
                            ring_v_desc0 + (uint64_t)((slot_off(p + sp) + ks * 2048) >> 4), C::IDESC_PV, ks > 0 ? 1u : 0u);
      };
      // O_t (+)= P_buf V for half h of the keys of the V tile at ring position p
      auto issue_pv = [&](int t, int buf, int p, bool acc, int h) {
#pragma unroll
        for (int sp = 0; sp < C::SPT; ++sp) {
          const uint32_t d_tmem = tmem + C::O_COL0 + t * D + sp * C::SLOT_D;
          const uint64_t v0 = ring_v_desc0 + (uint64_t)(slot_off(p + sp) >> 4);
#pragma unroll
          for (int ks = h * 4; ks < h * 4 + 4; ++ks)
            mma_ts_elect<0>(d_tmem, tmem + buf * kBN + ks * 8, v0 + (uint64_t)((ks * 2048) >> 4), C::IDESC_PV,
                            (acc || ks > 0) ? 1u : 0u);
        }
      };
      for (int r = 0; ok; ++r) {
        ok = warp_wait(&bars->unit_full[r & 1], (uint32_t)((r >> 1) & 1));
        if (!ok) break;
        const WinUnit w = bars->unit[r & 1];
        __syncwarp();  // every lane has read the slot before one of them releases it
        if (lane == 0) mbar_arrive(&bars->unit_empty[r & 1]);
        if (w.kz < 0) break;
        if (w.r1 <= w.r0) continue;
        ok = warp_wait(&bars->q_full, (uint32_t)(k & 1));
        if (!ok) break;
        tc_fence_after();
        const int n0 = win_count(w, 0), n1 = C::NQT == 2 ? win_count(w, 1) : 0;
        int qk_left = n0 + n1;
        auto qk_issued = [&]() {
          if (--qk_left == 0) mma_commit_elect(&bars->q_empty);  // the unit's Q has been read
        };
        if constexpr (C::ALT) {
          // per query tile: P V still to issue, and the next list index
          const WinPart part[2] = {WinPart(w, 0), WinPart(w, 1)};
          int left[2] = {n0, n1};
          int next[2] = {part[0].from(w.r0), part[1].from(w.r0)};
          bool begun[2] = {false, false};
          ok = wait_tile(pos);
          if (!ok) break;
          int l0 = w.r0;
          if (w.narrow && l0 == 0) {
            // both query tiles' narrow tile first; it is every valid tile's first
#pragma unroll
            for (int t = 0; t < 2; ++t)
              if (left[t] > 0 && next[t] == 0) {
                issue_qk_narrow(t, t, pos);
                mma_commit_elect(&bars->s_full[t]);
                qk_issued();
              }
            release_tile(pos);
            pos += C::SPT;
            const int v_pos = pos, k_pos = pos + C::SPT;
            ok = wait_tile(v_pos) && (w.r1 == 1 || wait_tile(k_pos));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok) break;
              if (left[t] > 0 && next[t] == 0) {
                ok = warp_wait(&bars->p_full[t][0], (uint32_t)(pc[t] & 1)) && warp_wait(&bars->p_full[t][1], (uint32_t)(pc[t] & 1));
                if (!ok) break;
                tc_fence_after();
                issue_pv_narrow(t, t, v_pos);
                ++pc[t];
                begun[t] = true;
                next[t] = part[t].from(1);
                if (--left[t] == 0) mma_commit_elect(&bars->o_full[t]);
              }
              if (left[t] > 0 && next[t] == 1) {
                issue_qk(t, t, k_pos);
                mma_commit_elect(&bars->s_full[t]);
                qk_issued();
              }
            }
            if (!ok) break;
            release_tile(v_pos);
            pos += C::SPT;
            l0 = 1;
            if (l0 >= w.r1) {
              ++k;
              continue;
            }
          } else {
#pragma unroll
            for (int t = 0; t < 2; ++t)
              if (left[t] > 0 && next[t] == l0) {
                issue_qk(t, t, pos);
                mma_commit_elect(&bars->s_full[t]);
                qk_issued();
              }
          }
          release_tile(pos);
          pos += C::SPT;
          for (int l = l0; l < w.r1 && ok; ++l) {
            const int pv_pos = pos, k_pos = pos + C::SPT;  // V_l, K_{l+1}
            bool v_ready = false, k_ready = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok) break;
              if (left[t] > 0 && next[t] == l) {
                if (!v_ready) {
                  ok = wait_tile(pv_pos);
                  v_ready = true;
                  if (!ok) break;
                }
#pragma unroll
                for (int h = 0; h < 2 && ok; ++h) {
                  ok = warp_wait(&bars->p_full[t][h], (uint32_t)(pc[t] & 1));
                  if (!ok) break;
                  tc_fence_after();
                  issue_pv(t, t, pv_pos, begun[t], h);
                }
                if (!ok) break;
                ++pc[t];
                begun[t] = true;
                next[t] = part[t].from(l + 1);
                if (--left[t] == 0) mma_commit_elect(&bars->o_full[t]);
              }
              if (left[t] > 0 && next[t] == l + 1) {
                if (!k_ready) {
                  ok = wait_tile(k_pos);
                  k_ready = true;
                  if (!ok) break;
                }
                issue_qk(t, t, k_pos);
                mma_commit_elect(&bars->s_full[t]);
                qk_issued();
              }
            }
            if (!ok) break;
            // (every list index has a query tile that takes part in it)
            release_tile(pv_pos);
            pos += C::SPT;
            if (l + 1 < w.r1) {
              release_tile(k_pos);
              pos += C::SPT;
            }
          }
        } else {
          // one query tile, S double-buffered: S(0), S(1), then PV(j), S(j+2)
          const int n = w.r1 - w.r0;
          const bool narrow = w.narrow && w.r0 == 0;
          for (int j = 0; j < 2 && j < n && ok; ++j) {
            ok = wait_tile(pos);
            if (!ok) break;
            if (j == 0 && narrow) issue_qk_narrow(0, it & 1, pos);
            else issue_qk(0, (it + j) & 1, pos);
            mma_commit_elect(&bars->s_full[(it + j) & 1]);
            qk_issued();
            release_tile(pos);
            pos += C::SPT;
          }
          for (int j = 0; j < n && ok; ++j) {
            const int x = it + j, b = x & 1;
            ok = wait_tile(pos);  // V_j
            if (!ok) break;
            if (j == 0 && narrow) {
              ok = warp_wait(&bars->p_full[b][0], (uint32_t)((x >> 1) & 1)) && warp_wait(&bars->p_full[b][1], (uint32_t)((x >> 1) & 1));
              if (!ok) break;
              tc_fence_after();
              issue_pv_narrow(0, b, pos);
            } else {
#pragma unroll
              for (int h = 0; h < 2 && ok; ++h) {
                ok = warp_wait(&bars->p_full[b][h], (uint32_t)((x >> 1) & 1));
                if (!ok) break;
                tc_fence_after();
                issue_pv(0, b, pos, j > 0, h);
              }
            }
            if (!ok) break;
            mma_commit_elect(&bars->o_ready[b]);
            release_tile(pos);
            pos += C::SPT;
            if (j + 2 < n) {
              ok = wait_tile(pos);  // K_{j+2}
              if (!ok) break;
              issue_qk(0, b, pos);
              mma_commit_elect(&bars->s_full[b]);
              qk_issued();
              release_tile(pos);
              pos += C::SPT;
            }
          }
          if (ok) mma_commit_elect(&bars->o_full[0]);
          it += n;
        }
        ++k;
      }
      // every MMA issued here has completed before TMEM is freed
      mma_commit_elect(&bars->drain);
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(&bars->drain, 0) && globaltimer() - t0 < FA_WAIT_LIMIT_NS) {
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------- softmax --
    if constexpr (C::REALLOC) regs_inc<C::SOFTMAX_REGS>();
    const int t = warp / 4;                  // query tile of this warp
    const int wq = warp % 4;                 // TMEM lane quarter
    const int r_in = wq * 32 + lane;         // row within the tile, and key row of a V tile
    const uint32_t lane_addr = (uint32_t)(wq * 32) << 16;
    const int tok_in = PAGED ? r_in / g : r_in;  // token within the tile
    const int head_in = r_in - tok_in * g;
    const int row_tok = C::FEW ? lane / g : tok_in;  // WIN_FEW: rows are lanes
    const bool neg = prm.scale_log2 < 0.0f;
    const float mask_val = neg ? INFINITY : -INFINITY;
    const float cj = prm.scale_log2;
    int sc = 0;        // S handshakes consumed
    int it = 0;        // S double-buffered: iterations so far
    int oc = 0;        // o_full phases consumed
    int pv_seen = 0;   // S double-buffered: P V completions consumed
    int ring = 0;      // ring position of the unit's first tile
    bool ok = true;
    bool left = false;  // WIN_FEW: the warps found together that one of them gave up

    for (int rr = 0; ok; ++rr) {
      // The unit is read where it stands in the queue, and its slot released
      // at the unit's end: what only the epilogue needs does not weigh on the
      // key-tile loop's registers.
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->unit_full[rr & 1], (uint32_t)((rr >> 1) & 1), abort_flag, prm.err));
      if (!ok) break;
      const WinUnit& w = bars->unit[rr & 1];
      if (w.kz < 0) break;
      const int r0 = w.r0, r1 = w.r1;
      const int nrun = r1 > r0 ? r1 - r0 : 0;
      const int ring0 = ring;
      ring += 2 * nrun * C::SPT;
      const int rows = min(rpt, (w.ntok - t * tpt) * g);  // valid rows of this tile
      const bool valid = r_in < rows;
      const int tok = t * tpt + tok_in;                      // token within the unit
      // where this row's results go
      auto out_row_of = [&]() -> size_t {
        if (w.part >= 0) return (size_t)w.part * (C::NQT * kBM) + t * rpt + r_in;
        if (PAGED) return (size_t)(w.qz + tok) * prm.Hq + w.kz * g + head_in;
        return (size_t)w.qz * prm.N + w.q_row + tok;
      };
      do {  // one unit (skipped when this tile has no valid row)
        if (rows <= 0) break;
        const WinPart mine(w, t);
        const int n = C::NQT == 2 ? mine.count(r0, r1) : nrun;
        if (C::SPLIT && n == 0) {
          reinterpret_cast<float2*>(smem + C::OFF_ML)[r_in] = make_float2(-INFINITY, 0.0f);
          break;
        }
        if (n == 0) {
          // no row of this tile sees a key of this run: O = 0, LSE = -inf
          if (valid) {
            const size_t out_row = out_row_of();
            if (w.part >= 0) {
              float4* dst = reinterpret_cast<float4*>(prm.o_part + out_row * D);
#pragma unroll 1
              for (int i = 0; i < D / 4; ++i) dst[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              prm.lse_part[out_row] = -INFINITY;
            } else {
              uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(prm.o) + out_row * D * 2);
#pragma unroll 1
              for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
              prm.lse[out_row] = -INFINITY;
            }
          }
          break;
        }
        // this row's last visible key, its own position (a valid row's lies in
        // the sequence); the tile's strictest last and first (window) ones
        const int last = w.p0 + tok;
        // the last key that all of the tile's rows see (but for their windows): its
        // first row's, or where the rows are a tree's nodes the last cached one
        int tile_last = w.p0 + t * tpt;
        if (TREE && win_is_tree(prm, w.nk - (w.p0 - w.q_row))) tile_last = w.p0 - w.q_row - 1;
        const int tile_lo = w.p0 + min(w.ntok, (t + 1) * tpt) - prm.window;    // of its last row
        float m_run = -INFINITY;  // reference maximum, log2 units
        float l_run = 0.0f;
        // S double-buffered: consume o_ready completions up to the P V of
        // iteration x (they complete in order)
        auto consume_o = [&](int x) -> bool {
          while (pv_seen <= x) {
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->o_ready[pv_seen & 1], (uint32_t)((pv_seen >> 1) & 1),
                                                   abort_flag, prm.err)))
              return false;
            ++pv_seen;
          }
          return true;
        };
        if constexpr (C::FEW) {
          // lane = row, this warp's columns 32 wq .. 32 wq + 31
          const int nr = w.ntok * g;
          const int lo = w.p0 + w.ntok - prm.window;  // first key of the last row's window
          const TreeRow node(prm, w, row_tok, lane < nr);
          const int masked_from = TREE && tile_last < w.p0 ? tile_last + 1 : w.p0 + 1;  // keys that not every row sees
          for (int j = 0; j < n && ok; ++j) {
            const int x = it + j, l = r0 + j;
            const int buf = C::ALT ? 0 : (x & 1);
            uint32_t seen = 0;  // TREE: asked for ahead of the scores
            if constexpr (TREE) {
              const int c0 = (l < w.ns ? l : l + w.skip) * kBN + 32 * wq;
              if (c0 + 32 > masked_from || (c0 < lo && c0 + 32 > prm.sinks)) seen = node.see(prm, c0);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[buf], (uint32_t)((C::ALT ? sc : x >> 1) & 1),
                                                   abort_flag, prm.err));
            ++sc;
            if (!ok) break;
            tc_fence_after();
            if (!C::ALT && x >= 2 && !consume_o(x - 2)) {
              ok = false;
              break;
            }
            const uint32_t s_addr = tmem + lane_addr + buf * kBN;
            const int col0 = (l < w.ns ? l : l + w.skip) * kBN;
            const bool narrow = w.narrow && l == 0;
            // rows of the V tile that no query of the unit sees become zeros, as below
            const bool gap = w.lo > prm.sinks && col0 < w.lo && col0 + kBN > prm.sinks;
            if (col0 + kBN > w.nk || gap) {
              if (!C::ALT && j > 0 && !consume_o(x - 1)) {
                ok = false;
                break;
              }
              const int key = col0 + r_in;
              const bool dead = key >= w.nk || (key < w.lo && key >= prm.sinks);
              ok = clear_v_row<C, Bars>(bars, smem_u32(smem + C::OFF_RING) + r_in * 128, ring0 + v_at(j, n), dead, prm.err);
              if (!ok) break;
            }
            uint32_t pk[16], zero[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = zero[i] = 0u;
            if (!narrow || wq == 0) {
              uint32_t u[32];
              tmem_ld32(s_addr + 32 * wq, u);
              tmem_wait_ld();
              const int c0 = col0 + 32 * wq;
              if (c0 + 32 > masked_from || (c0 < lo && c0 + 32 > prm.sinks)) {
                const uint32_t see = TREE ? seen : win_visible(w.p0 + row_tok, prm.window, prm.sinks, c0);
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = (see & (1u << i)) ? u[i] : __float_as_uint(mask_val);
              }
              float r4[4];
              if (!neg) {
#pragma unroll
                for (int i = 0; i < 4; ++i) r4[i] = fmaxf(__uint_as_float(u[i]), __uint_as_float(u[4 + i]));
#pragma unroll
                for (int c = 8; c < 32; c += 8)
#pragma unroll
                  for (int i = 0; i < 4; ++i) r4[i] = max3f(r4[i], __uint_as_float(u[c + i]), __uint_as_float(u[c + 4 + i]));
                r4[0] = fmaxf(max3f(r4[0], r4[1], r4[2]), r4[3]);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) r4[i] = fminf(__uint_as_float(u[i]), __uint_as_float(u[4 + i]));
#pragma unroll
                for (int c = 8; c < 32; c += 8)
#pragma unroll
                  for (int i = 0; i < 4; ++i) r4[i] = min3f(r4[i], __uint_as_float(u[c + i]), __uint_as_float(u[c + 4 + i]));
                r4[0] = fminf(min3f(r4[0], r4[1], r4[2]), r4[3]);
              }
              // (lanes without a row never move their maximum)
              const float mx2 = lane < nr ? r4[0] * cj : -INFINITY;
              float alpha = 1.0f;
              const bool move = (mx2 > m_run + C::TAU) || (m_run == -INFINITY && mx2 != -INFINITY);
              if (move) {
                alpha = ex2(m_run - mx2);  // 0 on the row's first visible columns
                m_run = mx2;
              }
              l_run *= alpha;
              if (j > 0 && __any_sync(0xffffffffu, move)) {
                if constexpr (!C::ALT) {
                  // O holds P V(x-1): wait for it
                  if (!consume_o(x - 1)) {
                    ok = false;
                    break;
                  }
                  tc_fence_after();
                }
                rescale_o_cols<D>(tmem + lane_addr + C::O_COL0, alpha);
              }
              const float nm = m_run == -INFINITY ? 0.0f : -m_run;
              float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 e = fma2(make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])),
                                      make_float2(cj, cj), make_float2(nm, nm));
                const float2 q = make_float2(ex2(e.x), ex2(e.y));
                acc[i & 1] = add2(acc[i & 1], q);
                pk[i] = (ELEM == kBF16) ? pack_bf16x2(q.x, q.y) : pack_f16x2(q.x, q.y);
              }
              const float2 tt = add2(acc[0], acc[1]);
              l_run += tt.x + tt.y;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (narrow && q > 0) break;  // (its first 32 keys alone are multiplied)
              if (q == wq) tmem_st16(s_addr + 16 * q, pk);
              else tmem_st16(s_addr + 16 * q, zero);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars->p_full[buf][0]);
            mbar_arrive(&bars->p_full[buf][1]);
          }
          // The copies' join.  O goes through query rows that no copy uses, 16
          // of each warp's 32: a line of 32 columns per row and column chunk, its
          // 16-byte pieces permuted by the row; all columns at once where they fit
          // (up to 8 rows of two lines each), else by halves.
          if (ok) {
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_full[0], (uint32_t)(oc & 1), abort_flag, prm.err));
            ++oc;
          }
          float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
          uint8_t* stage = smem + C::OFF_Q + 16 * 128;
          const bool once = !C::Q_PACKED && nr <= C::FEW_ROWS / 2;
          auto put = [&](int h) {
#pragma unroll
            for (int ch = 0; ch < C::NCH; ++ch) {
              uint32_t u[32];
              tmem_ld32(tmem + lane_addr + C::O_COL0 + h * (D / 2) + ch * 32, u);
              tmem_wait_ld();
              if (lane < nr) {
                const int at = once ? lane + h * (C::FEW_ROWS / 2) : lane;
                uint4* line = reinterpret_cast<uint4*>(stage + ch * C::Q_CHUNK + (wq * 32 + at) * 128);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  line[i ^ (at & 7)] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
              }
            }
          };
          if (ok) {
            tc_fence_after();
            if (lane < nr) ml[lane * 4 + wq] = make_float2(m_run, l_run);
            put(0);
            if (once) put(1);
            // this warp's reads of O (with more rows: of half of it; the others
            // come before the last barrier) are ordered before the next unit's S
            tc_fence_before();
          }
          // (a warp that gave up meets the others here or at its end, so no one waits for it)
          ok = bar_and(1, 128, ok);
          if (!ok) {
            left = true;
            break;
          }
          for (int h = 0; h < 2; ++h) {
            if (h == 1 && !once) {
              bar_sync_n(1, 128);
              put(1);
              tc_fence_before();
              bar_sync_n(1, 128);
            }
            for (int i = threadIdx.x; i < nr * (D / 8); i += 128) {
              const int row = i / (D / 8), c = i % (D / 8);  // 4 columns, from h * D / 2 + 4 c on
              float2 v[4];
              float m_all = -INFINITY, l_all = 0.0f;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                v[q] = ml[row * 4 + q];
                m_all = fmaxf(m_all, v[q].x);
              }
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                v[q].x = v[q].x == -INFINITY ? 0.0f : ex2(v[q].x - m_all);
                l_all = fmaf(v[q].x, v[q].y, l_all);
              }
              const float f = l_all > 0.0f ? 1.0f / l_all : 0.0f;
              const int at = once ? row + h * (C::FEW_ROWS / 2) : row;
              float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float4 b = reinterpret_cast<const float4*>(stage + (c / 8) * C::Q_CHUNK +
                                                                 (q * 32 + at) * 128)[(c % 8) ^ (at & 7)];
                a.x = fmaf(v[q].x, b.x, a.x);
                a.y = fmaf(v[q].x, b.y, a.y);
                a.z = fmaf(v[q].x, b.z, a.z);
                a.w = fmaf(v[q].x, b.w, a.w);
              }
              const size_t o_row = w.part >= 0 ? (size_t)w.part * kBM + row
                                               : (size_t)(w.qz + row / g) * prm.Hq + w.kz * g + row % g;
              const size_t o_at = o_row * D + h * (D / 2) + 4 * c;
              if (w.part >= 0) {
                *reinterpret_cast<float4*>(prm.o_part + o_at) = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
              } else {
                const uint2 pk = ELEM == kFP16 ? make_uint2(pack_f16x2(a.x * f, a.y * f), pack_f16x2(a.z * f, a.w * f))
                                               : make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
                *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(prm.o) + o_at) = pk;
              }
              if (h == 0 && c == 0)
                (w.part >= 0 ? prm.lse_part : prm.lse)[o_row] = (m_all + lg2(l_all)) * 0.69314718055994530942f;
            }
          }
          break;
        }
        if constexpr (PAGED && FORM == WIN_ONE && D == 64) {
          if (wq * 32 >= rows) {
            // None of this warp's rows exist: it keeps step with the others and
            // zeroes its rows of V tiles (see below), whatever P then holds, and
            // leaves its sub-partition to the other CTA (64 sequences of 8 tokens
            // over 500 to 3000 keys, 32/8 heads 73 -> 65 us; at d = 128, with one
            // CTA per SM, it gains nothing).
            for (int j = 0; j < n && ok; ++j, ++sc) {
              ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[0], (uint32_t)(sc & 1), abort_flag, prm.err));
              if (!ok) break;
              const int li = r0 + j, col0 = (li < w.ns ? li : li + w.skip) * kBN;
              const bool gap = w.lo > prm.sinks && col0 < w.lo && col0 + kBN > prm.sinks;
              if (col0 + kBN > w.nk || gap) {
                const int key = col0 + r_in;
                const bool dead = key >= w.nk || (key < w.lo && key >= prm.sinks);
                ok = clear_v_row<C, Bars>(bars, smem_u32(smem + C::OFF_RING) + r_in * 128, ring0 + v_at(j, n), dead, prm.err);
                if (!ok) break;
              }
              mbar_arrive(&bars->p_full[0][0]);
              mbar_arrive(&bars->p_full[0][1]);
            }
            if (!ok) break;
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_full[0], (uint32_t)(oc & 1), abort_flag, prm.err));
            ++oc;
            break;
          }
        }
        int l = C::NQT == 2 ? mine.from(r0) : r0;  // list index
        int j = 0;                                 // tiles done by this query tile
        if (w.narrow && l == 0) {
          const int buf = C::ALT ? t : (it & 1);
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[buf], (uint32_t)((C::ALT ? sc : it >> 1) & 1),
                                                 abort_flag, prm.err));
          ++sc;
          if (!ok) break;
          tc_fence_after();
          if (!C::ALT && it >= 2 && !consume_o(it - 2)) {
            ok = false;
            break;
          }
          if constexpr (PAGED) {
            // the keys behind the sinks have left the window (see below)
            ok = clear_v_row<C, Bars>(bars, smem_u32(smem + C::OFF_RING) + r_in * 128, ring0 + v_at(0, n),
                                      r_in >= prm.sinks, prm.err);
            if (!ok) break;
          }
          const float2 ml = narrow_softmax<ELEM>(tmem + lane_addr + buf * kBN,
                                                 TREE ? TreeRow(prm, w, tok, valid).see(prm, 0)
                                                      : win_visible(last, prm.window, prm.sinks, 0), cj);
          m_run = ml.x;
          l_run = ml.y;
          tc_fence_before();
          mbar_arrive(&bars->p_full[buf][0]);
          mbar_arrive(&bars->p_full[buf][1]);
          j = 1;
          l = C::NQT == 2 ? mine.from(1) : 1;
        }
        for (; j < n && ok; ++j, l = C::NQT == 2 ? mine.from(l + 1) : l + 1) {
          const int x = it + j;
          const int buf = C::ALT ? t : (x & 1);
          const uint32_t ph = C::ALT ? (uint32_t)(sc & 1) : (uint32_t)((x >> 1) & 1);
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[buf], ph, abort_flag, prm.err));
          ++sc;
          if (!ok) break;
          tc_fence_after();
          if constexpr (!C::ALT) {
            // P V(x-2) was issued before S(x): consume its o_ready phase to
            // keep at most one pending per buffer
            if (x >= 2 && !consume_o(x - 2)) {
              ok = false;
              break;
            }
          }
          const uint32_t s_addr = tmem + lane_addr + buf * kBN;
          const int col0 = (l < w.ns ? l : l + w.skip) * kBN;
          const bool need_mask = col0 + kBN - 1 > tile_last || (col0 < tile_lo && col0 + kBN > prm.sinks);
          if constexpr (PAGED) {
            // Rows of the V tile that no query of the unit may see can hold
            // anything; P = 0 there would still give NaN from a NaN, so they
            // become zeros before P is handed over (here, while few registers are
            // live).  Thread r clears key r; both query tiles do so (the writes
            // are the same), each before its own P V.
            const bool gap = w.lo > prm.sinks && col0 < w.lo && col0 + kBN > prm.sinks;
            if (col0 + kBN > w.nk || gap) {
              // (S double-buffered: the slot's previous fill may still be the V tile
              // before, so that one's P V is waited for first; else K of
              // this tile lies between)
              if (!C::ALT && j > 0 && !consume_o(x - 1)) {
                ok = false;
                break;
              }
              const int key = col0 + r_in;
              const bool dead = key >= w.nk || (key < w.lo && key >= prm.sinks);
              ok = clear_v_row<C, Bars>(bars, smem_u32(smem + C::OFF_RING) + r_in * 128, ring0 + v_at(C::NQT == 2 ? l - r0 : j, n),
                                        dead, prm.err);
              if (!ok) break;
            }
          }
          if constexpr (TREE) {
            if (need_mask) {
              const TreeRow node(prm, w, tok, valid);
              tree_mask_scores(s_addr, col0, node.row, prm.words, node.ctx, node.slot, node.pos, prm.window, prm.sinks, mask_val);
            }
          }
          float s[kBN];
          {
            uint32_t u[32];
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) {
              tmem_ld32(s_addr + c4 * 32, u);
#pragma unroll
              for (int i = 0; i < 32; ++i) s[c4 * 32 + i] = __uint_as_float(u[i]);
            }
            tmem_wait_ld();
          }
          if (!TREE && need_mask) {
            // visible columns of this row as four words
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t see = win_visible(last, prm.window, prm.sinks, col0 + 32 * q);
#pragma unroll
              for (int i = 0; i < 32; ++i) s[32 * q + i] = (see & (1u << i)) ? s[32 * q + i] : mask_val;
            }
          }
          // row maximum (minimum for a negative scale): eight chains of 3-input max
          float mx, r8[8];
          if (!neg) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r8[i] = fmaxf(s[i], s[8 + i]);
#pragma unroll
            for (int c = 16; c < kBN; c += 16)
#pragma unroll
              for (int i = 0; i < 8; ++i) r8[i] = max3f(r8[i], s[c + i], s[c + 8 + i]);
            mx = max3f(max3f(r8[0], r8[1], r8[2]), max3f(r8[3], r8[4], r8[5]), fmaxf(r8[6], r8[7]));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r8[i] = fminf(s[i], s[8 + i]);
#pragma unroll
            for (int c = 16; c < kBN; c += 16)
#pragma unroll
              for (int i = 0; i < 8; ++i) r8[i] = min3f(r8[i], s[c + i], s[c + 8 + i]);
            mx = min3f(min3f(r8[0], r8[1], r8[2]), min3f(r8[3], r8[4], r8[5]), fminf(r8[6], r8[7]));
          }
          const float mx2 = mx * cj;  // (a row that sees no key of this tile: -inf)
          float alpha = 1.0f;
          const bool move = (mx2 > m_run + C::TAU) || (m_run == -INFINITY && mx2 != -INFINITY);
          if (move) {
            alpha = ex2(m_run - mx2);  // 0 on the row's first visible tile
            m_run = mx2;
          }
          l_run *= alpha;
          if (j > 0 && __any_sync(0xffffffffu, move)) {
            if constexpr (!C::ALT) {
              // O holds P V(x-1): wait for it
              if (!consume_o(x - 1)) {
                ok = false;
                break;
              }
              tc_fence_after();
            }
            rescale_o_cols<D>(tmem + lane_addr + C::O_COL0 + t * D, alpha);
          }
          // P = 2^(s*cj - m); a masked score gives 2^-inf = 0 (a row without
          // a visible key yet takes 0 in place of -m)
          const float2 cj2 = make_float2(cj, cj);
          const float nm = m_run == -INFINITY ? 0.0f : -m_run;
          const float2 nm2 = make_float2(nm, nm);
          float2 acc[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q == 2) {
              // keys 0..63 of P are in TMEM: let their MMAs start
              tmem_wait_st();
              tc_fence_before();
              mbar_arrive(&bars->p_full[buf][0]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t u[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int c = q * 32 + h * 16 + 2 * i;
                const float2 e = fma2(make_float2(s[c], s[c + 1]), cj2, nm2);
                const float2 p = make_float2(ex2(e.x), ex2(e.y));
                acc[i & 3] = add2(acc[i & 3], p);
                u[i] = (ELEM == kBF16) ? pack_bf16x2(p.x, p.y) : pack_f16x2(p.x, p.y);
              }
              tmem_st8(s_addr + q * 16 + h * 8, u);
            }
          }
          const float2 tt = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
          l_run += tt.x + tt.y;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars->p_full[buf][1]);
        }

        // -------------------------------------------------------- epilogue --
        if (!ok) break;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_full[t], (uint32_t)(oc & 1), abort_flag, prm.err));
        ++oc;
        if (!ok) break;
        tc_fence_after();
        if constexpr (C::SPLIT) {
          // for the cluster's join: the row's maximum and sum, and O as it is,
          // in the ring (no copy or MMA uses it any more), 16-byte pieces
          // permuted by the row
          reinterpret_cast<float2*>(smem + C::OFF_ML)[r_in] = make_float2(m_run, l_run);
          const uint32_t row_at = smem_u32(smem + C::OFF_RING) + r_in * (D * 4);
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t u[32];
            tmem_ld32(tmem + lane_addr + C::O_COL0 + c0, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              st_shared_v4(row_at + (((c0 >> 2) + (i ^ (lane & 7))) << 4), u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
          }
          break;
        }
        const float f = (l_run > 0.0f) ? (1.0f / l_run) : 0.0f;
        const float lse_row = (m_run + lg2(l_run)) * 0.69314718055994530942f;
        const uint32_t o_addr = tmem + lane_addr + C::O_COL0 + t * D;
        const size_t out_row = valid ? out_row_of() : 0;
        if (w.part >= 0) {
          // fp32 partial: O normalised over this run's keys and the run's LSE
          float* prow = prm.o_part + out_row * D;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t u[32];
            tmem_ld32(o_addr + c0, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * f);
            if (valid) {
#pragma unroll
              for (int i = 0; i < 4; ++i) st_global_v8(prow + c0 + 8 * i, u + 8 * i);
            }
          }
          if (valid) prm.lse_part[out_row] = lse_row;
        } else if constexpr (C::EPI_TMA) {
          // this warp's 32 rows through its staging box, 64 columns at a time
          // (128-byte swizzle: 16-byte chunk c of row `lane` at c ^ (lane % 8))
          uint8_t* stg = smem + C::OFF_EPI + (t * 4 + wq) * C::EPI_WARP_BYTES;
          const uint32_t my_row = smem_u32(stg) + (uint32_t)lane * 128u;
          const int row0 = w.q_row + t * kBM + wq * 32;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 64) {
            uint32_t u[32], u2[32], pk[32];
            tmem_ld32(o_addr + c0, u);
            tmem_ld32(o_addr + c0 + 32, u2);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float a = __uint_as_float(u[2 * i]) * f, b = __uint_as_float(u[2 * i + 1]) * f;
              const float a2 = __uint_as_float(u2[2 * i]) * f, b2 = __uint_as_float(u2[2 * i + 1]) * f;
              pk[i] = (ELEM == kFP16) ? pack_f16x2(a, b) : pack_bf16x2(a, b);
              pk[16 + i] = (ELEM == kFP16) ? pack_f16x2(a2, b2) : pack_bf16x2(a2, b2);
            }
            if (lane == 0) bulk_wait_read_all();  // the previous box has been read out of the buffer
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 8; ++c)
              st_shared_v4(my_row + ((uint32_t)(c ^ (lane & 7)) << 4), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2],
                           pk[4 * c + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && row0 < prm.N) {  // rows at or past N are outside the map and not written
              tma_store_3d(&tm_o, stg, c0, row0, w.qz);
              bulk_commit_group();
            }
          }
          if (valid) prm.lse[out_row] = lse_row;
        } else {
          uint8_t* orow = reinterpret_cast<uint8_t*>(prm.o) + out_row * D * 2;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t u[32], pk[16];
            tmem_ld32(o_addr + c0, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float a = __uint_as_float(u[2 * i]) * f, b = __uint_as_float(u[2 * i + 1]) * f;
              pk[i] = (ELEM == kFP16) ? pack_f16x2(a, b) : pack_bf16x2(a, b);
            }
            if (valid) {
              if (prm.o_vec32) {
#pragma unroll
                for (int i = 0; i < 2; ++i) st_global_v8(orow + c0 * 2 + 32 * i, pk + 8 * i);
              } else {
                uint4* dst = reinterpret_cast<uint4*>(orow + c0 * 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) dst[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
              }
            }
          }
          if (valid) prm.lse[out_row] = lse_row;
        }
        // this warp's reads of O are ordered before the next unit's S, which
        // the MMA warp issues after this tile's next P arrives
        tc_fence_before();
      } while (0);
      if constexpr (!C::ALT) it += nrun;
      __syncwarp();  // every lane is done with the slot
      if (lane == 0) mbar_arrive(&bars->unit_empty[rr & 1]);
    }
    // a warp that others may wait for at their unit's join meets them there
    if (C::FEW && !left) bar_and(1, 128, false);
  }
  // the epilogue's bulk stores have completed before the CTA ends
  if (C::EPI_TMA && warp < C::SOFTMAX_WARPS && lane == 0) bulk_wait_all();
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if constexpr (C::SPLIT) {
    // the join; all threads arrive at both barriers, also after a wait that ran out
    cluster_sync();
    const WinUnit& w = bars->unit[0];
    const int n_cta = cluster_size();
    if (n_cta == 8) cluster_join<C, 8>(smem, w, prm);
    else if (n_cta == 4) cluster_join<C, 4>(smem, w, prm);
    else cluster_join<C, 2>(smem, w, prm);
    cluster_sync();  // the others have read this CTA's shared memory
  }
}

struct WinLaunch {
  CUtensorMap q, k, v;
  CUtensorMap o;      // dense d <= 128: O in boxes of 64 columns x 32 rows
  WinParams prm;
  int grid;           // paged: CTAs (the partial slots and desc are sized for it)
  int cluster;        // WIN_SPLIT: CTAs per query tile
  cudaStream_t stream;
};

template <int ELEM, int D, bool PAGED, int FORM = (D <= 128 ? WIN_PAIR : WIN_ONE), bool TREE = false>
cudaError_t launch_attn_window(const WinLaunch& L) {
  using C = WinCfg<ELEM, D, PAGED, FORM>;
  auto kern = attn_window_kernel<ELEM, D, PAGED, FORM, TREE>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  // per function and device: the shared memory limit, and that the register
  // split fits what the kernel is launched with (the growing warpgroups
  // would otherwise wait for registers that never come)
  static int ready[64] = {};
  if (ready[dev] == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, kern);
    if (e != cudaSuccess) return e;
    const bool fits = !C::REALLOC || at.numRegs * C::THREADS >= 128 * C::CTRL_REGS + C::SOFTMAX_WARPS * 32 * C::SOFTMAX_REGS;
    ready[dev] = fits ? 1 : -1;
  }
  if (ready[dev] != 1) return cudaErrorInvalidConfiguration;
  WinParams prm = L.prm;
  long long grid = L.grid;
  if constexpr (!PAGED) {
    // Groups of two query tiles.  When the last wave of SMs is at most half
    // full its groups run as two units of one tile, each of which takes 0.55
    // to 0.6 of a pair's time; a call of less than half a wave runs so whole.
    static int sms[64] = {};
    if (sms[dev] == 0) {
      e = cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return e;
    }
    const long long groups = (long long)prm.BH * ((prm.N + C::NQT * kBM - 1) / (C::NQT * kBM));
    const long long rem = groups % sms[dev];
    prm.pair_units = (int)(C::NQT == 2 && rem > 0 && 2 * rem <= sms[dev] ? groups - rem : groups);
    grid = prm.pair_units + C::NQT * (groups - prm.pair_units);
    if (C::SPLIT) grid *= L.cluster;
    // chunks of heads whose keys and values fill about half of L2, as in attn_fwd.cuh
    prm.head_chunk = prm.BH;
    const long long kv_head_bytes = 2LL * prm.Nk * C::ROW_BYTES;
    const int qgroup = prm.Hq / prm.Hkv;
    long long chunk = ((64LL << 20) / (kv_head_bytes > 0 ? kv_head_bytes : 1)) * qgroup;
    if (chunk < qgroup) chunk = qgroup;
    if (chunk < prm.BH) prm.head_chunk = (int)chunk;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[1];
  if constexpr (PAGED) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  } else {
    attr[0].id = cudaLaunchAttributeClusterDimension;  // work stealing asks for whole clusters
    attr[0].val.clusterDim.x = C::SPLIT ? L.cluster : 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, L.q, L.k, L.v, L.o, prm);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// How many WIN_SPLIT clusters of n CTAs (2, 4 or 8) run at once on a device
// (GB300: 76, 36 and 15, as clusters do not cross its GPCs).
int window_clusters(int dev, int n);

}  // namespace fa
