// What the kernels over a block-scaled 8-bit cache share: the work's units, parameters, windows, the
// schedule, a CTA's run of tiles.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "mfa.h"
#include "mfa_device.cuh"
#include "mfa_host.h"
#include "ptx.cuh"

namespace mfa {

constexpr int kBPage = 64;
constexpr int kBTile = 128;           // tokens of a tile (two pages)
constexpr int kBCostTile = 4;         // schedule: cost of a tile
// and of a unit boundary inside a CTA's range: the pipeline drains and fills again (61 ragged
// sequences, two new tokens: 67.8 us at a cost of 6, 65.0 at 12, 64.2 at 16)
constexpr int kBCostUnit = 16;
constexpr int kBMaxSeg = 256;         // units that one CTA can meet
constexpr int kBMaxShare = (kBMaxSeg - 2) * (kBCostTile + kBCostUnit);   // a range of this cost holds no more, whatever the lengths
constexpr uint64_t kBWsHeader = 256;
constexpr int kTreeRows = 128;        // query rows of a unit of a tree's kernel
constexpr int kBSmem = 227 * 1024 - 1024;   // dynamic shared memory after its alignment
// The work of one problem: a unit is (sequence, key/value head, group of new tokens); its rows
// are the group's new tokens x the query heads that read that head.
struct BlockShape {
  int group;      // query heads of a key/value head
  int unit_tokens;   // new tokens of a unit
  int token_groups;  // units along the new tokens
  int readers;    // units of a sequence
  int rows;       // rows of a unit (its last token group may use fewer)
  int rows8;      // and padded to 8, as partial results are laid out
};

inline BlockShape block_shape(const mfa_problem* pr, int most_rows) {
  BlockShape s;
  s.group = pr->num_q_heads / pr->num_kv_heads;
  s.unit_tokens = std::min(pr->tokens_per_seq, most_rows / s.group);
  s.token_groups = (pr->tokens_per_seq + s.unit_tokens - 1) / s.unit_tokens;
  s.readers = s.token_groups * pr->num_kv_heads;
  s.rows = s.group * s.unit_tokens;
  s.rows8 = (s.rows + 7) / 8 * 8;
  return s;
}

// Workspace: header; partial O; partial lse; and for each unit the slots of its first and last part.
inline uint64_t block_lse_offset(long long partials, const BlockShape& s, int d) {
  const uint64_t x = kBWsHeader + static_cast<uint64_t>(partials) * s.rows8 * d * 4;
  return (x + 255) / 256 * 256;
}
inline uint64_t block_parts_offset(long long partials, const BlockShape& s, int d) {
  return (block_lse_offset(partials, s, d) + static_cast<uint64_t>(partials) * s.rows8 * 4 + 255) / 256 * 256;
}
inline uint64_t block_workspace_bytes(long long partials, const BlockShape& s, int batch, int d) {
  return (block_parts_offset(partials, s, d) + static_cast<uint64_t>(batch) * s.readers * 8 + 255) / 256 * 256;
}

struct BlockDecodeParams {
  CUtensorMap tm_k, tm_v;    // codes [pages * heads][64][d], boxes of one page and head, 128 bytes wide
  const __nv_bfloat16* q;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  void* out;
  float* lse;
  float* part_o;             // [partials][rows8 / 8][d][8 rows]: 32 bytes a thread of the epilogue (trees: [partials][rows8][d])
  float* part_lse;           // [partials][rows8]
  unsigned int* status;
  int batch, tokens, heads, kv_heads;
  int group, unit_tokens, token_groups, readers, rows8;   // BlockShape
  int num_partials;
  int2* parts;               // split by cost: [units] slots of a unit's first and last part
  int narrow;                // split by cost: G times the whole cost fits 32 bits
  int quantum;               // even split: most tiles of a part; else 0
  int cluster;               // CTAs of a unit, one cluster; 0: split evenly or by cost
  int log_scale;             // log2(scale_tokens)
  int max_pages, num_blocks;
  int window, sinks;         // windowed instances: the tokens that a new token sees (0: all)
  const uint64_t* tree;      // trees: [batch][tokens] masks of the nodes that a node sees
  float scale_log2;          // softmax_scale * log2(e)
  int out_f32;
  int early_metadata;
};

// ------------------------------------------------------------------ windows
//
// With a window, new token i of a sequence's T, at position p = L - T + i, sees the tokens t <= p with
// t < sinks or t > p - window.  The pages between the sinks' and the first that the window of new token 0
// touches are left out, and the rest laid end to end: a sequence of L' = L - 64 skip tokens, on which
// everything else works as on any other, but for where a page lies and what a row sees:
//   page v is the sequence's page v, or v + skip from the sinks' pages on;
//   row i sees t' < L' - T + 1 + i with t' < sinks or t' >= low + i (both also where nothing is left out:
//   every t' in a sink's page behind the sinks is under low).
// A page's rows under the window's first token are not loaded, nor those behind the last sink, so that
// whatever they hold reaches nothing: the box starts at the first row that anyone sees and is filled with
// zeros behind the page, as the last page's box is before it.  Where a box cannot leave out what no one
// sees (the window starts in the last page, or in the last of the sinks'), the PV issuer's warp zeroes
// those rows of the values.
//
// What bounds it: a window's cache is read from the first row that counts (41 us of bytes for 128 sequences
// with windows of 4096, 64 heads of 256: 55.5 us, 51.1 without a window, on a kernel that has less to do at a
// tile's edges; grouped heads, 32 x 1024 of 16K to 128K tokens: 13.5 us, one sequence with a window of 128 11.5 and
// of 512 without one 11.1, a chain of latencies both; in a graph of twelve calls over three states).  The way
// there, for the 128 (a graph of one call, some 3 us more): the edge looked for in every tile 74 us, edge tiles
// known a segment ahead and the others' plain path 62, MMAs issued by a converged warp 57.4, q's lo part 16
// times larger (one multiplication more, log sums of a few tokens to 1e-7) 58.3.
struct BlockView {
  int L, skip, low, sink_pages;
  int plain;   // from this page on only the end of L cuts a page's rows
};
__host__ __device__ __forceinline__ BlockView block_view(int L, int tokens, int window, int sinks) {
  BlockView v;
  v.low = L - tokens - window + 1;   // new token 0's first token of its window (window <= the table's tokens)
  v.sink_pages = (sinks + kBPage - 1) / kBPage;
  v.skip = v.low > 0 ? v.low / kBPage - v.sink_pages : 0;
  if (v.skip < 0) v.skip = 0;
  v.L = L - kBPage * v.skip;
  v.low -= kBPage * v.skip;
  v.plain = v.low > 0 && v.low / kBPage >= v.sink_pages ? v.low / kBPage + 1 : v.sink_pages;
  return v;
}
// The tokens that a sequence of L has to go over.
template <bool kWindow>
__device__ __forceinline__ int view_length(const BlockDecodeParams& p, int L) {
  if constexpr (kWindow) return block_view(L, p.tokens, p.window, p.sinks).L;
  return L;
}

// ------------------------------------------------------------------ schedule
//
// The units of the batch lie end to end, reader-major (reader r = head * token groups + token
// group; unit (b, r) at position r B + b): tile k of a unit sits at cost 4 k past the unit's
// base, and the next unit's base is 4 T + c further (T tiles, c = kBCostUnit for the boundary;
// nothing for an empty sequence).  CTA g of G owns the tiles whose cost lies in
// [floor(g C / G), floor((g + 1) C / G)), C the whole cost: equal shares for any length mix.  Where lengths
// have grown so far past the plan's that such a range could hold more units than a CTA can meet, all CTAs
// take a higher c (grown_boundary).
//
// Two other ways, for few units:
// Clusters: every unit (b, r) has c CTAs of its own, CTA c (r B + b) + i taking part i, tiles
// [floor(i T / c), floor((i + 1) T / c)); c > 1: the CTAs are a cluster and exchange their results.
// Even split: a unit of T tiles is cut into n = ceil(T / quantum) parts as equal as they come.
// Part i of reader r of sequence b is item R P_b + r n + i (R readers, P_b parts of one reader of
// each sequence before b), and CTA g takes items g, g + G, ...: one part each, none with the end
// of one unit and the beginning of another.  Where lengths have grown past those of the plan the
// parts may be more than the workspace's slots: then every CTA takes the same larger quantum
// (wider_quantum), and some CTAs two items.
__device__ __forceinline__ int even_parts(int T, int quantum) {
  return T <= quantum ? (T > 0 ? 1 : 0) : (T + quantum - 1) / quantum;
}
// A quantum with which the units' parts are no more than the slots: with W tiles in N units
// (all readers), sum ceil(T / q) <= W / q + N, and W / q <= slots - N.  (One warp; out of the way.)
template <bool kWindow>
__device__ __noinline__ int wider_quantum(const BlockDecodeParams& p, int cap) {
  long long tiles = 0, units = 0;
  bool bad = false;
  for (int b = threadIdx.x & 31; b < p.batch; b += 32) {
    const int T = (view_length<kWindow>(p, clamp_len(p.seq_lens[b], cap, bad)) + kBTile - 1) / kBTile;
    tiles += T;
    units += T > 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
    units += __shfl_xor_sync(0xffffffffu, units, o);
  }
  const long long spare = p.num_partials - units * p.readers;   // (>= 0: a slot a unit is there)
  return spare < 1 ? INT_MAX : static_cast<int>(min((tiles * p.readers + spare - 1) / spare, static_cast<long long>(INT_MAX)));
}
// first of a unit's T tiles at cost >= X
template <typename I>
__device__ __forceinline__ int first_tile_at(I X, I base, int T) {
  return X <= base ? 0 : static_cast<int>(min(static_cast<I>(T), (X - base + kBCostTile - 1) / kBCostTile));
}
__device__ __forceinline__ int block_tiles(int L) { return (L + kBTile - 1) / kBTile; }

// Bounded wait on an mbarrier phase; what runs when the phase is not over yet stays out of line.
// False (after wait_bar's limit, or at once when the CTA is aborting): the caller carries on and
// leaves at its next common exit.
static __device__ __noinline__ bool block_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return wait_bar(bar, parity, abort_flag);
}
__device__ __forceinline__ bool block_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || block_wait_slow(bar, parity, abort_flag);
}

// A value that is one for the warp, told to the compiler.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Four e4m3 codes of two pairs of halves, and back; four e5m2 codes.
__device__ __forceinline__ uint32_t cvt_e4m3x4(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b16 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 x, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 y, %2;\n\t"
      "mov.b32 %0, {x, y};\n\t}"
      : "=r"(r)
      : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t cvt_e5m2x4(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b16 x, y;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 x, %1;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 y, %2;\n\t"
      "mov.b32 %0, {x, y};\n\t}"
      : "=r"(r)
      : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void cvt_f16x4(uint32_t codes, uint32_t& a, uint32_t& b) {
  asm("{\n\t.reg .b16 x, y;\n\t"
      "mov.b32 {x, y}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, x;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(codes));
}

// A segment: one unit's tiles of this CTA.
struct __align__(16) BlockSegment {
  int b, kvh, tg, L;       // sequence, key/value head, group of new tokens, length
  int lo, hi;              // tiles
  int slot;                // of the partial result; -1: the whole unit; -2: a part, for the cluster's exchange
};

template <bool kWindow>
__device__ __forceinline__ void add_segment(const BlockDecodeParams& p, BlockSegment* seg, int at, int b, int r, int L, int lo,
                                            int hi, long long slot) {
  if (at >= kBMaxSeg) return;
  BlockSegment x;
  x.b = b;
  x.kvh = p.token_groups == 1 ? r : r / p.token_groups;
  x.tg = r - x.kvh * p.token_groups;
  x.L = L;
  x.lo = lo;
  x.hi = hi;
  x.slot = lo == 0 && hi == block_tiles(view_length<kWindow>(p, L)) ? -1 : static_cast<int>(slot);
  seg[at] = x;
}

// This CTA's segments, by one warp (a lane a sequence), into shared memory; their number and this
// lane's tiles in (nseg, tiles).  Every CTA runs it before its first load, so it is kept short (61
// sequences by cost: 2.3 us, evenly 1.0, one unit a cluster 0.8).
template <bool kWindow>
__device__ __forceinline__ void even_segments(const BlockDecodeParams& p, int cap, BlockSegment* seg, int& nseg, int& tiles,
                                              bool& bad) {
  const int lane = threadIdx.x & 31;
  int quantum = p.quantum;
#pragma unroll 1
  while (true) {
    long long item = blockIdx.x, carry = 0;   // the item that is looked for; items of the sequences passed
    int next = lane < p.batch ? p.seq_lens[lane] : 0;
#pragma unroll 1
    for (int c0 = 0; c0 < p.batch; c0 += 32) {
      const int L = clamp_len(next, cap, bad);
      next = c0 + 32 + lane < p.batch ? p.seq_lens[c0 + 32 + lane] : 0;
      const int T = block_tiles(view_length<kWindow>(p, L)), n = even_parts(T, quantum);
      const long long own = static_cast<long long>(n) * p.readers;
      long long incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const long long before = carry + incl - own;
      carry += __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll 1
      while (item < carry && nseg <= kBMaxSeg) {
        if (item >= before && item < before + own) {
          int r = static_cast<int>(item - before), lo = 0, hi = T;
          if (n > 1) {   // part i: T / n tiles, the first T % n parts one more
            const int i = r % n, each = T / n, more = T - each * n;
            r /= n;
            lo = i * each + min(i, more);
            hi = lo + each + (i < more ? 1 : 0);
          }
          add_segment<kWindow>(p, seg, nseg, c0 + lane, r, L, lo, hi, item);
          tiles += hi - lo;
        }
        ++nseg;
        item += gridDim.x;
      }
    }
    if (carry <= p.num_partials) return;
    quantum = wider_quantum<kWindow>(p, cap);
    nseg = tiles = 0;
  }
}

// I: the type that holds G times the whole cost (32 bits nearly always: its divisions are short).  With a boundary's cost of
// `boundary`; in 32 bits false where a CTA's range could then hold too many units.
template <typename I, bool kWindow>
__device__ __forceinline__ bool cost_segments(const BlockDecodeParams& p, int cap, BlockSegment* seg, int& nseg, int& tiles,
                                              bool& bad, I boundary) {
  const int lane = threadIdx.x & 31;
  auto length = [&](int b) { return b < p.batch ? clamp_len(p.seq_lens[b], cap, bad) : 0; };
  auto cost = [boundary](int T) { return T > 0 ? static_cast<I>(kBCostTile) * T + boundary : I{0}; };
  const int L0 = length(lane);
  I per = cost(block_tiles(view_length<kWindow>(p, L0)));   // of one reader of every sequence
#pragma unroll 1
  for (int b = lane + 32; b < p.batch; b += 32) per += cost(block_tiles(view_length<kWindow>(p, length(b))));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) per += __shfl_xor_sync(0xffffffffu, per, o);
  if (per == 0) return true;
  // the whole cost; with less of it than a tile for each CTA the last CTAs have nothing, so that
  // no CTA lies between two tiles
  const I total = per * p.readers - boundary;
  if (sizeof(I) == 4 && (total - 1) / kBMaxShare >= gridDim.x) return false;
  const I G = min(static_cast<I>(gridDim.x), total / kBCostTile), g = blockIdx.x;
  if (g >= G) return true;
  const I X0 = g * total / G, X1 = (g + 1) * total / G;
  I rbase = X0 / per;   // the reader at X0, then its base
  int r = static_cast<int>(rbase);
  rbase *= per;
#pragma unroll 1
  for (; rbase < X1 && nseg <= kBMaxSeg; ++r, rbase += per) {
    I carry = rbase;
    int next = L0;
#pragma unroll 1
    for (int c0 = 0; c0 < p.batch && carry < X1; c0 += 32) {
      const int L = next;
      next = length(c0 + 32 + lane);
      const int T = block_tiles(view_length<kWindow>(p, L));
      const I own = cost(T);
      I incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const I v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const I base = carry + incl - own;
      const int lo = first_tile_at(X0, base, T), hi = first_tile_at(X1, base, T);
      const unsigned has = __ballot_sync(0xffffffffu, lo < hi);
      if (lo < hi) {
        add_segment<kWindow>(p, seg, nseg + __popc(has & ((1u << lane) - 1u)), c0 + lane, r, L, lo, hi,
                    static_cast<long long>(r) * p.batch + c0 + lane + blockIdx.x);
        tiles += hi - lo;
      }
      nseg += __popc(has);
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  return true;
}
// A boundary's cost c with which no CTA's range holds more than kBMaxSeg units: units begin at least 4 + c apart, so a
// range of X holds ceil(X / (4 + c)) + 1 at most, and with W tiles in N units X <= (4 W + c (N - 1)) / G + 1.  The usual c
// where that does, or where units are few; and with too few CTAs (N - 1 > (kBMaxSeg - 2) G), which a plan makes only where its
// grid is forced.
template <bool kWindow>
__device__ __forceinline__ long long grown_boundary(const BlockDecodeParams& p, int cap) {
  long long tiles = 0, units = 0;
  bool bad = false;
#pragma unroll 1
  for (int b = threadIdx.x & 31; b < p.batch; b += 32) {
    const int T = block_tiles(view_length<kWindow>(p, clamp_len(p.seq_lens[b], cap, bad)));
    tiles += T;
    units += T > 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
    units += __shfl_xor_sync(0xffffffffu, units, o);
  }
  tiles *= p.readers;
  units *= p.readers;
  const long long G = gridDim.x, spare = (kBMaxSeg - 1) * G - (units - 1);
  if (units <= kBMaxSeg || spare < 1 || kBCostTile * tiles + kBCostUnit * (units - 1) <= kBMaxShare * G) return kBCostUnit;
  return max((kBCostTile * (tiles - (kBMaxSeg - 1) * G) + spare - 1) / spare, static_cast<long long>(kBCostUnit));
}
// The wide form, for problems of millions of tiles and lengths far past the plan's, out of the way of the usual one's code and
// in one copy: waits for instructions are a part of the decode's time (61 ragged sequences, two new tokens, a graph of one
// call: 65.7 us, 67.8 with two copies, 68.1 with the usual form out of line too).
template <bool kWindow>
__device__ __noinline__ void cost_segments_wide(const BlockDecodeParams& p, int cap, BlockSegment* seg, int& nseg, int& tiles,
                                                bool& bad) {
  cost_segments<long long, kWindow>(p, cap, seg, nseg, tiles, bad, grown_boundary<kWindow>(p, cap));
}

// A unit's CTAs: only its own sequence's length is read.
template <bool kWindow>
__device__ __forceinline__ void unit_segment(const BlockDecodeParams& p, int cap, BlockSegment* seg, int& nseg, int& tiles,
                                             bool& bad) {
  if ((threadIdx.x & 31) != 0) return;
  const unsigned c = p.cluster, unit = c == 1 ? blockIdx.x : blockIdx.x / c, i = blockIdx.x - unit * c;
  const int r = unit / p.batch, b = unit - r * p.batch;
  const int L = clamp_len(p.seq_lens[b], cap, bad);
  const unsigned T = block_tiles(view_length<kWindow>(p, L));
  const int lo = c == 1 ? 0 : i * T / c, hi = c == 1 ? T : (i + 1) * T / c;
  add_segment<kWindow>(p, seg, 0, b, r, L, lo, hi, -2);   // (without tiles too: the exchange wants the unit)
  nseg = lo < hi ? 1 : 0;
  tiles = hi - lo;
}

template <bool kWindow>
__device__ __forceinline__ void block_segments(const BlockDecodeParams& p, int cap, BlockSegment* seg, int* counts) {
  int nseg = 0, tiles = 0;
  bool bad = false;
  if (p.cluster > 0)
    unit_segment<kWindow>(p, cap, seg, nseg, tiles, bad);
  else if (p.quantum > 0)
    even_segments<kWindow>(p, cap, seg, nseg, tiles, bad);
  else if (!p.narrow || !cost_segments<uint32_t, kWindow>(p, cap, seg, nseg, tiles, bad, kBCostUnit))
    cost_segments_wide<kWindow>(p, cap, seg, nseg, tiles, bad);
  if (bad) atomicOr(p.status, MFA_DEV_BAD_LENGTH);
  tiles = __reduce_add_sync(0xffffffffu, tiles);
  if (nseg > kBMaxSeg) {
    if ((threadIdx.x & 31) == 0) atomicOr(p.status, MFA_DEV_SCHEDULE);
    nseg = tiles = 0;
  }
  if ((threadIdx.x & 31) == 0) {
    counts[0] = nseg;
    counts[1] = tiles;
  }
}

// The rows of page v of a sequence that any new token sees: [from, to), none where to <= 0; page row
// `first` lies in the box's row 0.
struct BlockRows {
  int from, to, first;
};
template <bool kWindow>
__device__ __forceinline__ BlockRows view_rows(const BlockView& w, int sinks, int v) {
  BlockRows r = {0, min(kBPage, w.L - kBPage * v), 0};
  if constexpr (kWindow) {
    if (v < w.plain && w.low >= kBPage * w.sink_pages) {   // the window starts behind the sinks' pages
      if (v == w.sink_pages - 1) r.to = min(r.to, sinks - kBPage * v);
      if (v == w.low / kBPage) r.from = w.low % kBPage;
    }
  }
  r.first = kWindow && r.from > 0 && r.to == kBPage ? r.from : r.to - kBPage;
  return r;
}

// The page, of one sequence, whose box has rows that are loaded and that no new token sees: box rows
// [from, to) of page v; v < 0 where there is none.
struct BlockGap {
  int v, from, to;
};
__device__ __forceinline__ BlockGap view_gap(const BlockView& w, int sinks) {
  const int v = w.low >= kBPage * w.sink_pages ? w.low / kBPage : w.sink_pages - 1;
  const BlockRows r = view_rows<true>(w, sinks, v);
  int from = 0, to = 0;
  if (w.low >= kBPage * w.sink_pages)
    to = r.first < 0 ? r.from : 0;   // (the box starts at the window's first token where it can)
  else
    from = sinks - kBPage * v, to = min(w.low - kBPage * v, r.to);
  return {from < to ? v : -1, from - r.first, to - r.first};
}

// A role's place in its CTA's run of tiles.
template <bool kWindow>
struct BlockTile {
  int s, j, end;           // segment, tile of the sequence, end of the segment
  int b, kvh;
  BlockView w;
  bool again;              // another unit reads the tile's pages after this one
  __device__ __forceinline__ void load(const BlockDecodeParams& p, const BlockSegment* seg, int at) {
    const BlockSegment x = seg[at];
    s = at;
    b = x.b;
    kvh = x.kvh;
    if constexpr (kWindow)
      w = block_view(x.L, p.tokens, p.window, p.sinks);
    else
      w.L = x.L;
    j = x.lo;
    end = x.hi;
    again = x.tg != p.token_groups - 1;
  }
  // the next tile; false past the last
  __device__ __forceinline__ bool next(const BlockDecodeParams& p, const BlockSegment* seg, int nseg) {
    if (++j < end) return true;
    if (s + 1 >= nseg) return false;
    load(p, seg, s + 1);
    return true;
  }
  // the tile's page pg in the sequence's table, and its rows
  __device__ __forceinline__ int page(int pg) const {
    const int v = 2 * j + pg;
    return kWindow && v >= w.sink_pages ? v + w.skip : v;
  }
  __device__ __forceinline__ BlockRows rows(const BlockDecodeParams& p, int pg) const { return view_rows<kWindow>(w, p.sinks, 2 * j + pg); }
};

using BlockDecodeFn = void (*)(BlockDecodeParams);

// The kernel of drafted trees for a head width, and its threads (defined in mfa_tree_decode.cu).
BlockDecodeFn tree_kernel(int head_dim);
int tree_threads();
// Enqueues the merge of the units' parts that the kernel's CTAs left (cfg: stream and attributes).
cudaError_t launch_tree_combine(const BlockDecodeParams& p, int units, int ctas, int head_dim, cudaLaunchConfig_t cfg);

}  // namespace mfa
