// Decode attention over a block-scaled 8-bit KV cache (GB300, sm_103a): e4m3 codes with one
// fp32 scale for each block of tokens and key/value head.
//
// For token i of sequence b and query head h, over the tokens t that it sees:
//     s_t = softmax_scale * sk_t * dot(q, k_t),  out = sum_t e^(s_t) sv_t v_t / sum_t e^(s_t),
//     lse = ln sum_t e^(s_t),
// k_t and v_t being the e4m3 codes' values and sk_t, sv_t their blocks' scales.
//
// A unit is a sequence, a key/value head and as many new tokens as fit 64 rows (tokens x the head's
// query heads); a tile is 128 tokens.  Both contractions run on the codes as they lie in the cache:
//   S^T [128 tokens x rows] = K Q^T, q split into e4m3 hi + lo parts under one power of two a row
//     (exact, but for elements under 2^-9 of the row's largest, which err by 2^-16 of it), in
//     columns of their own; a token's key scale multiplies its fp32 scores;
//   O^T [128 of d x rows] += V^T P^T, the weights (with the token's value scale) split likewise.
// Tokens as the MMAs' M = 128 keep the tensor core full however few the rows, and let a softmax
// thread own a token, so that a token's scales are its own two registers.  Sums, references and
// accumulators are fp32.
//
// Warps: a producer (TMA boxes of one page into rings of 16 KB slots, K's and V's apart, so that a
// tile's keys never wait behind another's values), the issuers of the two MMAs, one that fetches
// block scales a tile ahead, and 2 or 4 warpgroups of softmax, each with all tokens and a share of
// the rows.  The running maximum is a reference that moves only when weights leave a range around
// it (then O is rescaled in tensor memory), so that an ordinary tile costs one vote.
//
// What bounds it: for one new token a sequence the cache's bytes (512 a token at d = 256);
// 64 rows, 128 sequences of 4096, one CTA each: 51.3 us, 5.4 TB/s, 79% of the copy rate; of the
// rest some 5 us are the beginning (lengths, q, the first tile's way through five stages), 2 us the
// end and 2 us moves of references.  Short batches are bound by that chain (one sequence of 512:
// 10.8 us).  Several tokens' units of a sequence read the same pages (from L2), and nothing alone
// bounds them: a tile of 64 rows takes some 2300 clocks, of which its 208 KB are 1625 of shared
// memory at 128 bytes a clock, and whole captures show shared memory's pipe and the tensor cores at
// a third, issue slots at a half.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdint>
#include <cstring>
#include <vector>

#include "mfa.h"
#include "mfa_host.h"
#include "ptx.cuh"
#include "mfa_device.cuh"

namespace mfa {

constexpr int kBPage = 64;
constexpr int kBTile = 128;           // tokens of a tile (two pages)
constexpr int kBRows = 64;            // query rows (new tokens x heads of one group) a unit holds at most
constexpr int kBCostTile = 4;         // schedule: cost of a tile
// and of a unit boundary inside a CTA's range: the pipeline drains and fills again (61 ragged
// sequences, two new tokens: 67.8 us at a cost of 6, 65.0 at 12, 64.2 at 16)
constexpr int kBCostUnit = 16;
constexpr int kBMaxSeg = 256;         // units that one CTA can meet
constexpr uint64_t kBWsHeader = 256;
constexpr int kBScaleWarp = 2, kBPvWarp = 3, kBSoftmaxWarp0 = 4;   // warps: producer, QK issuer, scales, PV issuer, softmax
constexpr int kBCombineThreads = 256;
constexpr int kBSmem = 227 * 1024 - 1024;   // dynamic shared memory after its alignment
constexpr int kBMisc = 12288;         // of it, behind the ring: segments, scratch, barriers (the last 512)
// Weights: p = 2^x, x a score in powers of two relative to its row's reference, goes into the row's
// sum as it is; P = p s_v, s_v the token's value scale, is what is rounded.  The reference
// is set by x + e, e the exponent of s_v, so that rounding is relative to the row's own P whatever
// scales there are elsewhere.  Two parts, the second 32 times larger, resolve P to 2^-14 from 2^8
// down (448 is e4m3's largest, and the first part leaves up to 8), and a P under 2^-15 is lost; so
// the reference follows what a row is made of.  It is set under a tile's largest x + e (in powers of
// two, as all here): 1 under it, or as far, up to 6, as brings the other tokens up where few outweigh
// them, as first tokens do (a quarter of the tile outweighs the others by 4 and more, or one of them by
// 7 and more):
//   it rises when x + e passes 7 over it, and then for the warpgroup's other rows too where that is a
//   rise (rows that rise by themselves only come to half as many moves again);
//   it falls, to 24 below its highest at most, in a tile that is looked at and whose largest x + e is 4
//   under it (without that, 32768 tokens behind one of 0.8 of the weight came out as 0.1 of their sum).
// A tile is looked at where the one before holds few tokens 11 over the others, or the eighth after it
// if that happens again and again, and 32 tiles after the last look.
// Measured on 8000 tokens of normal scores behind one to three of next to no value that stand 5 to 11
// nats above: the output row is off by 0.005 at most, by 0.4 to 0.6 with a reference that only rises.
// Every move costs its CTA a microsecond or two.  128 sequences of 4096 with the queries as they are /
// 2 / 3 times as large (deviations of the scores up to 2, 4, 6): 51.1 / 64.7 / 76.8 us, 49.3 / 52.6 /
// 55.5 with a reference that only rises; 62 for the first with 6 of room for all rows.
// Scales are taken 2^-24 times smaller, the results as many times larger: p = 2^(x - reference)
// and its sums then stay in fp32's range for scales from 2^-50 (smaller ones count as that: an
// empty block's is 2^-126, and its P next to nothing either way) to the largest.
constexpr float kBThreshold = 7.0f, kBLow = -4.0f, kBDepth = 24.0f, kBRoom = 1.0f, kBRoomFew = 6.0f, kBOver = 11.0f, kBNear = 4.0f;
constexpr int kBLookEvery = 32;
constexpr float kBScaleDown = 0x1p-24f, kBScaleUp = 0x1p24f;
constexpr int kBEMin = -50 - 24, kBEMax = 127 - 24;
constexpr float kBPart = 32.0f;   // the second part's factor

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

static BlockShape block_shape(const mfa_problem* pr) {
  BlockShape s;
  s.group = pr->num_q_heads / pr->num_kv_heads;
  s.unit_tokens = std::min(pr->tokens_per_seq, kBRows / s.group);
  s.token_groups = (pr->tokens_per_seq + s.unit_tokens - 1) / s.unit_tokens;
  s.readers = s.token_groups * pr->num_kv_heads;
  s.rows = s.group * s.unit_tokens;
  s.rows8 = (s.rows + 7) / 8 * 8;
  return s;
}

// Workspace: header; partial O; partial lse; and for each unit the slots of its first and last part.
static uint64_t block_lse_offset(long long partials, const BlockShape& s, int d) {
  const uint64_t x = kBWsHeader + static_cast<uint64_t>(partials) * s.rows8 * d * 4;
  return (x + 255) / 256 * 256;
}
static uint64_t block_parts_offset(long long partials, const BlockShape& s, int d) {
  return (block_lse_offset(partials, s, d) + static_cast<uint64_t>(partials) * s.rows8 * 4 + 255) / 256 * 256;
}
static uint64_t block_workspace_bytes(long long partials, const BlockShape& s, int batch, int d) {
  return (block_parts_offset(partials, s, d) + static_cast<uint64_t>(batch) * s.readers * 8 + 255) / 256 * 256;
}

// Shared memory and tensor memory of an instance: kDim the head width, kNR the unit's rows
// padded to 16, 32 or 64 (the MMAs' N).
template <int kDim, int kNR>
struct BlockLayout {
  static constexpr int kHalves = kDim / 128;            // 128-byte swizzle rows of a cache row
  // softmax warpgroups: a tile's latency is what bounds them, so each owns no more than 16 rows
  // (64 rows, four warpgroups / two: 32 sequences of 4096 29.2 / 31.1 us, 61 ragged ones with two
  // new tokens 68.8 / 79.7 us, as the kernel stood when both were built)
  static constexpr int kWgs = kNR == 64 ? 4 : 2;
  static constexpr int kC = kNR / kWgs;                 // rows a softmax warpgroup owns
  static constexpr int kThreads = 32 * kBSoftmaxWarp0 + 128 * kWgs;
  static constexpr int kBoxes = 2 * kHalves;            // TMA boxes [64 tokens x 128 B] of a tile of K or V
  static constexpr int kSlotBytes = 16384;              // a ring slot: one half of a tile's two pages
  static constexpr int kPBufs = (kDim == 256 && kNR == 64) ? 1 : 2;
  static constexpr int kOffQ = 0;                       // q: kHalves boxes of [kNR hi rows, kNR lo rows][128 B]
  static constexpr int kOffP = 2 * kNR * kDim;          // weights: [128 tokens][kNR hi, kNR lo], 128-byte rows
  static constexpr int kOffRing = kOffP + kPBufs * 16384;
  static constexpr int kSlots = (kBSmem - kBMisc - kOffRing) / kSlotBytes;
  static constexpr int kKSlots = kSlots / 2, kVSlots = kSlots - kKSlots;   // K and V have rings of their own
  static constexpr int kOffMisc = kOffRing + kSlots * kSlotBytes;
  static constexpr uint32_t kTmemS = 0;                 // S^T, two buffers of kNR hi and kNR lo columns
  static constexpr uint32_t kTmemO = 4 * kNR;           // O^T, for each half kNR hi and kNR lo columns
  static constexpr uint32_t kTmemUsed = 2 * kNR * (2 + kHalves);
  static constexpr uint32_t kTmemCols = kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static_assert(kSlots * kSlotBytes >= (kDim + 1) * kNR * 4, "a part fits the rings");
  static_assert(kTmemUsed <= 512 && kKSlots >= 2 * kHalves && kOffP % 1024 == 0 && kOffRing % 1024 == 0, "layout");
};

struct BlockDecodeParams {
  CUtensorMap tm_k, tm_v;    // codes [pages * heads][64][d], boxes of one page and head, 128 bytes wide
  const __nv_bfloat16* q;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  void* out;
  float* lse;
  float* part_o;             // [partials][rows8 / 8][d][8 rows]: 32 bytes a thread of the epilogue
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
  float scale_log2;          // softmax_scale * log2(e)
  int out_f32;
  int early_metadata;
};

// ------------------------------------------------------------------ schedule
//
// The units of the batch lie end to end, reader-major (reader r = head * token groups + token
// group; unit (b, r) at position r B + b): tile k of a unit sits at cost 4 k past the unit's
// base, and the next unit's base is 4 T + c further (T tiles, c = kBCostUnit for the boundary;
// nothing for an empty sequence).  CTA g of G owns the tiles whose cost lies in
// [floor(g C / G), floor((g + 1) C / G)), C the whole cost: equal shares for any length mix.
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
__device__ __noinline__ int wider_quantum(const BlockDecodeParams& p, int cap) {
  long long tiles = 0, units = 0;
  bool bad = false;
  for (int b = threadIdx.x & 31; b < p.batch; b += 32) {
    const int T = (clamp_len(p.seq_lens[b], cap, bad) + kBTile - 1) / kBTile;
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
__device__ __noinline__ bool block_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return wait_bar(bar, parity, abort_flag);
}
__device__ __forceinline__ bool block_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || block_wait_slow(bar, parity, abort_flag);
}

// Four e4m3 codes of two pairs of halves, and back.
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
__device__ __forceinline__ void cvt_f16x4(uint32_t codes, uint32_t& a, uint32_t& b) {
  asm("{\n\t.reg .b16 x, y;\n\t"
      "mov.b32 {x, y}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, x;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(codes));
}

// Sum kC per-thread values over the 32 lanes: halving exchanges while values are left,
// then whole exchanges of the last one.  Lane l ends with column l / (32 / kC).
template <int kC>
__device__ __forceinline__ float reduce_columns(float (&v)[kC]) {
  const int lane = threadIdx.x & 31;
  int step = 16;
#pragma unroll
  for (int n = kC / 2; n >= 1; n /= 2, step /= 2) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool hi = lane & step;
      const float keep = hi ? v[i + n] : v[i], send = hi ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, step);
    }
  }
#pragma unroll
  for (; step >= 1; step /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], step);
  return v[0];
}

// A segment: one unit's tiles of this CTA.
struct __align__(16) BlockSegment {
  int b, kvh, tg, L;       // sequence, key/value head, group of new tokens, length
  int lo, hi;              // tiles
  int slot;                // of the partial result; -1: the whole unit; -2: a part, for the cluster's exchange
};

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
  x.slot = lo == 0 && hi == block_tiles(L) ? -1 : static_cast<int>(slot);
  seg[at] = x;
}

// This CTA's segments, by one warp (a lane a sequence), into shared memory; their number and this
// lane's tiles in (nseg, tiles).  Every CTA runs it before its first load, so it is kept short (61
// sequences by cost: 2.3 us, evenly 1.0, one unit a cluster 0.8).
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
      const int T = block_tiles(L), n = even_parts(T, quantum);
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
          add_segment(p, seg, nseg, c0 + lane, r, L, lo, hi, item);
          tiles += hi - lo;
        }
        ++nseg;
        item += gridDim.x;
      }
    }
    if (carry <= p.num_partials) return;
    quantum = wider_quantum(p, cap);
    nseg = tiles = 0;
  }
}

// I: the type that holds G times the whole cost (32 bits nearly always: its divisions are short).
template <typename I>
__device__ __forceinline__ void cost_segments(const BlockDecodeParams& p, int cap, BlockSegment* seg, int& nseg, int& tiles,
                                              bool& bad) {
  const int lane = threadIdx.x & 31;
  auto length = [&](int b) { return b < p.batch ? clamp_len(p.seq_lens[b], cap, bad) : 0; };
  auto cost = [](int T) { return T > 0 ? static_cast<I>(kBCostTile) * T + kBCostUnit : I{0}; };
  const int L0 = length(lane);
  I per = cost(block_tiles(L0));   // of one reader of every sequence
#pragma unroll 1
  for (int b = lane + 32; b < p.batch; b += 32) per += cost(block_tiles(length(b)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) per += __shfl_xor_sync(0xffffffffu, per, o);
  if (per == 0) return;
  // the whole cost; with less of it than a tile for each CTA the last CTAs have nothing, so that
  // no CTA lies between two tiles
  const I total = per * p.readers - kBCostUnit, G = min(static_cast<I>(gridDim.x), total / kBCostTile), g = blockIdx.x;
  if (g >= G) return;
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
      const int T = block_tiles(L);
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
        add_segment(p, seg, nseg + __popc(has & ((1u << lane) - 1u)), c0 + lane, r, L, lo, hi,
                    static_cast<long long>(r) * p.batch + c0 + lane + blockIdx.x);
        tiles += hi - lo;
      }
      nseg += __popc(has);
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
}
// (the wide form, for problems of millions of tiles, out of the way of the usual one's code)
__device__ __noinline__ void cost_segments_wide(const BlockDecodeParams& p, int cap, BlockSegment* seg, int& nseg, int& tiles,
                                                bool& bad) {
  cost_segments<long long>(p, cap, seg, nseg, tiles, bad);
}

__device__ __forceinline__ void store_bf16x4(__nv_bfloat16* to, const float (&a)[4], float scale) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a[0] * scale, a[1] * scale), hi = __floats2bfloat162_rn(a[2] * scale, a[3] * scale);
  *reinterpret_cast<uint2*>(to) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// A unit's CTAs: only its own sequence's length is read.
__device__ __forceinline__ void unit_segment(const BlockDecodeParams& p, int cap, BlockSegment* seg, int& nseg, int& tiles,
                                             bool& bad) {
  if ((threadIdx.x & 31) != 0) return;
  const unsigned c = p.cluster, unit = c == 1 ? blockIdx.x : blockIdx.x / c, i = blockIdx.x - unit * c;
  const int r = unit / p.batch, b = unit - r * p.batch;
  const int L = clamp_len(p.seq_lens[b], cap, bad);
  const unsigned T = block_tiles(L);
  const int lo = c == 1 ? 0 : i * T / c, hi = c == 1 ? T : (i + 1) * T / c;
  add_segment(p, seg, 0, b, r, L, lo, hi, -2);   // (without tiles too: the exchange wants the unit)
  nseg = lo < hi ? 1 : 0;
  tiles = hi - lo;
}

__device__ __forceinline__ void block_segments(const BlockDecodeParams& p, int cap, BlockSegment* seg, int* counts) {
  int nseg = 0, tiles = 0;
  bool bad = false;
  if (p.cluster > 0)
    unit_segment(p, cap, seg, nseg, tiles, bad);
  else if (p.quantum > 0)
    even_segments(p, cap, seg, nseg, tiles, bad);
  else if (p.narrow)
    cost_segments<uint32_t>(p, cap, seg, nseg, tiles, bad);
  else
    cost_segments_wide(p, cap, seg, nseg, tiles, bad);
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

// A role's place in its CTA's run of tiles.
struct BlockTile {
  int s, j, end;           // segment, tile of the sequence, end of the segment
  int b, kvh, L;
  bool again;              // another unit reads the tile's pages after this one
  __device__ __forceinline__ void load(const BlockDecodeParams& p, const BlockSegment* seg, int at) {
    const BlockSegment x = seg[at];
    s = at;
    b = x.b;
    kvh = x.kvh;
    L = x.L;
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
  __device__ __forceinline__ int page_rows(int pg) const { return min(kBPage, L - kBTile * j - kBPage * pg); }
};

// ------------------------------------------------------------------ decode kernel
template <int kDim, int kNR>
__global__ void __launch_bounds__(BlockLayout<kDim, kNR>::kThreads, 1)
mfa_block_decode_kernel(const __grid_constant__ BlockDecodeParams p) {
  using Lay = BlockLayout<kDim, kNR>;
  constexpr int kHalves = Lay::kHalves, kC = Lay::kC, kBoxes = Lay::kBoxes;
  constexpr int kKSlots = Lay::kKSlots, kVSlots = Lay::kVSlots, kPBufs = Lay::kPBufs;
  constexpr int kSoftmaxWarps = 4 * Lay::kWgs;
  static_assert(kC == 8 || kC == 16, "rows of a warpgroup");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint8_t* misc = smem + Lay::kOffMisc;
  BlockSegment* seg = reinterpret_cast<BlockSegment*>(misc);
  float* red = reinterpret_cast<float*>(misc + sizeof(BlockSegment) * kBMaxSeg);   // [warpgroups][4 quarters][kC]
  float* q_inv = red + 256;                                                       // [2 segments][64] what undoes a row's q scaling
  int* row_off = reinterpret_cast<int*>(q_inv + 128);                // [64] element offset of a row's output
  int* row_tok = row_off + 64;                                       // [64] new token of a row within the unit
  float* neg_ref = reinterpret_cast<float*>(row_tok + 64);           // [64] minus the rows' reference maxima
  float* alpha = neg_ref + 64;                                       // [64] what old sums are multiplied by
  float* top_neg = alpha + 64;                                       // [64] minus the highest references so far
  int* look = reinterpret_cast<int*>(top_neg + 64);                  // [64] at a warpgroup's first row: its next tile to look at
  float2* meta = reinterpret_cast<float2*>(look + 64);               // [2 tiles][2 pages][4 blocks] {K, V} scales
  int* ctl = reinterpret_cast<int*>(meta + 16);              // tensor memory, abort flag, segments, tiles
  volatile int* abort_flag = ctl + 1;
  const uint32_t bars = sbase + Lay::kOffMisc + kBMisc - 512;
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  // slots: K's, then V's
  constexpr int kFull = 0, kEmpty = Lay::kSlots, kSFull = 2 * Lay::kSlots, kSEmpty = kSFull + 2, kPFull = kSEmpty + 2,
                kPvDone = kPFull + 2, kQReady = kPvDone + 2, kOEmpty = kQReady + 1, kQEmpty = kOEmpty + 1,
                kDrain = kQEmpty + 1, kBars = kDrain + 1;
  static_assert(kBars * 8 <= 512, "barrier area");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = p.max_pages * kBPage;

  if (warp == 0) {
    for (int i = lane; i < kBars; i += 32) {
      // arrivals a phase: one for each page of a slot; the QK issuer's and the scale warp's for a
      // tile's scores; one for each softmax warp; one for each MMA issuer (drain); else one
      const bool by_warps = (i >= kSEmpty && i < kPvDone) || i == kQReady || i == kOEmpty;
      const bool by_two = i < kEmpty || i == kSFull || i == kSFull + 1 || i == kDrain;
      mbar_init(bar(i), by_two ? 2 : by_warps ? kSoftmaxWarps : 1);
    }
    if (lane == 0) ctl[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(ctl), Lay::kTmemCols);
    tmem_relinquish();
  }
  if (tid >= 32 * kBSoftmaxWarp0 && tid < 32 * kBSoftmaxWarp0 + kNR) {
    const int row = tid - 32 * kBSoftmaxWarp0, tok = row / p.group;
    row_off[row] = (tok * p.heads + row % p.group) * kDim;
    row_tok[row] = tok;
  }
  if (tid == 32 * kBPvWarp) {
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  // nothing that the preceding kernel may write is read before this; with early metadata the
  // lengths are (the caller says that it does not write them)
  if (!p.early_metadata) grid_dep_wait();
  if (warp == 0) block_segments(p, cap, seg, ctl + 2);
  __syncthreads();
  if (p.early_metadata) grid_dep_wait();
  grid_dep_launch();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(ctl[0]);
  const int nseg = ctl[2], ntiles = ctl[3];

  if (warp == 0) {
    // ---------------- producer: lane i loads box i of each tile of K (i < kBoxes) or of V (half
    // i / 2, page i % 2), each on its own as its slots free
    if (lane < 2 * kBoxes && ntiles > 0) {
      const bool is_v = lane >= kBoxes;
      const int half = (lane % kBoxes) >> 1, pg = lane & 1;
      const int slots = is_v ? kVSlots : kKSlots, slot0 = is_v ? kKSlots : 0;
      const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_last();
      BlockTile it;
      it.load(p, seg, 0);
      auto page_id = [&]() -> int {
        return it.page_rows(pg) > 0 ? p.block_table[static_cast<size_t>(it.b) * p.max_pages + 2 * it.j + pg] : 0;
      };
      int id = page_id();
      int slot = half, phase = 0;   // (half < slots)
      bool ok = true;
      int n = 0;
      // V a round behind K: when every CTA fills its rings at once, the keys that all wait for
      // come first
      for (int round = is_v ? -1 : 0; n < ntiles; ++round) {
        if (round < 0) continue;
        const int rows = it.page_rows(pg);
        int z = id * p.kv_heads + it.kvh;
        if (rows > 0 && (id < 0 || id >= p.num_blocks)) {
          z = -1;   // outside the pool: the whole box reads as zeros
          if (lane < 2) atomicOr(p.status, MFA_DEV_BAD_BLOCK);
        }
        const uint64_t pol = it.again ? again : once;
        if (it.next(p, seg, nseg)) id = page_id();
        ok = block_wait(bar(kEmpty + slot0 + slot), phase ^ 1, abort_flag);
        if (!ok) break;
        const uint32_t fb = bar(kFull + slot0 + slot);
        if (rows <= 0) {
          mbar_arrive(fb);
        } else {
          // the last page's rows land at the end of the box: rows before them are filled with zeros
          mbar_arrive_expect_tx(fb, 8192);
          tma_load_3d_hint(sbase + Lay::kOffRing + (slot0 + slot) * Lay::kSlotBytes + pg * 8192, is_v ? &p.tm_v : &p.tm_k,
                           fb, 128 * half, rows - kBPage, z, pol);
        }
        ++n;
        slot += kHalves;
        if (slot >= slots) {
          slot -= slots;
          phase ^= 1;
        }
      }
      if (!ok) {
        atomicOr(p.status, MFA_DEV_TIMEOUT);
        // let every copy already issued land before the CTA can exit
        for (int u = max(half, (n - kVSlots) * kHalves + half); u < n * kHalves + half; u += kHalves)
          wait_slow(bar(kFull + slot0 + u % slots), (u / slots) & 1, nullptr, kDrainLimitNs);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- QK issuer: S^T(n) = K(n) Q^T, q's hi and lo parts in columns of their own: one
    // MMA for both reads K from shared memory once (as two MMAs into the same columns, four long
    // sequences 41.3 us against 40.5, two new tokens 58.1 against 57.0)
    if (lane == 0 && ntiles > 0) {
      constexpr uint32_t kIdescQK = idesc_e4m3(false, false, 128, 2 * kNR);
      bool ok = true;
      int slot = 0, phase = 0, n = 0;
      for (int s = 0; s < nseg && ok; ++s) {
        const int count = seg[s].hi - seg[s].lo;
        ok = block_wait(bar(kQReady), s & 1, abort_flag);
        for (int i = 0; i < count && ok; ++i, ++n) {
          if (n >= 2) ok = block_wait(bar(kSEmpty + (n & 1)), ((n >> 1) - 1) & 1, abort_flag);
          const uint32_t d = tmem + Lay::kTmemS + 2 * kNR * (n & 1);
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            if (ok) ok = block_wait(bar(kFull + slot), phase, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = smem_desc(sbase + Lay::kOffRing + slot * Lay::kSlotBytes, 16, 1024);
            const uint64_t bd = smem_desc(sbase + Lay::kOffQ + h * (2 * kNR * 128), 16, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)   // 32 elements a step: 2 in the descriptors' 16-byte units
              umma_f8_ss(d, ad + 2 * kk, bd + 2 * kk, kIdescQK, (h | kk) != 0);
            umma_commit(bar(kEmpty + slot));
            if (++slot == kKSlots) {
              slot = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          umma_commit(bar(kSFull + (n & 1)));
          if (i == count - 1) umma_commit(bar(kQEmpty));
        }
      }
      if (!ok) atomicOr(p.status, MFA_DEV_TIMEOUT);
      // every MMA must be complete before tensor memory is released
      umma_commit(bar(kDrain));
      wait_slow(bar(kDrain), 0, nullptr, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp == kBPvWarp) {
    // ---------------- PV issuer: O^T += V^T P^T, the weights' hi and lo parts in columns of their own
    if (lane == 0 && ntiles > 0) {
      constexpr uint32_t kIdescPV = idesc_e4m3(true, true, 128, 2 * kNR);
      bool ok = true;
      int slot = 0, phase = 0, n = 0;
      for (int s = 0; s < nseg && ok; ++s) {
        const int lo = seg[s].lo, hi = seg[s].hi, L = seg[s].L;
        for (int j = lo; j < hi && ok; ++j, ++n) {
          ok = block_wait(bar(kPFull + n % kPBufs), (n / kPBufs) & 1, abort_flag);
          if (ok && j == lo && s > 0) ok = block_wait(bar(kOEmpty), (s - 1) & 1, abort_flag);
          const bool both = L > kBTile * j + kBPage;   // the tile has its second page
          const uint64_t bd = smem_desc(sbase + Lay::kOffP + (n % kPBufs) * 16384, 8192, 1024);
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            if (ok) ok = block_wait(bar(kFull + kKSlots + slot), phase, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = smem_desc(sbase + Lay::kOffRing + (kKSlots + slot) * Lay::kSlotBytes, 8192, 1024);
            const uint32_t d = tmem + Lay::kTmemO + 2 * kNR * h;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)     // 32 tokens a step: 4096 bytes, two steps a page
              if (kk < 2 || both) umma_f8_ss(d, ad + 256 * kk, bd + 256 * kk, kIdescPV, !(j == lo && kk == 0));
            umma_commit(bar(kEmpty + kKSlots + slot));
            if (++slot == kVSlots) {
              slot = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          umma_commit(bar(kPvDone + (n & 1)));
        }
      }
      if (!ok) atomicOr(p.status, MFA_DEV_TIMEOUT);
      umma_commit(bar(kDrain));
      wait_slow(bar(kDrain), 0, nullptr, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp == kBScaleWarp) {
    // ---------------- scales: a tile's up to 2 x 4 block scales of K and of V, ahead of the softmax
    // (lane = V? page, block); page ids two tiles ahead, scales one tile ahead
    const int pg = (lane >> 2) & 1, blk = lane & 3;
    const bool is_v = (lane & 8) != 0, mine = lane < 16 && blk < (kBPage >> p.log_scale);
    const float* src = is_v ? p.v_scale : p.k_scale;
    const float mul = is_v ? kBScaleDown : p.scale_log2;
    if (p.quantum == 0 && p.cluster == 0) {   // where the combine finds a unit's parts
      for (int i = lane; i < nseg; i += 32) {
        const BlockSegment x = seg[i];
        int2* at = p.parts + static_cast<size_t>(x.kvh * p.token_groups + x.tg) * p.batch + x.b;
        if (x.lo == 0) at->x = x.slot;
        if (x.hi == block_tiles(x.L)) at->y = x.slot;
      }
    }
    if (ntiles > 0) {
      BlockTile it;
      it.load(p, seg, 0);
      auto page_id = [&]() -> int {
        return mine && it.page_rows(pg) > 0 ? p.block_table[static_cast<size_t>(it.b) * p.max_pages + 2 * it.j + pg] : -1;
      };
      auto scale_of = [&](int id) -> float {
        if (id < 0 || id >= p.num_blocks) return 0.f;
        return src[((static_cast<size_t>(id) * p.kv_heads + it.kvh) << (6 - p.log_scale)) + blk];
      };
      float value = scale_of(page_id());
      int s = 0;
      bool more = it.next(p, seg, nseg);
      int id = more ? page_id() : -1;
      for (int n = 0; n < ntiles; ++n) {
        float value_next = 0.f;
        if (more) {
          if (it.s != s) {
            s = it.s;
            // the next segment's q, for its conversion to find in L2
            const char* q = reinterpret_cast<const char*>(
                p.q + ((static_cast<size_t>(it.b) * p.tokens + seg[s].tg * p.unit_tokens) * p.heads +
                       static_cast<size_t>(it.kvh) * p.group) * kDim);
            const int lines = p.group * kDim * 2 / 128;
            for (int i = lane; i < lines; i += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + i * 128));
          }
          value_next = scale_of(id);
          more = it.next(p, seg, nseg);
          if (more) id = page_id();
        }
        // the tile's scores and scales are read together: one barrier, one buffer each
        if (n >= 2 && !__all_sync(0xffffffffu, block_wait(bar(kSEmpty + (n & 1)), ((n >> 1) - 1) & 1, abort_flag))) {
          if (lane == 0) atomicOr(p.status, MFA_DEV_TIMEOUT);
          break;
        }
        if (mine) reinterpret_cast<float*>(meta + (n & 1) * 8 + pg * 4 + blk)[is_v ? 1 : 0] = value * mul;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSFull + (n & 1)));
        value = value_next;
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax and epilogue: each warpgroup has the whole tile (lane = token) for
    // its kC rows
    const int sw = warp - kBSoftmaxWarp0, wg = sw >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;          // token row of a tile; element of an O half
    const int pg = row >> 6, ri = row & 63;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const int c0 = wg * kC;                       // this warpgroup's first row
    float* my_red = red + wg * 4 * kC;            // [4 quarters][kC]
    const uint32_t vote_bar = 1 + wg;
    const bool f32 = p.out_f32 != 0;

    // A wait that gives up raises the CTA's abort flag, and its warp waits no more; a warpgroup
    // leaves together, by a vote at its segment's end, so that its barriers stay in step.
    bool aborted = false, stop = false;
    // q of a segment, split into e4m3 hi + lo parts under one power of two a row (split_e4m3):
    // eight lanes a row, four rows a warp at a time; lane i has the 8-element chunks i, i + 8, ...
    auto convert_q = [&](int sidx) {
      constexpr int kChunks = kDim / 64, kRounds = (kNR + 4 * kSoftmaxWarps - 1) / (4 * kSoftmaxWarps);
      const BlockSegment sg = seg[sidx];
      const int valid = p.group * min(p.unit_tokens, p.tokens - sg.tg * p.unit_tokens);
      const __nv_bfloat16* src = p.q + ((static_cast<size_t>(sg.b) * p.tokens + sg.tg * p.unit_tokens) * p.heads +
                                        static_cast<size_t>(sg.kvh) * p.group) * kDim;
      const int r0 = sw * 4 + (lane >> 3), i8 = lane & 7;
      uint4 wr[kRounds][kChunks];
#pragma unroll
      for (int x = 0; x < kRounds; ++x) {
        const int r = r0 + 4 * kSoftmaxWarps * x;
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
          wr[x][k] = r < valid ? __ldg(reinterpret_cast<const uint4*>(src + row_off[r]) + i8 + 8 * k) : make_uint4(0, 0, 0, 0);
      }
      // (the previous segment's last scores are made: its q is read no more)
      if (sidx > 0 && !block_wait(bar(kQEmpty), (sidx - 1) & 1, abort_flag)) aborted = true;
#pragma unroll
      for (int x = 0; x < kRounds; ++x) {
        const int r = r0 + 4 * kSoftmaxWarps * x;
        const uint4(&w)[kChunks] = wr[x];
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          const uint32_t e[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
          for (int x = 0; x < 4; ++x)
            m = fmaxf(m, fmaxf(fabsf(__uint_as_float(e[x] << 16)), fabsf(__uint_as_float(e[x] & 0xFFFF0000u))));
        }
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        int sig = 0;   // the row's largest |q| goes to [64, 128)
        if (m > 0.f) sig = min(126, max(-126, 6 + 127 - static_cast<int>(__float_as_uint(m) >> 23)));
        const float up = __uint_as_float(static_cast<uint32_t>(127 + sig) << 23);
        if (r < kNR) {
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            const uint32_t e[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              split_e4m3(__uint_as_float(e[x] << 16) * up, __uint_as_float(e[x] & 0xFFFF0000u) * up, hi[x], lo[x]);
            const int byte = 8 * (i8 + 8 * k) % 128;   // chunk of a half's 128-byte row
            uint8_t* dst = smem + Lay::kOffQ + (k / 2) * (2 * kNR * 128) + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 8);
            *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
            *reinterpret_cast<uint2*>(dst + kNR * 128) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
          }
          if (i8 == 0) q_inv[(sidx & 1) * 64 + r] = m < INFINITY ? __uint_as_float(static_cast<uint32_t>(127 - sig) << 23) : NAN;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQReady));
    };

    // a tile's scores for this lane's token: q's hi parts' and lo parts' sums
    auto load_scores = [&](uint32_t (&sr)[kC], int buffer) {
      uint32_t lo[kC];
      const uint32_t at = tmem + Lay::kTmemS + 2 * kNR * buffer + c0 + lane_base;
      tmem_ld(at, sr);
      tmem_ld(at + kNR, lo);
      tmem_ld_wait(sr);
      tmem_ld_wait(lo);
#pragma unroll
      for (int i = 0; i < kC; i += 2) {
        float a, b;
        unpack_f32x2(add_f32x2(pack_f32x2(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])),
                               pack_f32x2(__uint_as_float(lo[i]), __uint_as_float(lo[i + 1]))), a, b);
        sr[i] = __float_as_uint(a);
        sr[i + 1] = __float_as_uint(b);
      }
    };

    if (ntiles > 0) convert_q(0);
    int n = 0;
    for (int s = 0; s < nseg && !stop; ++s) {
      const BlockSegment sg = seg[s];
      const int L = sg.L;
      const int seen0 = L - (p.tokens - 1) + sg.tg * p.unit_tokens;   // tokens that the unit's first row sees
      uint64_t l2[kC / 2] = {};   // row sums over this lane's tokens, pairs of rows
      if (row < kC) neg_ref[c0 + row] = top_neg[c0 + row] = INFINITY;
      if (row == 0) look[c0] = n;
      if (!block_wait(bar(kQReady), s & 1, abort_flag)) aborted = true;
      named_bar_sync(vote_bar, 128);
      const ulonglong2* w4 = reinterpret_cast<const ulonglong2*>(q_inv + (s & 1) * 64 + c0);
      const ulonglong2* m4 = reinterpret_cast<const ulonglong2*>(neg_ref + c0);
      for (int j = sg.lo; j < sg.hi; ++j, ++n) {
        const int pr = ri - (kBPage - min(kBPage, L - kBTile * j - kBPage * pg));   // page row of this lane's box row
        const int t = pr >= 0 ? kBTile * j + kBPage * pg + pr : INT_MAX;            // and its token
        if (!block_wait(bar(kSFull + (n & 1)), (n >> 1) & 1, abort_flag)) aborted = true;
        tc_fence_after();
        const float2 sc = pr >= 0 ? meta[(n & 1) * 8 + pg * 4 + (pr >> p.log_scale)] : make_float2(0.f, 0.f);
        const uint64_t a2 = pack_f32x2(sc.x, sc.x);
        const float e = static_cast<float>(min(max(static_cast<int>(__float_as_uint(sc.y) >> 23) - 127, kBEMin), kBEMax));
        uint64_t x2[kC / 2];
        bool o_ready = false;   // the previous tile's PV is known to be complete
        for (bool settled = false, first = j == sg.lo;; settled = true) {
          // scores relative to the reference, in powers of two; -inf for what a row does not see
          // (a segment's first tile has no reference yet)
          if (settled || !first) {
            uint32_t sr[kC];
            load_scores(sr, n & 1);
#pragma unroll
            for (int i = 0; i < kC / 2; i += 2) {
              const ulonglong2 w = w4[i / 2], m = m4[i / 2];
              x2[i] = fma_f32x2(pack_f32x2(__uint_as_float(sr[2 * i]), __uint_as_float(sr[2 * i + 1])), mul_f32x2(a2, w.x), m.x);
              x2[i + 1] = fma_f32x2(pack_f32x2(__uint_as_float(sr[2 * i + 2]), __uint_as_float(sr[2 * i + 3])), mul_f32x2(a2, w.y), m.y);
            }
          }
          if (kBTile * (j + 1) <= seen0) {
            // every row sees the whole tile
          } else if (p.unit_tokens == 1) {
            if (t >= seen0) {
#pragma unroll
              for (int i = 0; i < kC / 2; ++i) x2[i] = pack_f32x2(-INFINITY, -INFINITY);
            }
          } else {
#pragma unroll
            for (int i = 0; i < kC / 2; ++i) {
              float lo, hi;
              unpack_f32x2(x2[i], lo, hi);
              const int2 tok = *reinterpret_cast<const int2*>(row_tok + c0 + 2 * i);
              x2[i] = pack_f32x2(t < seen0 + tok.x ? lo : -INFINITY, t < seen0 + tok.y ? hi : -INFINITY);
            }
          }
          if (settled) break;
          if (!first) {
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < kC / 2; ++i) {
              float lo, hi;
              unpack_f32x2(x2[i], lo, hi);
              top = fmaxf(top, fmaxf(lo, hi));
            }
            if (!named_bar_or(vote_bar, 128, look[c0] == n || top + e > kBThreshold)) break;
          }
          // ---- new references, from each row's largest x + e in this tile; the sums and O move to
          // them (by powers of two).  Rare after a segment's first two tiles.
          {
            uint32_t sr[kC];
            float y[kC];
            load_scores(sr, n & 1);
#pragma unroll
            for (int i = 0; i < kC; i += 4) {
              const float4 w = *reinterpret_cast<const float4*>(q_inv + (s & 1) * 64 + c0 + i);
              y[i] = fmaf(__uint_as_float(sr[i]), sc.x * w.x, e);
              y[i + 1] = fmaf(__uint_as_float(sr[i + 1]), sc.x * w.y, e);
              y[i + 2] = fmaf(__uint_as_float(sr[i + 2]), sc.x * w.z, e);
              y[i + 3] = fmaf(__uint_as_float(sr[i + 3]), sc.x * w.w, e);
            }
            if (kBTile * (j + 1) > seen0) {
#pragma unroll
              for (int i = 0; i < kC; ++i) y[i] = t < seen0 + row_tok[c0 + i] ? y[i] : -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < kC; ++i) y[i] = warp_max(y[i]);
            if (lane == 0) {
#pragma unroll
              for (int i = 0; i < kC; i += 4)
                *reinterpret_cast<float4*>(my_red + quarter * kC + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            }
          }
          named_bar_sync(vote_bar, 128);
          if (row < kC) {
            const float a = my_red[row], b = my_red[kC + row], c = my_red[2 * kC + row], d = my_red[3 * kC + row];
            const float ab = fmaxf(a, b), cd = fmaxf(c, d), m = fmaxf(ab, cd);
            const float second = fmaxf(fminf(ab, cd), ab > cd ? fminf(a, b) : fminf(c, d)), least = fminf(fminf(a, b), fminf(c, d));
            const float over = m - fminf(second, least + 3.f);   // how far few tokens outweigh the others
            const float was = neg_ref[c0 + row], top = top_neg[c0 + row];
            const float to = fminf(fmaxf(floorf(over) - 2.f, kBRoom), kBRoomFew) - floorf(m);
            const int at = look[c0];
            float now = fminf(was, to);   // (as it was where the row sees nothing of the tile, or m is NaN)
            if (at == n && m + was < kBLow && m > -INFINITY) now = fminf(to, top + kBDepth);
            const bool soon = __any_sync((1u << kC) - 1, over >= kBOver && m + was > kBNear);
            if (row == 0 && (soon || at == n)) look[c0] = n + (!soon ? kBLookEvery : at - n <= kBLookEvery - 7 ? 1 : 8);   // (8: the last look is near)
            neg_ref[c0 + row] = now;
            top_neg[c0 + row] = fminf(top, now);
            alpha[c0 + row] = now < INFINITY ? ex2_approx(now - was) : 1.f;
          }
          named_bar_sync(vote_bar, 128);
#pragma unroll
          for (int i = 0; i < kC / 2; i += 2) {
            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(alpha + c0 + 2 * i);
            l2[i] = mul_f32x2(l2[i], f.x);
            l2[i + 1] = mul_f32x2(l2[i + 1], f.y);
          }
          if (j > sg.lo) {   // O holds something
            if (!block_wait(bar(kPvDone + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort_flag)) aborted = true;
            o_ready = true;
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < 2 * kHalves; ++h) {   // halves x (hi, lo)
              uint32_t o[kC];
              const uint32_t at = tmem + Lay::kTmemO + kNR * h + c0 + lane_base;
              tmem_ld(at, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int i = 0; i < kC; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(alpha + c0 + i);
                o[i] = __float_as_uint(__uint_as_float(o[i]) * f.x);
                o[i + 1] = __float_as_uint(__uint_as_float(o[i + 1]) * f.y);
                o[i + 2] = __float_as_uint(__uint_as_float(o[i + 2]) * f.z);
                o[i + 3] = __float_as_uint(__uint_as_float(o[i + 3]) * f.w);
              }
              tmem_st(at, o);
            }
            tmem_st_wait();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSEmpty + (n & 1)));
        // p = 2^x and its sums in fp32; P = p s_v rounded to f16 (2^-12) and split into e4m3 parts
        // P = hi + lo / 32: each part keeps four bits, and the lo part's own accumulator lets it be 32
        // times larger (see kBThreshold)
        const uint64_t v2 = pack_f32x2(sc.y, sc.y);
        const __half2 part = __half2half2(__float2half_rn(kBPart));
        uint32_t hi[kC / 4], lo[kC / 4];
#pragma unroll
        for (int i = 0; i < kC / 4; ++i) {
          uint32_t pu[2], back[2], rest[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x0, x1;
            unpack_f32x2(x2[2 * i + k], x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            l2[2 * i + k] = add_f32x2(l2[2 * i + k], pack_f32x2(p0, p1));
            float w0, w1;
            unpack_f32x2(mul_f32x2(pack_f32x2(p0, p1), v2), w0, w1);
            const __half2 v = __floats2half2_rn(w0, w1);
            pu[k] = *reinterpret_cast<const uint32_t*>(&v);
          }
          hi[i] = cvt_e4m3x4(pu[0], pu[1]);
          cvt_f16x4(hi[i], back[0], back[1]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const __half2 v = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&pu[k]), *reinterpret_cast<const __half2*>(&back[k])), part);
            rest[k] = *reinterpret_cast<const uint32_t*>(&v);
          }
          lo[i] = cvt_e4m3x4(rest[0], rest[1]);
        }
        // the P buffer is free once the PV that read it is complete
        if (n >= kPBufs && !(kPBufs == 1 && o_ready))
          if (!block_wait(bar(kPvDone + ((n - kPBufs) & 1)), ((n - kPBufs) >> 1) & 1, abort_flag)) aborted = true;
        {
          uint8_t* dst = smem + Lay::kOffP + (n % kPBufs) * 16384 + row * 128;
          const int sx = row & 7;
          if constexpr (kC >= 16) {
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) {
              *reinterpret_cast<uint4*>(dst + (((c0 / 16 + k) ^ sx) << 4)) =
                  make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
              *reinterpret_cast<uint4*>(dst + ((((kNR + c0) / 16 + k) ^ sx) << 4)) =
                  make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
            }
          } else {
            *reinterpret_cast<uint2*>(dst + (sx << 4) + c0) = make_uint2(hi[0], hi[1]);          // chunk 0: rows 0..15
            *reinterpret_cast<uint2*>(dst + ((1 ^ sx) << 4) + c0) = make_uint2(lo[0], lo[1]);    // chunk 1: lo parts
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull + n % kPBufs));
      }
      if (s + 1 < nseg) convert_q(s + 1);

      // ---------------- the segment's result
      {
        float l[kC];
#pragma unroll
        for (int i = 0; i < kC / 2; ++i) unpack_f32x2(l2[i], l[2 * i], l[2 * i + 1]);
        const float lsum = reduce_columns<kC>(l);
        named_bar_sync(vote_bar, 128);   // (the scratch may still be read from the last new reference)
        if (lane % (32 / kC) == 0) my_red[quarter * kC + lane / (32 / kC)] = lsum;
        if (!block_wait(bar(kPvDone + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort_flag)) aborted = true;
        if (named_bar_or(vote_bar, 128, aborted || *abort_flag)) {
          stop = true;
          break;
        }
        tc_fence_after();
        const int slot = sg.slot;
        const bool whole = slot == -1;
        const int valid = p.group * min(p.unit_tokens, p.tokens - sg.tg * p.unit_tokens);
        const size_t first = (static_cast<size_t>(sg.b) * p.tokens + sg.tg * p.unit_tokens) * p.heads + static_cast<size_t>(sg.kvh) * p.group;
        const int own = min(row, kC - 1);
        const float sum = my_red[own] + my_red[kC + own] + my_red[2 * kC + own] + my_red[3 * kC + own];
        if (row < kC) alpha[c0 + row] = sum == 0.f ? 0.f : kBScaleUp / sum;   // (a row that sees nothing: zeros)
        named_bar_sync(vote_bar, 128);
        // A partial result keeps the accumulator's order, a thread's eight rows of one element side
        // by side; bf16 outputs go out as pairs of elements, a lane and its neighbour exchanging a
        // row each.
        float* part = p.part_o + static_cast<size_t>(max(slot, 0)) * p.rows8 * kDim;
        float* ring = reinterpret_cast<float*>(smem + Lay::kOffRing);   // (free: this was the CTA's only segment, if slot is -2)
        uint8_t* out = static_cast<uint8_t*>(p.out) + first * kDim * (f32 ? 4 : 2);
#pragma unroll 1
        for (int h = 0; h < kHalves; ++h) {
          uint32_t o[kC], o2[kC];
          const uint32_t at = tmem + Lay::kTmemO + 2 * kNR * h + c0 + lane_base;
          tmem_ld(at, o);
          tmem_ld(at + kNR, o2);
          tmem_ld_wait(o);
          tmem_ld_wait(o2);
          if (h == kHalves - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kOEmpty));   // the next segment may accumulate
          }
          const int col = 128 * h + row;
          float v[kC];
#pragma unroll
          for (int i = 0; i < kC; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(alpha + c0 + i);
            v[i] = fmaf(__uint_as_float(o2[i]), 1.f / kBPart, __uint_as_float(o[i])) * f.x;
            v[i + 1] = fmaf(__uint_as_float(o2[i + 1]), 1.f / kBPart, __uint_as_float(o[i + 1])) * f.y;
            v[i + 2] = fmaf(__uint_as_float(o2[i + 2]), 1.f / kBPart, __uint_as_float(o[i + 2])) * f.z;
            v[i + 3] = fmaf(__uint_as_float(o2[i + 3]), 1.f / kBPart, __uint_as_float(o[i + 3])) * f.w;
          }
          if (slot == -2) {
#pragma unroll
            for (int i = 0; i < kC; ++i) ring[(c0 + i) * kDim + col] = v[i];
          } else if (!whole) {
#pragma unroll
            for (int i = 0; i < kC; i += 8) {
              const float v8[8] = {v[i], v[i + 1], v[i + 2], v[i + 3], v[i + 4], v[i + 5], v[i + 6], v[i + 7]};
              if (c0 + i < p.rows8) st_global_f32x8(part + (static_cast<size_t>((c0 + i) >> 3) * kDim + col) * 8, v8);
            }
          } else if (f32) {
#pragma unroll
            for (int i = 0; i < kC; ++i)
              if (c0 + i < valid) reinterpret_cast<float*>(out)[row_off[c0 + i] + col] = v[i];
          } else {
            const bool odd = lane & 1;
#pragma unroll
            for (int i = 0; i < kC; i += 2) {
              const float got = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 1);
              const __nv_bfloat162 pair = odd ? __floats2bfloat162_rn(got, v[i + 1]) : __floats2bfloat162_rn(v[i], got);
              const int r = c0 + i + (odd ? 1 : 0);
              if (r < valid) *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(out) + row_off[r] + (col & ~1)) = pair;
            }
          }
        }
        if (row < kC && c0 + row < valid) {
          // (the sum's exponent joins the reference first: their logarithms alone would cancel)
          const int k = min(static_cast<int>(__float_as_uint(sum) >> 23), 253) - 127;
          const float v = sum == 0.f ? -INFINITY
                                     : fmaf(static_cast<float>(k) - neg_ref[c0 + row], 0.6931471805599453f,
                                            logf(sum * __uint_as_float(static_cast<uint32_t>(127 - k) << 23)));
          if (slot == -2)
            ring[kNR * kDim + c0 + row] = v;
          else if (!whole)
            p.part_lse[static_cast<size_t>(slot) * p.rows8 + c0 + row] = v;
          else if (p.lse != nullptr)
            p.lse[first + row_off[c0 + row] / kDim] = v;
        }
      }
    }
    // sequences without tokens: zeros and -inf, in turn over the CTAs
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
      bool dummy = false;
      if (clamp_len(p.seq_lens[b], cap, dummy) != 0) continue;
      const size_t n = static_cast<size_t>(p.tokens) * p.heads, at = static_cast<size_t>(b) * n;
      const size_t chunks = n * kDim * (f32 ? 4 : 2) / 16;
      uint4* o = static_cast<uint4*>(p.out) + at * kDim * (f32 ? 4 : 2) / 16;
      for (size_t i = tid - 32 * kBSoftmaxWarp0; i < chunks; i += 32 * kSoftmaxWarps) o[i] = make_uint4(0, 0, 0, 0);
      if (p.lse != nullptr)
        for (size_t i = tid - 32 * kBSoftmaxWarp0; i < n; i += 32 * kSoftmaxWarps) p.lse[at + i] = -INFINITY;
    }
    if (stop && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.status, MFA_DEV_TIMEOUT);
    }
  }
  __syncthreads();
  if (p.cluster > 1) {
    // ---------------- the cluster's exchange, in place of partial results in the workspace and a
    // second kernel (32 sequences of 4096, four CTAs each: 23.3 us against 26.4): CTA i takes rows
    // i, i + c, ... of the unit and adds up
    // the parts, in order, as they lie in the CTAs' rings.  (Every CTA comes here, whatever its roles
    // have met, and both barriers are the hardware's.)
    const unsigned c = p.cluster, rank = blockIdx.x % c;
    const BlockSegment sg = seg[0];
    const unsigned T = block_tiles(sg.L);
    const unsigned parts = __ballot_sync(0xffffffffu, lane < c && lane * T / c < (lane + 1) * T / c);   // those with tiles
    cluster_sync();
    if (T > 1 && warp >= kBSoftmaxWarp0) {
      const int valid = p.group * min(p.unit_tokens, p.tokens - sg.tg * p.unit_tokens);
      const size_t first = (static_cast<size_t>(sg.b) * p.tokens + sg.tg * p.unit_tokens) * p.heads + static_cast<size_t>(sg.kvh) * p.group;
      constexpr int kQuads = kDim / 4;
      const int t = tid - 32 * kBSoftmaxWarp0, el = t % kQuads * 4;
      uint32_t from[8];
#pragma unroll
      for (unsigned k = 0; k < 8; ++k) from[k] = cluster_map(sbase + Lay::kOffRing, min(k, c - 1));
#pragma unroll 1
      for (int row = t / kQuads * c + rank; row < valid; row += 32 * kSoftmaxWarps / kQuads * c) {
        float l[8], o[8][4], top = -INFINITY, sum = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          l[k] = -INFINITY;
          if (parts >> k & 1) {
            l[k] = ld_cluster_f32(from[k] + (kNR * kDim + row) * 4);
            ld_cluster_f32x4(from[k] + (row * kDim + el) * 4, o[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, l[k]);
        const float ref = top == -INFINITY ? 0.f : top;   // (a row that sees nothing)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (parts >> k & 1) {
            const float w = ex2_approx((l[k] - ref) * 1.4426950408889634f);
            sum += w;
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = fmaf(w, o[k][i], a[i]);
          }
        const float back = sum == 0.f ? 0.f : 1.f / sum;
        const size_t to = first + (p.unit_tokens == 1 ? row : row / p.group * p.heads + row % p.group);
        if (p.out_f32)
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to * kDim + el) =
              make_float4(a[0] * back, a[1] * back, a[2] * back, a[3] * back);
        else
          store_bf16x4(static_cast<__nv_bfloat16*>(p.out) + to * kDim + el, a, back);
        if (el == 0 && p.lse != nullptr) p.lse[to] = sum == 0.f ? -INFINITY : top + logf(sum);
      }
    }
    cluster_sync();   // (the rings may be read until here: a CTA's reads come before its arrival)
  }
  if (warp == 1) tmem_dealloc(tmem, Lay::kTmemCols);
}

// ------------------------------------------------------------------ combine kernel
//
// Units in parts: out = sum_s w_s O_s with w_s = e^(lse_s - lse), lse = ln sum_s e^lse_s.  First a
// warp a row makes the weights, while the first parts' values are on their way; then a thread has
// eight rows of one element, as the parts hold them: one 32-byte load and eight multiply-adds a part.
// kTeams teams of threads share the parts, in a fixed order, each CTA with 256 / kTeams elements of
// eight rows (kTeams = 1, d = 128: all elements of sixteen).  Latency bounds it: four dependent
// steps after the decode kernel's end, 2 to 5 us; with a running maximum in every thread instead of
// weights made once a row it took 64.2 us for the two-token batch against 60.5.
constexpr int kBHeld = 5;               // a lane's parts whose lse stays in a register
constexpr int kBChunk = 32 * kBHeld;    // parts whose weights are held at a time

template <int kDim, int kTeams>
__global__ void __launch_bounds__(kBCombineThreads, 3) mfa_block_combine_kernel(const __grid_constant__ BlockDecodeParams p) {
  constexpr int kSlice = kDim < kBCombineThreads / kTeams ? kDim : kBCombineThreads / kTeams;   // elements of a CTA
  constexpr int kOcts = kBCombineThreads / (kTeams * kSlice);                                   // groups of eight rows
  __shared__ float so[kTeams > 1 ? kTeams - 1 : 1][kTeams > 1 ? kSlice : 1][9];   // (odd pitch: no bank conflicts)
  __shared__ __align__(16) float sw[kBChunk][8 * kOcts];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int team = tid / (kSlice * kOcts), oct = tid / kSlice % kOcts, el = blockIdx.z * kSlice + tid % kSlice;
  const int pos = blockIdx.x, b = pos % p.batch, r = pos / p.batch;
  const int row0 = blockIdx.y * kOcts * 8;   // the CTA's first row
  // The parts, slots at.x .. at.y.  The decode kernel lets this one start once its own wait for
  // what came before is over, so the lengths are final; what the decode writes is read after this
  // kernel's wait.
  int2 at = make_int2(0, -1);
  const int cap = p.max_pages * kBPage;
  bool bad = false;
  const int T = block_tiles(clamp_len(p.seq_lens[b], cap, bad));
  if (p.quantum > 0) {
    int quantum = p.quantum;
#pragma unroll 1
    while (true) {
      int before = 0;        // parts of the sequences before b, in every warp
      long long all = 0;     // and of all
#pragma unroll 1
      for (int i = lane; i < p.batch; i += 32) {
        const int n = even_parts(block_tiles(clamp_len(p.seq_lens[i], cap, bad)), quantum);
        all += n;
        before += i < b ? n : 0;
      }
      const long long low = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(all & 0xFFFFF));
      all = low + (static_cast<long long>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(all >> 20))) << 20);
      if (all * p.readers <= p.num_partials) {
        const int n = even_parts(T, quantum), first_part = __reduce_add_sync(0xffffffffu, before) * p.readers + r * n;
        if (n > 1) at = make_int2(first_part, first_part + n - 1);
        break;
      }
      quantum = wider_quantum(p, cap);
    }
  }
  const int kvh = r / p.token_groups, tg = r - kvh * p.token_groups;
  const int valid = p.group * min(p.unit_tokens, p.tokens - tg * p.unit_tokens);
  const size_t first = (static_cast<size_t>(b) * p.tokens + tg * p.unit_tokens) * p.heads + static_cast<size_t>(kvh) * p.group;
  grid_dep_wait();
  grid_dep_launch();
  if (p.quantum == 0 && T > 0) at = p.parts[pos];
  // one part, the output itself; no tokens; or past the plan, as the decode reports
  if (at.y <= at.x || at.x < 0 || at.y >= p.num_partials) return;
  // the first parts' values come while the weights are made
  constexpr int kRound = kTeams > 1 ? 4 : 2;
  const bool rows = row0 + 8 * oct < p.rows8;
  const float* src = p.part_o + (static_cast<size_t>(row0 / 8 + (rows ? oct : 0)) * kDim + el) * 8;
  const size_t pitch = static_cast<size_t>(p.rows8) * kDim;
  float o[kRound][8];
  auto fetch = [&](int k) {   // parts k, k + kTeams, ... of at.x .. (past the last: weight 0 or not taken)
#pragma unroll
    for (int x = 0; x < kRound; ++x) ld_global_f32x8(src + static_cast<size_t>(min(at.x + k + x * kTeams, at.y)) * pitch, o[x]);
  };
  fetch(team);
  // a warp's rows: the largest lse and the sum of what is over it; a lane has every 32nd part
  float held[kOcts][kBHeld], top[kOcts], back[kOcts];
#pragma unroll
  for (int x = 0; x < kOcts; ++x) {
    const int row = row0 + warp + 8 * x;
    const float* lse = p.part_lse + min(row, p.rows8 - 1);
    auto of = [&](int k) { return lse[static_cast<size_t>(k) * p.rows8]; };
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int j = 0; j < kBHeld; ++j) {
      const int k = at.x + lane + 32 * j;
      held[x][j] = k <= at.y && row < valid ? of(k) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < kBHeld; ++j) m = fmaxf(m, held[x][j]);
#pragma unroll 1
    for (int k = at.x + kBChunk + lane; k <= at.y; k += 32) m = fmaxf(m, of(k));
#pragma unroll 1
    for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    top[x] = m == -INFINITY ? 0.f : m;   // (a row that sees nothing)
#pragma unroll
    for (int j = 0; j < kBHeld; ++j) {
      held[x][j] = ex2_approx((held[x][j] - top[x]) * 1.4426950408889634f);
      s += held[x][j];
    }
#pragma unroll 1
    for (int k = at.x + kBChunk + lane; k <= at.y; k += 32) s += ex2_approx((of(k) - top[x]) * 1.4426950408889634f);
#pragma unroll 1
    for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0 && blockIdx.z == 0 && p.lse != nullptr && row < valid)
      p.lse[first + (p.unit_tokens == 1 ? row : row / p.group * p.heads + row % p.group)] = s == 0.f ? -INFINITY : m + logf(s);
    back[x] = s == 0.f ? 0.f : 1.f / s;
#pragma unroll
    for (int j = 0; j < kBHeld; ++j) sw[lane + 32 * j][warp + 8 * x] = held[x][j] * back[x];
  }
  __syncthreads();
  float acc[8] = {};
#pragma unroll 1
  for (int k0 = 0;;) {
    const int n = min(kBChunk, at.y + 1 - at.x - k0);
#pragma unroll 1
    for (int k = team; k < n;) {
#pragma unroll
      for (int x = 0; x < kRound; ++x) {
        if (k + x * kTeams >= n) break;
        const float4* w = reinterpret_cast<const float4*>(&sw[k + x * kTeams][8 * oct]);
        const float4 w0 = w[0], w1 = w[1];
        acc[0] = fmaf(w0.x, o[x][0], acc[0]);
        acc[1] = fmaf(w0.y, o[x][1], acc[1]);
        acc[2] = fmaf(w0.z, o[x][2], acc[2]);
        acc[3] = fmaf(w0.w, o[x][3], acc[3]);
        acc[4] = fmaf(w1.x, o[x][4], acc[4]);
        acc[5] = fmaf(w1.y, o[x][5], acc[5]);
        acc[6] = fmaf(w1.z, o[x][6], acc[6]);
        acc[7] = fmaf(w1.w, o[x][7], acc[7]);
      }
      k += kRound * kTeams;
      if (k < n) fetch(k0 + k);
    }
    k0 += kBChunk;
    if (at.x + k0 > at.y) break;
    fetch(k0 + team);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kOcts; ++x) {
      const int row = row0 + warp + 8 * x;
#pragma unroll 1
      for (int k = lane; k < min(kBChunk, at.y + 1 - at.x - k0); k += 32)
        sw[k][warp + 8 * x] = row >= valid ? 0.f
                              : ex2_approx((p.part_lse[static_cast<size_t>(at.x + k0 + k) * p.rows8 + row] - top[x]) * 1.4426950408889634f) * back[x];
    }
    __syncthreads();
  }
  if constexpr (kTeams > 1) {
    if (team > 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) so[team - 1][tid % kSlice][i] = acc[i];
    }
    __syncthreads();
    if (team > 0) return;
#pragma unroll 1
    for (int k = 0; k < kTeams - 1; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += so[k][tid % kSlice][i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 8 * oct + i;
    if (row >= valid) break;
    const size_t to = (first + (p.unit_tokens == 1 ? row : row / p.group * p.heads + row % p.group)) * kDim + el;
    if (p.out_f32)
      static_cast<float*>(p.out)[to] = acc[i];
    else
      static_cast<__nv_bfloat16*>(p.out)[to] = __float2bfloat16_rn(acc[i]);
  }
}

// ------------------------------------------------------------------ host side

using BlockDecodeFn = void (*)(BlockDecodeParams);
using BlockCombineFn = void (*)(BlockDecodeParams);

// The instance of a problem: width and rows padded to 16, 32 or 64.
static int block_instance(const mfa_problem* pr, const BlockShape& sh) {
  return (pr->head_dim == 256 ? 3 : 0) + (sh.rows <= 16 ? 0 : sh.rows <= 32 ? 1 : 2);
}
static BlockDecodeFn block_kernel_of(int i) {
  constexpr BlockDecodeFn k[6] = {mfa_block_decode_kernel<128, 16>, mfa_block_decode_kernel<128, 32>,
                                  mfa_block_decode_kernel<128, 64>, mfa_block_decode_kernel<256, 16>,
                                  mfa_block_decode_kernel<256, 32>, mfa_block_decode_kernel<256, 64>};
  return k[i];
}

static int block_threads(int i) {
  constexpr int t[3] = {BlockLayout<128, 16>::kThreads, BlockLayout<128, 32>::kThreads, BlockLayout<128, 64>::kThreads};
  return t[i % 3];
}

// cudaFuncSetAttribute for an instance's dynamic shared memory, once per device and instance.
static mfa_status ensure_block_smem(int i) {
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> done[6][kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const bool cacheable = dev >= 0 && dev < kMaxDevices;
  if (cacheable && done[i][dev].load(std::memory_order_acquire)) return MFA_OK;
  e = cudaFuncSetAttribute(block_kernel_of(i), cudaFuncAttributeMaxDynamicSharedMemorySize, kBSmem + 1024);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  if (cacheable) done[i][dev].store(true, std::memory_order_release);
  return MFA_OK;
}

}  // namespace mfa

using namespace mfa;

extern "C" mfa_status mfa_block_decode_plan(const mfa_problem* pr, int32_t scale_tokens, const int32_t* host_seq_lens,
                                            int32_t max_seq_len, int32_t num_sms, int32_t force_ctas, uint32_t flags,
                                            mfa_plan* plan) {
  const mfa_status st = check_block_problem(pr, scale_tokens);
  if (st != MFA_OK) return st;
  if (plan == nullptr || force_ctas < 0) return MFA_ERR_INVALID_ARG;
  if (flags & ~(MFA_PLAN_CHECK | MFA_PLAN_EARLY_METADATA)) return MFA_ERR_INVALID_ARG;
  const long long cap = static_cast<long long>(pr->max_pages_per_seq) * kBPage;
  const BlockShape sh = block_shape(pr);
  long long tiles = 0, nonempty = 0, longest = 0;   // tiles of one reader of each sequence
  if (host_seq_lens != nullptr) {
    for (int b = 0; b < pr->batch; ++b) {
      if (host_seq_lens[b] < 0 || host_seq_lens[b] > cap) return MFA_ERR_INVALID_ARG;
      tiles += (host_seq_lens[b] + kBTile - 1) / kBTile;
      nonempty += host_seq_lens[b] > 0;
      longest = std::max<long long>(longest, (host_seq_lens[b] + kBTile - 1) / kBTile);
    }
  } else {
    if (max_seq_len < 0 || max_seq_len > cap) return MFA_ERR_INVALID_ARG;
    tiles = static_cast<long long>(pr->batch) * ((max_seq_len + kBTile - 1) / kBTile);
    nonempty = max_seq_len > 0 ? pr->batch : 0;
    longest = (max_seq_len + kBTile - 1) / kBTile;
  }
  if (num_sms <= 0) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
  }
  const long long W = tiles * sh.readers, N = nonempty * sh.readers, units = static_cast<long long>(pr->batch) * sh.readers;
  const long long C = kBCostTile * W + kBCostUnit * std::max(N - 1, 0ll);
  const long long most = force_ctas > 0 ? force_ctas : num_sms;
  // Split by cost.  A CTA's share of at most ceil(C / G) holds that over (tile + boundary) whole
  // units and two parts of units.
  const long long share = static_cast<long long>(kBMaxSeg - 2) * (kBCostTile + kBCostUnit);
  const long long least = std::max(1ll, (C + share - 1) / share);
  long long G = std::max(1ll, std::max(std::min(W, most), force_ctas > 0 ? 0ll : least));
  if (force_ctas > 0) G = force_ctas;
  // The way that takes the fewest clocks by these measured figures (bf16 outputs, 152 SMs; other counts
  // of SMs take them over).  us for equal sequences of 64 rows and 4096 tokens, clusters / even / by
  // cost: 1 of them 16.3 / 11.5 / 12.0, 8 17.1 / 15.4 / 16.3, 32 23.2 / 26.4 / 27.6, 48 33.7 / 30.1 /
  // 31.6, 128 51.3 / 55.8 / 60.9; for 16 rows of 128 x 4 heads: 1 9.3 / 8.4 / 9.4, 8 12.7 / 14.2 /
  // 14.9, 12 17.5 / 17.0 / 18.3, 32 26.9 / 28.5 / 30.9; 61 ragged ones with two new tokens 90 / 85 / 63.
  const long long tile = pr->head_dim == 128 && sh.rows <= 32 ? 1400 : 2600;   // a tile
  constexpr long long kExchange = 3000;   // a cluster's exchange
  constexpr long long kSwitch = 18000;    // a second unit's beginning and end in a CTA's range
  auto combine = [&](long long ctas) {    // the combine kernel, launch and all
    return (pr->head_dim == 256 && sh.rows > 32 ? 1500 : 3000) + 25 * ctas;
  };
  long long best = (C + G * kBCostTile - 1) / (G * kBCostTile) * tile + (G > 1 ? combine(G) + kSwitch : 0);
  uint32_t mode = 0;
  int per_cta = static_cast<int>(std::min<long long>((C + G - 1) / G / kBCostTile + 1, std::max(W, 1ll)));
  const bool by_cost = G >= least;
  if (!by_cost) best = LLONG_MAX;
  if (N > 0) {
    // Clusters: 152 SMs hold 76, 46, 36, 28, 23 and 15 clusters of 2, 3, 4, 5, 6 and 8 such CTAs
    for (const int c : {1, 2, 3, 4, 5, 6, 8}) {
      const long long room = c == 1 || force_ctas > 0 ? most : c < 8 ? most * 9 / 10 : most * 3 / 4;
      const long long q = (longest + c - 1) / c, cost = q * tile + (c > 1 ? kExchange : 0);
      if (units * c > room || (c > 1 && q == (longest + c - 2) / (c - 1)) || cost >= best) continue;
      best = cost;
      mode = MFA_PLAN_UNIT_CLUSTERS;
      per_cta = static_cast<int>(std::max(q, 1ll));
      G = units * c;
    }
    // Even split: the smallest quantum whose parts are no more than the CTAs
    if (N <= most) {
      auto parts_at = [&](long long q) {
        long long parts = 0;
        if (host_seq_lens != nullptr)
          for (int b = 0; b < pr->batch; ++b) parts += ((host_seq_lens[b] + kBTile - 1) / kBTile + q - 1) / q;
        else
          parts = static_cast<long long>(pr->batch) * ((longest + q - 1) / q);
        return parts * sh.readers;
      };
      long long lo = 1, hi = std::max(longest, 1ll);   // parts_at(hi) = N fits
      while (lo < hi) {
        const long long mid = (lo + hi) / 2;
        if (parts_at(mid) <= most) hi = mid; else lo = mid + 1;
      }
      if (lo * tile + combine(parts_at(lo)) < best) {
        mode = MFA_PLAN_EVEN_SPLIT;
        per_cta = static_cast<int>(lo);
        G = parts_at(lo);
      }
    }
  }
  if (mode == 0 && !by_cost) return MFA_ERR_INVALID_ARG;   // (a forced grid of too few CTAs)
  const long long partials = units + G - 1;   // (in every mode: a plan for another problem shows)
  if (G > INT_MAX / 2 || partials > INT_MAX / 2 / sh.rows8 || W > INT_MAX) return MFA_ERR_INVALID_ARG;
  std::memset(plan, 0, sizeof(*plan));
  plan->num_ctas = static_cast<int32_t>(G);
  plan->tile_tokens = kBTile;
  plan->max_tiles_per_cta = per_cta;
  plan->num_partials = static_cast<int32_t>(partials);
  plan->batch = pr->batch;
  plan->tokens_per_seq = pr->tokens_per_seq;
  plan->kv_dtype = pr->kv_dtype;
  plan->flags = flags | mode;
  plan->num_sms = num_sms;
  plan->total_tiles = static_cast<uint64_t>(W);
  plan->workspace_bytes = block_workspace_bytes(partials, sh, pr->batch, pr->head_dim);
  return MFA_OK;
}

extern "C" mfa_status mfa_block_decode_run(const mfa_plan* plan, const mfa_problem* pr, int32_t scale_tokens,
                                           const void* q, const void* k_cache, const void* v_cache,
                                           const float* k_scale, const float* v_scale, const int32_t* block_table,
                                           const int32_t* seq_lens, void* out, float* lse, void* workspace,
                                           uint64_t workspace_bytes, void* stream_ptr) {
  const mfa_status st = check_block_problem(pr, scale_tokens);
  if (st != MFA_OK) return st;
  if (plan == nullptr) return MFA_ERR_INVALID_ARG;
  const BlockShape sh = block_shape(pr);
  const long long units = static_cast<long long>(pr->batch) * sh.readers;
  const bool clusters = (plan->flags & MFA_PLAN_UNIT_CLUSTERS) != 0;
  if (plan->batch != pr->batch || plan->kv_dtype != pr->kv_dtype || plan->tokens_per_seq != pr->tokens_per_seq ||
      plan->num_ctas < 1 || (plan->flags & ~(MFA_PLAN_CHECK | MFA_PLAN_EARLY_METADATA | MFA_PLAN_EVEN_SPLIT | MFA_PLAN_UNIT_CLUSTERS)) != 0 ||
      ((plan->flags & MFA_PLAN_EVEN_SPLIT) && (clusters || plan->max_tiles_per_cta < 1)) ||
      (clusters && (units == 0 || plan->num_ctas % units != 0 || plan->num_ctas / units > 8)) ||
      plan->num_partials != units + plan->num_ctas - 1 ||
      plan->workspace_bytes != block_workspace_bytes(plan->num_partials, sh, pr->batch, pr->head_dim))
    return MFA_ERR_INVALID_ARG;
  if (pr->batch == 0) return MFA_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !out || !workspace)
    return MFA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 16) ||
      !aligned(v_scale, 16) || !aligned(out, 16) || !aligned(workspace, 256) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || (lse && !aligned(lse, 4)))
    return MFA_ERR_INVALID_ARG;
  if (workspace_bytes < plan->workspace_bytes) return MFA_ERR_WORKSPACE;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  BlockDecodeParams p;
  std::memset(&p, 0, sizeof(p));
  const void* pools[2] = {k_cache, v_cache};
  CUtensorMap* maps[2] = {&p.tm_k, &p.tm_v};
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return cuda_fail_msg("cuTensorMapEncodeTiled is not available from the driver");
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t d = static_cast<cuuint64_t>(pr->head_dim);
    const cuuint64_t dims[3] = {d, kBPage, static_cast<cuuint64_t>(pr->num_blocks) * pr->num_kv_heads};
    const cuuint64_t strides[2] = {d, d * kBPage};
    const cuuint32_t box[3] = {128, kBPage, 1}, es[3] = {1, 1, 1};
    if (enc(maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pools[i]), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cuda_fail_msg("cuTensorMapEncodeTiled rejected a tensor map");
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = out;
  p.lse = lse;
  p.part_o = reinterpret_cast<float*>(ws + kBWsHeader);
  p.part_lse = reinterpret_cast<float*>(ws + block_lse_offset(plan->num_partials, sh, pr->head_dim));
  p.parts = reinterpret_cast<int2*>(ws + block_parts_offset(plan->num_partials, sh, pr->head_dim));
  p.narrow = static_cast<double>(pr->batch) * sh.readers * plan->num_ctas *
                     (kBCostTile * ((static_cast<double>(pr->max_pages_per_seq) * kBPage + kBTile - 1) / kBTile) + kBCostUnit) <
                 4.0e9;
  p.status = reinterpret_cast<unsigned int*>(ws);
  p.batch = pr->batch;
  p.tokens = pr->tokens_per_seq;
  p.heads = pr->num_q_heads;
  p.kv_heads = pr->num_kv_heads;
  p.group = sh.group;
  p.unit_tokens = sh.unit_tokens;
  p.token_groups = sh.token_groups;
  p.readers = sh.readers;
  p.rows8 = sh.rows8;
  p.num_partials = plan->num_partials;
  p.quantum = (plan->flags & MFA_PLAN_EVEN_SPLIT) ? plan->max_tiles_per_cta : 0;
  p.cluster = clusters ? static_cast<int>(plan->num_ctas / units) : 0;
  p.log_scale = scale_tokens == 64 ? 6 : scale_tokens == 32 ? 5 : 4;
  p.max_pages = pr->max_pages_per_seq;
  p.num_blocks = pr->num_blocks;
  p.scale_log2 = static_cast<float>(static_cast<double>(pr->softmax_scale) * 1.4426950408889634);
  p.out_f32 = pr->out_dtype == MFA_OUT_FP32 ? 1 : 0;
  p.early_metadata = (plan->flags & MFA_PLAN_EARLY_METADATA) ? 1 : 0;
  const bool check = (plan->flags & MFA_PLAN_CHECK) != 0;
  cudaError_t e = cudaSuccess;
  if (check && (e = cudaMemsetAsync(workspace, 0, 4, stream)) != cudaSuccess) return cuda_fail(e, "memset");
  const int inst = block_instance(pr, sh);
  const mfa_status sst = ensure_block_smem(inst);
  if (sst != MFA_OK) return sst;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(plan->num_ctas), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(block_threads(inst)), 1, 1);
  cfg.dynamicSmemBytes = kBSmem + 1024;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(std::max(p.cluster, 1));
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, block_kernel_of(inst), p);
  cfg.numAttrs = 1;
  if (e != cudaSuccess) return cuda_fail(e, "block decode launch");
  if (plan->num_ctas > 1 && !clusters) {
    // Teams that share a unit's parts, and then its elements' slices in CTAs of their own, while the
    // parts and the grid's size pay for them.  Measured at 152 SMs (graph, us), 1 / 2 / 4 / 8 teams;
    // d = 256, 64 rows: 1 unit of 32 parts 16.0 / 12.7 / 11.8 / 11.3, 8 of 16 15.2 / 14.2 / 13.2 / 15.2,
    // 24 of 6 14.4 / 13.0 / 15.9 / 21.4, 48 of 3 14.2 / 16.4 / 21.9 / 32.0; d = 128, 64 rows: the same
    // 15.9 / 11.3 / 10.5 / 9.9, 14.9 / 12.0 / 11.6 / 11.5, 14.2 / 11.5 / 11.5 / 14.5, 14.2 / 12.0 / 15.1 /
    // 20.7; d = 128, 16 rows: 4 of 32 15.1 / 9.6 / 8.5 / 8.4, 8 of 16 11.7 / 8.5 / 8.2 / 8.7, 24 of 6
    // 11.6 / 9.2 / 9.1 / 9.2, 48 of 3 11.3 / 8.9 / 9.1 / 9.6.
    const long long octs = sh.rows8 / 8;
    auto grid_of = [&](int teams) { return units * octs * (pr->head_dim / std::min(pr->head_dim, kBCombineThreads / teams)); };
    int teams = 1;
    if (grid_of(2) <= 512) teams = 2;
    for (const int t : {4, 8})
      if (plan->num_ctas >= 4 * t * units && grid_of(t) <= 256) teams = t;
    const int slice = std::min(pr->head_dim, kBCombineThreads / teams), rows = 8 * (kBCombineThreads / (teams * slice));
    cfg.gridDim = dim3(static_cast<unsigned>(units), static_cast<unsigned>((sh.rows8 + rows - 1) / rows),
                       static_cast<unsigned>(pr->head_dim / slice));
    cfg.blockDim = dim3(kBCombineThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    const BlockCombineFn wide[] = {mfa_block_combine_kernel<256, 1>, mfa_block_combine_kernel<256, 2>,
                                   mfa_block_combine_kernel<256, 4>, mfa_block_combine_kernel<256, 8>};
    const BlockCombineFn narrow[] = {mfa_block_combine_kernel<128, 1>, mfa_block_combine_kernel<128, 2>,
                                     mfa_block_combine_kernel<128, 4>, mfa_block_combine_kernel<128, 8>};
    const int at = teams == 8 ? 3 : teams / 2;
    const BlockCombineFn fn = pr->head_dim == 256 ? wide[at] : narrow[at];
    e = cudaLaunchKernelEx(&cfg, fn, p);
    if (e != cudaSuccess) return cuda_fail(e, "block combine launch");
  }
  if (check) {
    uint32_t word = 0;
    if ((e = cudaMemcpyAsync(&word, workspace, 4, cudaMemcpyDeviceToHost, stream)) != cudaSuccess)
      return cuda_fail(e, "copy");
    if ((e = cudaStreamSynchronize(stream)) != cudaSuccess) return cuda_fail(e, "sync");
    if (word != 0) return MFA_ERR_DEVICE_CHECK;
  }
  return MFA_OK;
}
