// Attention of drafted trees over a block-scaled 8-bit KV cache (GB300, sm_103a).
//
// Node i of a sequence's T drafted tokens, the last T of its L cached ones, sees the tokens before the tree
// and the nodes j whose bit is set in its mask.  With the codes' values k_t, v_t and their blocks' scales
// sk_t, sv_t, over the tokens that it sees:
//     s_t = softmax_scale * sk_t * dot(q, k_t),  out = sum_t e^(s_t) sv_t v_t / sum_t e^(s_t),
//     lse = ln sum_t e^(s_t).
//
// A unit is a sequence, a key/value head and as many nodes as fit 128 rows (nodes x the head's query heads);
// a tile is 128 tokens.  Rows are the MMAs' M = 128:
//   S [rows x 128 tokens] = Q K^T, q split into e4m3 hi + lo parts under one power of two a row, both into
//     the same columns; a token's key scale multiplies its fp32 scores;
//   O [rows x d] += P V, P the weights times the tokens' value scales in two parts, e4m3 hi and e5m2 lo, that
//     lie in tensor memory over the scores that they come from.
// A softmax thread has one row and half of a tile's tokens (a page), so that a row's maximum and sum need no
// shuffles, one exchange with the other half's thread, and a block's scale is one value for all lanes.
//
// P: hi keeps four bits and lo three of what is left: off by 2^-7 of itself at most, where it is at least
// 2^-6; hi's subnormals and lo's go on to 2^-17.  A row's reference R, P = 2^(x + e - R) with x its score and
// e its value scale's logarithm, is set so that a tile's largest P is 2^4.  It rises when one would pass 2^8.75
// (448 is e4m3's largest), and falls when a tile's largest is under 2^-2 (to 24 under its highest at most),
// so that what follows a far larger token keeps its precision; sums and O are fp32 and move by powers of two.
//
// Warps: a producer (TMA boxes of a page, K's and V's rings apart), the issuers of the two MMAs, which take
// turns (the next tile's scores go before a tile's weights, so that the softmax has them in time), one that fetches
// block scales, eight of softmax, and four that keep O: they move it when references do and write the results
// while the softmax begins the next unit.
//
// What bounds it: a tile's products are 128 x 128 x d for S and as many for O, each twice (hi and lo), 2048
// clocks of the tensor cores at d = 256; operands from shared memory are 192 KB of it and the tile's TMA
// writes 64 KB, 2048 clocks at 128 bytes a clock.  A tile takes some 2760 clocks, at 1.93 GHz (read in the kernel, from
// tile 8 to 24 of 32): beside the products the waits between scores, weights and products, of which some 130 are
// the one for the product under the next scores.  At d = 128 a tile takes 2400 clocks: the softmax's chain (scores,
// maxima, their exchange, exponentials, two conversions to eight bits, stores) in two warps a scheduler, which
// issue in half of the clocks; the tensor cores are active for 1024.  A unit's beginning and end take 8 us
// beside its tiles, a boundary inside a CTA's range 4 to 5, parts and their combine 5.
// Measured in a graph of twelve calls over three states: eight trees of 32 nodes over 4096 tokens, 64 heads of 256
// over one, 58.1 us (1.2 PFLOP/s of the products' 1.9 in bf16); seven ragged ones of 61 nodes, 29400 tokens, 103 us;
// 48 of 8 nodes, 64 heads of 128 over four, 64.8 us (214 MB); one of 8 over 2048 tokens 14.9 us.
// Measured for the 48, and slower: sixteen softmax warps, with half the registers, 79.2 us against 77.9 at the time;
// warpgroups that take the tiles in turn, each with an accumulator of its own, 88 against 65; P and V as f16, V by
// the warps that keep O, 77.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "mfa.h"
#include "mfa_block.cuh"
#include "mfa_device.cuh"
#include "mfa_host.h"
#include "ptx.cuh"

namespace mfa {

constexpr int kTRows = kTreeRows;      // rows of a unit
constexpr int kTWgs = 2;               // softmax warpgroups, a page of a tile each
constexpr int kTSoftmaxWarp0 = 4;      // warps: producer, QK issuer, scales, PV issuer, softmax, O's
constexpr int kTSoftmaxWarps = 4 * kTWgs;
constexpr int kTOutWarp0 = kTSoftmaxWarp0 + kTSoftmaxWarps;   // four warps that keep O
constexpr int kTThreads = 32 * (kTOutWarp0 + 4);
// registers a thread, of 128 at launch: the first four warps, softmax (two times four), O's
constexpr int kTRegsRoles = 80, kTRegsSoftmax = 168, kTRegsOut = 96;
static_assert(kTRegsRoles + kTWgs * kTRegsSoftmax + kTRegsOut <= 512, "registers");
// shared memory behind the rings: segments, scratch, barriers (the last 512 bytes)
constexpr int kTMisc = 17408;
constexpr int kTFin = (kTWgs + 1) * kTRows + 4;   // floats of a segment's sums, references and scale
constexpr int kTurnStep = 2;
constexpr float kTTop = 4.f, kTMost = 8.75f, kTLeast = -2.f, kTDepth = 24.f;   // exponents of P, see above
// Value scales are taken 2^-24 times smaller, so that p = 2^(x - R) stays in range for scales up to 2^127; and then, where
// a segment's first scale is small, up to 2^24 times larger again, so that x - R is a number of few digits before its
// point (with a first scale of 2^-6 and the factor alone: 2^-19 off in every exponent).
constexpr float kTScaleDown = 0x1p-24f, kTScaleUp = 0x1p24f;
constexpr float kTEMin = -50.f - 24.f;   // and their logarithms at least this (smaller scales count as 2^-50)

template <int kDim>
struct TreeLayout {
  static constexpr int kHalves = kDim / 128;
  static constexpr int kBoxes = 2 * kHalves;            // TMA boxes [64 tokens x 128 B] of a tile of K or V
  static constexpr int kSlotBytes = kBoxes * 8192;      // a ring slot: a tile's keys or values, by 128-wide halves
  static constexpr int kOffQ = 0;                       // q: kHalves boxes of [128 hi rows, 128 lo rows][128 B]
  static constexpr int kOffRing = 2 * kTRows * kDim;
  static constexpr int kSlots = (kBSmem - kTMisc - kOffRing) / kSlotBytes;
  static constexpr int kKSlots = kSlots / 2, kVSlots = kSlots - kKSlots;   // K and V have rings of their own
  static constexpr int kOffMisc = kOffRing + kSlots * kSlotBytes;
  static constexpr uint32_t kTmemS = 0;                 // two buffers of 128 columns; then P, 64 columns a page: hi, lo
  static constexpr uint32_t kTmemO = 256;               // kDim columns
  static_assert(kKSlots >= 2 && kOffRing % 1024 == 0, "layout");
};

// Of four neighbouring lanes, each with four quarters of kWords words: lane l ends with quarter l of all four, in the
// lanes' order.
template <int kWords>
__device__ __forceinline__ void exchange_quarters(uint32_t (&v)[4 * kWords]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int step = 1; step <= 2; step *= 2) {
    const bool hi = lane & step;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q & step) continue;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {   // quarters q and q + step: keep one, send the other
        uint32_t& a = v[q * kWords + i];
        uint32_t& b = v[(q + step) * kWords + i];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? a : b, step);
        a = hi ? got : a;
        b = hi ? b : got;
      }
    }
  }
}
// A converged warp's bounded wait (see wait_bar; inline, as calls and register budgets do not go together).
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag)) != 0;
}

// The nodes that a row sees of the 64 tokens from t0 on, as bits; `prefix` tokens come before the tree.
__device__ __forceinline__ uint64_t tree_bits(uint64_t mask, int t0, int prefix, int L) {
  const int o = t0 - prefix;   // the first token's node
  uint64_t bits = o >= 64 ? 0 : o >= 0 ? mask >> o : o <= -64 ? ~0ull : (mask << -o) | ((1ull << -o) - 1);
  const int there = L - t0;
  if (there < 64) bits &= there > 0 ? (1ull << there) - 1 : 0;
  return bits;
}

template <int kDim>
__global__ void __launch_bounds__(kTThreads, 1) mfa_tree_decode_kernel(const __grid_constant__ BlockDecodeParams p) {
  using Lay = TreeLayout<kDim>;
  constexpr int kHalves = Lay::kHalves, kBoxes = Lay::kBoxes, kKSlots = Lay::kKSlots, kVSlots = Lay::kVSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint8_t* misc = smem + Lay::kOffMisc;
  BlockSegment* seg = reinterpret_cast<BlockSegment*>(misc);
  float* red = reinterpret_cast<float*>(misc + sizeof(BlockSegment) * kBMaxSeg);   // [2 tiles][warpgroups][128 rows]
  float* alpha = red + 2 * kTWgs * kTRows;                          // [2 tiles][128] what O is multiplied by
  float* fin = alpha + 2 * kTRows;                                  // [2 segments][sums of the warpgroups, reference][128], scale
  float* q_inv = fin + 2 * kTFin;                         // [2 segments][128] what undoes a row's q scaling
  int* row_off = reinterpret_cast<int*>(q_inv + 2 * kTRows);        // [128] element offset of a row's output
  int* moved = row_off + kTRows;                                    // [2 tiles][4 quarters of the rows] whether it is
  float4* meta = reinterpret_cast<float4*>(moved + 8);       // [2 tiles][2 pages][4 blocks] {K, V scales, log2 of V's}
  int* ctl = reinterpret_cast<int*>(meta + 16);                     // tensor memory, abort flag, segments, tiles
  volatile int* abort_flag = ctl + 1;
  static_assert(sizeof(BlockSegment) * kBMaxSeg + (2 * kTWgs + 2 + 3) * kTRows * 4 + 2 * kTFin * 4 + 8 * 4 + 16 * 16 + 16 + 512 <=
                    kTMisc, "misc");
  const uint32_t bars = sbase + Lay::kOffMisc + kTMisc - 512;
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  // slots: K's, then V's
  constexpr int kFull = 0, kEmpty = Lay::kSlots, kSFull = 2 * Lay::kSlots, kPFull = kSFull + 2, kPvDone = kPFull + 2,
                kQReady = kPvDone + 2, kOEmpty = kQReady + 1, kQEmpty = kOEmpty + 1, kDrain = kQEmpty + 1, kWeightsTurn = kDrain + 1,
                kMoved = kWeightsTurn + 1, kOReady = kMoved + 8, kFinal = kOReady + 2,
                kFinEmpty = kFinal + 2, kBars = kFinEmpty + 2;
  static_assert(kBars * 8 <= 512, "barrier area");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = p.max_pages * kBPage;

  if (warp == 0) {
    for (int i = lane; i < kBars; i += 32) {
      // arrivals a phase: one for each box of a slot; the issuer's and the scale warp's for a tile's
      // scores; one for each softmax warp; one for each MMA issuer (drain); else one
      const bool by_warps = i == kPFull || i == kPFull + 1 || i == kQReady || i == kFinal || i == kFinal + 1;
      const bool by_four = i == kOEmpty || i == kOReady || i == kOReady + 1 || i == kFinEmpty || i == kFinEmpty + 1;   // O's warps
      const bool by_two = i == kSFull || i == kSFull + 1 || i == kDrain;
      mbar_init(bar(i), i < kEmpty ? kBoxes : by_two ? 2 : by_four ? 4 : by_warps ? kTSoftmaxWarps : 1);
    }
    if (lane == 0) ctl[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(ctl), 512);
    tmem_relinquish();
  }
  if (tid >= 32 * kTSoftmaxWarp0 && tid < 32 * kTSoftmaxWarp0 + kTRows) {
    const int row = tid - 32 * kTSoftmaxWarp0;
    row_off[row] = (row / p.group * p.heads + row % p.group) * kDim;
  }
  if (tid == 96) {
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  // nothing that the preceding kernel may write is read before this; with early metadata the
  // lengths are (the caller says that it does not write them)
  if (!p.early_metadata) grid_dep_wait();
  if (warp == 0) block_segments<false>(p, cap, seg, ctl + 2);
  tc_fence_before();
  __syncthreads();
  if (p.early_metadata) grid_dep_wait();
  grid_dep_launch();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(ctl[0]);
  const int nseg = ctl[2], ntiles = ctl[3];

  // (each role's budget begins its branch and so covers all of its code)
  if (warp == 0) {
    reg_dealloc<kTRegsRoles>();
    // ---------------- producer: lane i loads box i of each tile of K (i < kBoxes) or of V (half
    // i / 2, page i % 2), each on its own as its slots free
    if (lane < 2 * kBoxes && ntiles > 0) {
      const bool is_v = lane >= kBoxes;
      const int half = (lane % kBoxes) >> 1, pg = lane & 1;
      const int slots = is_v ? kVSlots : kKSlots, slot0 = is_v ? kKSlots : 0;
      const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_last();
      BlockTile<false> it;
      it.load(p, seg, 0);
      auto page_id = [&]() -> int {
        return it.rows(p, pg).to > 0 ? p.block_table[static_cast<size_t>(it.b) * p.max_pages + it.page(pg)] : 0;
      };
      int id = page_id();
      int slot = 0, phase = 0;
      bool ok = true;
      int n = 0;
      for (; n < ntiles;) {
        const int rows = it.rows(p, pg).to;
        int z = id * p.kv_heads + it.kvh;
        if (rows > 0 && (id < 0 || id >= p.num_blocks)) {
          z = -1;   // outside the pool: the whole box reads as zeros
          if (lane < 2) atomicOr(p.status, MFA_DEV_BAD_BLOCK);
        }
        const uint64_t pol = it.again ? again : once;
        if (it.next(p, seg, nseg)) id = page_id();
        ok = wait_bar(bar(kEmpty + slot0 + slot), phase ^ 1, abort_flag);
        if (!ok) break;
        const uint32_t fb = bar(kFull + slot0 + slot);
        if (rows <= 0) {
          mbar_arrive(fb);
        } else {   // (the rows past the sequence's end come along: scores and weights leave them out, and the issuer zeroes V's)
          mbar_arrive_expect_tx(fb, 8192);
          tma_load_3d_hint(sbase + Lay::kOffRing + (slot0 + slot) * Lay::kSlotBytes + (2 * half + pg) * 8192, is_v ? &p.tm_v : &p.tm_k, fb,
                           128 * half, 0, z, pol);
        }
        ++n;
        if (++slot == slots) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (!ok) {
        atomicOr(p.status, MFA_DEV_TIMEOUT);
        // let every copy already issued land before the CTA can exit
        for (int u = max(0, n - slots); u < n; ++u)
          wait_slow(bar(kFull + slot0 + u % slots), (u / slots) & 1, nullptr, kDrainLimitNs);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    reg_dealloc<kTRegsRoles>();
    // ---------------- QK issuer: S(n) = Q K(n)^T
    if (ntiles > 0) {
      constexpr uint32_t kIdescQK = idesc_e4m3(false, false, kTRows, kBTile);
      const uint32_t lead = elect_lane(), base = uniform(sbase), tm = uniform(tmem);
      const int segments = uniform(nseg);
      bool ok = true;
      int slot = 0, phase = 0, n = 0;
#pragma unroll 1
      for (int s = 0; s < segments && ok; ++s) {
        const int count = uniform(seg[s].hi - seg[s].lo);
        ok = wait_all(bar(kQReady), s & 1, abort_flag);
#pragma unroll 1
        for (int i = 0; i < count && ok; ++i, ++n) {
          ok = wait_all(bar(kFull + slot), phase, abort_flag);
          const uint32_t d = tm + Lay::kTmemS + kBTile * (n & 1);
          uint64_t bd = smem_desc(base + Lay::kOffRing + slot * Lay::kSlotBytes, 16, 1024);
          uint64_t ad = smem_desc(base + Lay::kOffQ, 16, 1024);
          // The product that reads the weights where these scores go is complete: two warps' MMAs into different
          // accumulators have no order but this.  (With a wait for its issue alone, which is not enough, the eight of
          // 4096 tokens took 56.0 us against 58.1, the ragged ones 99.9 against 103, the 48 64.0 against 64.8.)
          if (ok && n >= 2) ok = wait_all(bar(kPvDone + (n & 1)), ((n >> 1) - 1) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          uint32_t more = 0;
#pragma unroll 1
          for (int h = 0; h < kHalves; ++h) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {   // 32 elements a step: 2 of the descriptors' 16-byte units
              // (the other issuer's turn begins while the last steps, which share nothing with its product, wait their own)
              if (kk == kTurnStep && h == kHalves - 1 && i > 0 && lead) mbar_arrive(bar(kWeightsTurn));
              umma_f8_ss_by(lead, d, ad + 2 * kk, bd + 2 * kk, kIdescQK, more);
              more = 1;
              umma_f8_ss_by(lead, d, ad + 1024 + 2 * kk, bd + 2 * kk, kIdescQK, 1);   // lo: 16 KB on
            }
            ad += 2048;
            bd += 1024;
          }
          umma_commit_by(lead, bar(kSFull + (n & 1)));
          umma_commit_by(lead, bar(kEmpty + slot));
          if (i == count - 1) umma_commit_by(lead, bar(kQEmpty));
          if (++slot == kKSlots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok && lane == 0) atomicOr(p.status, MFA_DEV_TIMEOUT);
      // every MMA must be complete before tensor memory is released
      umma_commit_by(lead, bar(kDrain));
      wait_slow(bar(kDrain), 0, nullptr, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp == 3) {
    reg_dealloc<kTRegsRoles>();
    // ---------------- PV issuer: O += P(n) V(n)
    if (ntiles > 0) {
      constexpr uint32_t kIdescHi = idesc_e4m3(false, true, kTRows, 128), kIdescLo = kIdescHi | (1u << 7);   // (A: e5m2)
      const uint32_t lead = elect_lane(), base = uniform(sbase), tm = uniform(tmem);
      const int segments = uniform(nseg);
      bool ok = true;
      int slot = 0, phase = 0, n = 0, turn = 0;
#pragma unroll 1
      for (int s = 0; s < segments && ok; ++s) {
        const int lo = uniform(seg[s].lo), hi = uniform(seg[s].hi), L = uniform(seg[s].L);
#pragma unroll 1
        for (int j = lo; j < hi && ok; ++j, ++n) {
          ok = wait_all(bar(kFull + kKSlots + slot), phase, abort_flag);
          const int box = Lay::kOffRing + (kKSlots + slot) * Lay::kSlotBytes;
          const int rest = L - kBTile * j;            // tokens of the tile
          const bool both = rest > kBPage;            // it has its second page
          if (ok && rest < kBTile && rest % kBPage != 0) {   // whatever lies past the end of the last page: zeros
#pragma unroll 1
            for (int h = 0; h < kHalves; ++h) {
              uint8_t* at = smem + box + h * 16384 + (both ? 8192 : 0);
              for (int r = rest % kBPage + (lane >> 3); r < kBPage; r += 4)
                *reinterpret_cast<uint4*>(at + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          const uint32_t ap = tm + Lay::kTmemS + kBTile * (n & 1);
          uint64_t bd = smem_desc(base + box, 8192, 1024);
          if (ok && j == lo && s > 0) ok = wait_all(bar(kOEmpty), (s - 1) & 1, abort_flag);
          if (ok) ok = wait_all(bar(kPFull + (n & 1)), (n >> 1) & 1, abort_flag);
          if (ok) ok = wait_all(bar(kOReady + (n & 1)), (n >> 1) & 1, abort_flag);
          // the next tile's scores go first: the softmax waits for them
          if (ok && j + 1 < hi) ok = wait_all(bar(kWeightsTurn), turn++ & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < kHalves; ++h) {
            const uint32_t d = tm + Lay::kTmemO + 128 * h;
            // 32 tokens a step: 8 columns of P, 4096 bytes of V, two steps a page
            umma_f8_ts_by(lead, d, ap, bd, kIdescHi, j != lo);
            umma_f8_ts_by(lead, d, ap + 16, bd, kIdescLo, 1);
            umma_f8_ts_by(lead, d, ap + 8, bd + 256, kIdescHi, 1);
            umma_f8_ts_by(lead, d, ap + 24, bd + 256, kIdescLo, 1);
            if (both) {
              umma_f8_ts_by(lead, d, ap + 64, bd + 512, kIdescHi, 1);
              umma_f8_ts_by(lead, d, ap + 80, bd + 512, kIdescLo, 1);
              umma_f8_ts_by(lead, d, ap + 72, bd + 768, kIdescHi, 1);
              umma_f8_ts_by(lead, d, ap + 88, bd + 768, kIdescLo, 1);
            }
            bd += 1024;
          }
          umma_commit_by(lead, bar(kPvDone + (n & 1)));
          umma_commit_by(lead, bar(kEmpty + kKSlots + slot));
          if (++slot == kVSlots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok && lane == 0) atomicOr(p.status, MFA_DEV_TIMEOUT);
      umma_commit_by(lead, bar(kDrain));
      wait_slow(bar(kDrain), 0, nullptr, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp == 2) {
    reg_dealloc<kTRegsRoles>();
    // ---------------- scales: a tile's up to 2 x 4 block scales of K and of V, ahead of the softmax
    // (lane = V? page, block); page ids two tiles ahead, scales one tile ahead
    const int pg = (lane >> 2) & 1, blk = lane & 3;
    const bool is_v = (lane & 8) != 0, mine = lane < 16 && blk < (kBPage >> p.log_scale);
    const float* src = is_v ? p.v_scale : p.k_scale;
    const float mul = is_v ? kTScaleDown : p.scale_log2;
    for (int i = lane; i < nseg && p.cluster == 0; i += 32) {   // where the combine finds a unit's parts
      const BlockSegment x = seg[i];
      int2* at = p.parts + static_cast<size_t>(x.kvh * p.token_groups + x.tg) * p.batch + x.b;
      if (x.lo == 0) at->x = x.slot;
      if (x.hi == block_tiles(x.L)) at->y = x.slot;
    }
    if (ntiles > 0) {
      BlockTile<false> it;
      it.load(p, seg, 0);
      // a block without a token (its scale may hold any bits) and one outside the pool: keys as they are, no value
      auto page_id = [&]() -> int {
        return mine && it.rows(p, pg).to > blk << p.log_scale ? p.block_table[static_cast<size_t>(it.b) * p.max_pages + it.page(pg)] : -1;
      };
      auto scale_of = [&](int id) -> float {
        if (id < 0 || id >= p.num_blocks) return is_v ? 0.f : 1.f;
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
            const int first = seg[s].tg * p.unit_tokens, nodes = min(p.unit_tokens, p.tokens - first);
            const int lines = p.group * kDim * 2 / 128;
            for (int i = lane; i < nodes * lines; i += 32) {
              const char* q = reinterpret_cast<const char*>(
                  p.q + ((static_cast<size_t>(it.b) * p.tokens + first + i / lines) * p.heads + static_cast<size_t>(it.kvh) * p.group) * kDim);
              asm volatile("prefetch.global.L2 [%0];" ::"l"(q + i % lines * 128));
            }
          }
          value_next = scale_of(id);
          more = it.next(p, seg, nseg);
          if (more) id = page_id();
        }
        // the softmax has read the tile before last's when its weights are there
        if (n >= 2 && !__all_sync(0xffffffffu, wait_bar(bar(kPFull + (n & 1)), ((n >> 1) - 1) & 1, abort_flag))) {
          if (lane == 0) atomicOr(p.status, MFA_DEV_TIMEOUT);
          break;
        }
        if (mine) {
          float* at = reinterpret_cast<float*>(meta + (n & 1) * 8 + pg * 4 + blk);
          at[is_v ? 1 : 0] = value * mul;
          if (is_v) at[2] = fmaxf(log2f(value * mul), kTEMin);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSFull + (n & 1)));
        value = value_next;
      }
    }
    __syncwarp();
  } else if (warp < kTOutWarp0) {
    reg_alloc<kTRegsSoftmax>();
    // ---------------- softmax: warpgroup wg has page wg of each tile, a thread one row
    const int sw = warp - kTSoftmaxWarp0, wg = sw >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t pair_bar = 1 + quarter;   // the two warps that have the same rows
    const bool f32 = p.out_f32 != 0;
    // A wait that gives up raises the CTA's abort flag, and its warp waits no more; the warps leave together,
    // by a vote at their segment's end, so that their barriers stay in step.
    bool aborted = false, stop = false;
    // q of a segment, split into e4m3 hi + lo parts under one power of two a row (split_e4m3):
    // eight lanes a row, four rows a warp at a time; lane i has the 8-element chunks i, i + 8, ...
    auto convert_q = [&](int sidx) {
      constexpr int kChunks = kDim / 64, kRounds = kTRows / (4 * kTSoftmaxWarps), kAtOnce = 4;
      const BlockSegment sg = seg[sidx];
      const int valid = p.group * min(p.unit_tokens, p.tokens - sg.tg * p.unit_tokens);
      const __nv_bfloat16* src = p.q + ((static_cast<size_t>(sg.b) * p.tokens + sg.tg * p.unit_tokens) * p.heads +
                                        static_cast<size_t>(sg.kvh) * p.group) * kDim;
      const int r0 = sw * 4 + (lane >> 3), i8 = lane & 7;
#pragma unroll 1
      for (int x0 = 0; x0 < kRounds; x0 += kAtOnce) {
        uint4 wr[kAtOnce][kChunks];
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
          const int r = r0 + 4 * kTSoftmaxWarps * (x0 + x);
#pragma unroll
          for (int k = 0; k < kChunks; ++k)
            wr[x][k] = r < valid ? __ldg(reinterpret_cast<const uint4*>(src + row_off[r]) + i8 + 8 * k) : make_uint4(0, 0, 0, 0);
        }
        // (the previous segment's last scores are made: its q is read no more)
        if (x0 == 0 && sidx > 0 && !wait_bar(bar(kQEmpty), (sidx - 1) & 1, abort_flag)) aborted = true;
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
          const int r = r0 + 4 * kTSoftmaxWarps * (x0 + x);
          const uint4(&w)[kChunks] = wr[x];
          float m = 0.f;
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            const uint32_t e[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int y = 0; y < 4; ++y)
              m = fmaxf(m, fmaxf(fabsf(__uint_as_float(e[y] << 16)), fabsf(__uint_as_float(e[y] & 0xFFFF0000u))));
          }
#pragma unroll
          for (int o = 4; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          int sig = 0;   // the row's largest |q| goes to [128, 256): what is under 2^-9 of it errs by up to 2^-17 of it
          if (m > 0.f) sig = min(126, max(-126, 7 + 127 - static_cast<int>(__float_as_uint(m) >> 23)));
          const float up = __uint_as_float(static_cast<uint32_t>(127 + sig) << 23);
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            const uint32_t e[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              split_e4m3(__uint_as_float(e[y] << 16) * up, __uint_as_float(e[y] & 0xFFFF0000u) * up, hi[y], lo[y]);
            const int byte = 8 * (i8 + 8 * k) % 128;   // chunk of a half's 128-byte row
            uint8_t* dst = smem + Lay::kOffQ + (k / 2) * (2 * kTRows * 128) + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 8);
            *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
            *reinterpret_cast<uint2*>(dst + kTRows * 128) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
          }
          if (i8 == 0) q_inv[(sidx & 1) * kTRows + r] = m < INFINITY ? __uint_as_float(static_cast<uint32_t>(127 - sig) << 23) : NAN;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQReady));
    };

    if (ntiles > 0) convert_q(0);
    int n = 0;
    for (int s = 0; s < nseg && !stop; ++s) {
      const BlockSegment sg = seg[s];
      const int L = sg.L, prefix = L - p.tokens;   // tokens before the tree (all nodes see them)
      const int node0 = sg.tg * p.unit_tokens;
      const int valid = p.group * min(p.unit_tokens, p.tokens - node0);
      const uint64_t mask = row < valid ? p.tree[static_cast<size_t>(sg.b) * p.tokens + node0 + row / p.group] : 0;
      if (!wait_bar(bar(kQReady), s & 1, abort_flag)) aborted = true;
      const float inv = q_inv[(s & 1) * kTRows + row];
      float shift = 0.f, up = 1.f;   // see kTScaleDown
      float ref = 0.f, top = -INFINITY, most = -INFINITY;   // the reference, its highest, and what x + e may reach
      uint64_t l2 = 0;                                      // the row's sum over this page's tokens, in two parts
      for (int j = sg.lo; j < sg.hi; ++j, ++n) {
        if (!wait_bar(bar(kSFull + (n & 1)), (n >> 1) & 1, abort_flag)) aborted = true;
        tc_fence_after();
        uint32_t sr[2][32];
        const uint32_t at = tmem + Lay::kTmemS + kBTile * (n & 1) + 64 * wg + lane_base;
        tmem_ld32(at, sr[0]);
        tmem_ld32(at + 32, sr[1]);
        if (j == sg.lo) {
          shift = fminf(fmaxf(-rintf(meta[(n & 1) * 8].z), 0.f), 24.f);
          up = __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(shift)) << 23);
        }
        float a[4], sv[4], e[4];   // by 16 tokens: key scale with the row's, value scale and its exponent
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float4 sc = meta[(n & 1) * 8 + wg * 4 + ((16 * g) >> p.log_scale)];
          a[g] = sc.x * inv;
          sv[g] = sc.y * up;
          e[g] = sc.z + shift;
        }
        tmem_ld_wait(sr[0]);
        tmem_ld_wait(sr[1]);
        if (kBTile * (j + 1) > prefix) {   // the tree's tokens, and what lies past the end
          const uint64_t bits = tree_bits(mask, kBTile * j + kBPage * wg, prefix, L);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (!(static_cast<uint32_t>(bits) >> i & 1)) sr[0][i] = 0xFF800000u;
            if (!(static_cast<uint32_t>(bits >> 32) >> i & 1)) sr[1][i] = 0xFF800000u;
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) a[g] = fmaxf(a[g], 0x1p-126f);   // (-inf stays -inf)
          if (!(inv < INFINITY)) a[0] = a[1] = a[2] = a[3] = NAN;
        }
        float m = -INFINITY;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t(&r)[32] = sr[g >> 1];
          const int c = 16 * (g & 1);
          float x = __uint_as_float(r[c + 15]);
#pragma unroll
          for (int i = 0; i < 14; i += 2) x = max3(x, __uint_as_float(r[c + i]), __uint_as_float(r[c + i + 1]));
          x = fmaxf(x, __uint_as_float(r[c + 14]));
          m = fmaxf(m, fmaf(x, a[g], e[g]));
        }
        // the row's largest x + e, of both pages
        float* mine = red + (n & 1) * (kTWgs * kTRows);
        mine[wg * kTRows + row] = m;
        named_bar_sync(pair_bar, 64);
        m = fmaxf(m, mine[(wg ^ 1) * kTRows + row]);
        const bool rise = m > most;
        const bool fall = m < ref + kTLeast && m > -INFINITY && most > -INFINITY && fmaxf(m - kTTop, top - kTDepth) < ref - 1.f;
        const bool moves = __any_sync(0xffffffffu, rise || fall);
        float factor = 1.f;
        if (moves) {   // new references: the sums move to them here, O by its warps
          float to = ref;
          if (fall) to = fmaxf(m - kTTop, top - kTDepth);
          if (m > ref + kTTop + 1.f || rise) to = m - kTTop;
          if (!(m > -INFINITY && m < INFINITY)) to = ref;
          const bool set = most > -INFINITY;
          factor = set ? ex2_approx(ref - to) : 1.f;
          ref = to;
          if (set || (m > -INFINITY && m < INFINITY)) {
            most = ref + kTMost;
            top = fmaxf(top, ref);
          }
          l2 = mul_f32x2(l2, pack_f32x2(factor, factor));
        }
        if (wg == 0) {
          if (moves) alpha[(n & 1) * kTRows + row] = factor;
          if (lane == 0) moved[(n & 1) * 4 + quarter] = moves && j > sg.lo;   // (before a segment's second tile O holds nothing)
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kMoved + 4 * (n & 1) + quarter));
        }
        // p = 2^(x - R) and its sum in fp32; P = p sv rounded to f16 (2^-11) and split
        const uint64_t nref = pack_f32x2(-ref, -ref);
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {   // four tokens
          const int g = i >> 2;
          const uint64_t a2 = pack_f32x2(a[g], a[g]), v2 = pack_f32x2(sv[g], sv[g]);
          uint32_t pu[2], back[2], rest[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int c = (4 * i + 2 * k) & 31;
            float x0, x1;
            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(sr[i >> 3][c]), __uint_as_float(sr[i >> 3][c + 1])), a2, nref), x0, x1);
            const uint64_t p2 = pack_f32x2(ex2_approx(x0), ex2_approx(x1));
            l2 = add_f32x2(l2, p2);
            float w0, w1;
            unpack_f32x2(mul_f32x2(p2, v2), w0, w1);
            const __half2 v = __floats2half2_rn(w0, w1);
            pu[k] = *reinterpret_cast<const uint32_t*>(&v);
          }
          hi[i] = cvt_e4m3x4(pu[0], pu[1]);
          cvt_f16x4(hi[i], back[0], back[1]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&pu[k]), *reinterpret_cast<const __half2*>(&back[k]));
            rest[k] = *reinterpret_cast<const uint32_t*>(&v);
          }
          lo[i] = cvt_e5m2x4(rest[0], rest[1]);
        }
        tmem_st16(at, hi);
        tmem_st16(at + 16, lo);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull + (n & 1)));
      }
      {   // what the segment's result takes beside O
        if (s >= 2 && !wait_bar(bar(kFinEmpty + (s & 1)), ((s >> 1) - 1) & 1, abort_flag)) aborted = true;
        float l0, l1;
        unpack_f32x2(l2, l0, l1);
        float* mine = fin + (s & 1) * kTFin + row;
        mine[wg * kTRows] = l0 + l1;
        if (wg == 0) {
          mine[kTWgs * kTRows] = ref;
          if (row == 0) mine[(kTWgs + 1) * kTRows] = kTScaleUp / up;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kFinal + (s & 1)));
      }
      if (s + 1 < nseg) convert_q(s + 1);
      if (named_bar_or(1 + 4, 32 * kTSoftmaxWarps, aborted || *abort_flag)) stop = true;
    }
    // sequences without tokens: zeros and -inf, in turn over the CTAs
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
      bool dummy = false;
      if (clamp_len(p.seq_lens[b], cap, dummy) != 0) continue;
      const size_t rows = static_cast<size_t>(p.tokens) * p.heads, first = static_cast<size_t>(b) * rows;
      const size_t chunks = rows * kDim * (f32 ? 4 : 2) / 16;
      uint4* o = static_cast<uint4*>(p.out) + first * kDim * (f32 ? 4 : 2) / 16;
      for (size_t i = tid - 32 * kTSoftmaxWarp0; i < chunks; i += 32 * kTSoftmaxWarps) o[i] = make_uint4(0, 0, 0, 0);
      if (p.lse != nullptr)
        for (size_t i = tid - 32 * kTSoftmaxWarp0; i < rows; i += 32 * kTSoftmaxWarps) p.lse[first + i] = -INFINITY;
    }
    if (stop && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.status, MFA_DEV_TIMEOUT);
    }
  } else {
    reg_dealloc<kTRegsOut>();
    // ---------------- O: a warp has 32 rows.  References that move: O moves with them between two products, while the
    // softmax goes on (by the softmax's own threads, in between, such a tile took half as long again).  A segment's
    // result: written while the next one's q is converted.
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t at = tmem + Lay::kTmemO + (static_cast<uint32_t>(quarter * 32) << 16);
    const bool f32 = p.out_f32 != 0;
    bool ok = true;
    int n = 0;
#pragma unroll 1
    for (int s = 0; s < nseg && ok; ++s) {
      const BlockSegment sg = seg[s];
#pragma unroll 1
      for (int j = sg.lo; j < sg.hi && ok; ++j, ++n) {
        ok = wait_all(bar(kMoved + 4 * (n & 1) + quarter), (n >> 1) & 1, abort_flag);
        if (ok && moved[(n & 1) * 4 + quarter]) {
          const float f = alpha[(n & 1) * kTRows + row];
          ok = wait_all(bar(kPvDone + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort_flag);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kDim && ok; c += 32) {
            uint32_t o[32];
            tmem_ld32(at + c, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32(at + c, o);
          }
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kOReady + (n & 1)));
      }
      if (ok) ok = wait_all(bar(kFinal + (s & 1)), (s >> 1) & 1, abort_flag);
      if (!ok) break;
      const float* mine = fin + (s & 1) * kTFin;
      const float sum = mine[row] + mine[kTRows + row], ref = mine[kTWgs * kTRows + row], unit = mine[(kTWgs + 1) * kTRows];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kFinEmpty + (s & 1)));
      ok = wait_all(bar(kPvDone + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const int node0 = sg.tg * p.unit_tokens, valid = p.group * min(p.unit_tokens, p.tokens - node0);
      const float back = sum == 0.f ? 0.f : unit / sum;   // (a row that sees nothing: zeros)
      const bool whole = sg.slot == -1;
      const size_t first = (static_cast<size_t>(sg.b) * p.tokens + node0) * p.heads + static_cast<size_t>(sg.kvh) * p.group;
      float* part = p.part_o + static_cast<size_t>(max(sg.slot, 0)) * p.rows8 * kDim;
      uint8_t* out = static_cast<uint8_t*>(p.out) + first * kDim * (f32 ? 4 : 2);
#pragma unroll 1
      for (int c = 0; c < kDim; c += 32) {
        uint32_t o[32];
        tmem_ld32(at + c, o);
        tmem_ld_wait(o);
        if (c + 32 == kDim) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kOEmpty));   // the next segment may accumulate
        }
        // Four lanes exchange quarters of their rows, so that each writes its quarter of all four rows and a store
        // touches eight lines in place of 32.
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * back);
        if (whole && !f32) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
            w[k] = *reinterpret_cast<const uint32_t*>(&x);
          }
          exchange_quarters<4>(w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = row - (lane & 3) + i;
            if (r < valid)
              *reinterpret_cast<uint4*>(out + static_cast<size_t>(row_off[r]) * 2 + c * 2 + (lane & 3) * 16) =
                  make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        } else {   // (parts: rows as they are in the outputs)
          exchange_quarters<8>(o);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = row - (lane & 3) + i;
            float* to = whole ? reinterpret_cast<float*>(out) + row_off[r] : part + static_cast<size_t>(r) * kDim;
            if (r < valid) {
              const uint4 x = make_uint4(o[8 * i], o[8 * i + 1], o[8 * i + 2], o[8 * i + 3]);
              const uint4 y = make_uint4(o[8 * i + 4], o[8 * i + 5], o[8 * i + 6], o[8 * i + 7]);
              *reinterpret_cast<uint4*>(to + c + (lane & 3) * 8) = x;
              *reinterpret_cast<uint4*>(to + c + (lane & 3) * 8 + 4) = y;
            }
          }
        }
      }
      if (row < valid) {
        // (the sum's exponent joins the reference first: their logarithms alone would cancel)
        const int k = min(static_cast<int>(__float_as_uint(sum) >> 23), 253) - 127;
        const float v = sum == 0.f ? -INFINITY
                                   : fmaf(static_cast<float>(k) + ref, 0.6931471805599453f,
                                          logf(sum * __uint_as_float(static_cast<uint32_t>(127 - k) << 23)));
        if (!whole)
          p.part_lse[static_cast<size_t>(sg.slot) * p.rows8 + row] = v;
        else if (p.lse != nullptr)
          p.lse[first + row_off[row] / kDim] = v;
      }
    }
    if (!ok && lane == 0) atomicOr(p.status, MFA_DEV_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ combine kernel
//
// Units in parts: out = sum_s w_s O_s with w_s = e^(lse_s - lse), lse = ln sum_s e^lse_s.  A thread has eight elements
// of a row (32 bytes of a part), so that a part's weight is one for them, and goes over the parts with a running
// maximum.  kTeams warps share a row's parts, in a fixed order, where they are many; where units have two or
// three parts, or none, CTAs are short and an SM holds many.
template <int kDim, int kTeams>
__global__ void __launch_bounds__(256, 6) mfa_tree_combine_kernel(const __grid_constant__ BlockDecodeParams p) {
  constexpr int kLanes = kDim / 8, kRows = 32 / kLanes * (8 / kTeams);   // lanes of a row, rows of a CTA
  constexpr int kAhead = 2;                                             // parts that are loaded together
  __shared__ float other[kTeams > 1 ? 8 : 1][kTeams > 1 ? 32 : 1][11];   // of the warps (odd pitch: no bank conflicts)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, team = warp % kTeams;
  const int row = blockIdx.y * kRows + warp / kTeams * (32 / kLanes) + lane / kLanes, el = lane % kLanes * 8;
  const int pos = blockIdx.x, b = pos % p.batch, r = pos / p.batch;
  const int kvh = r / p.token_groups, tg = r - kvh * p.token_groups;
  const int valid = p.group * min(p.unit_tokens, p.tokens - tg * p.unit_tokens);
  bool bad = false;
  const int L = clamp_len(p.seq_lens[b], p.max_pages * kBPage, bad);   // (final: the decode kernel has waited for what came before)
  grid_dep_wait();
  grid_dep_launch();
  if (L == 0) return;
  const int2 at = p.parts[pos];
  if (at.y <= at.x || at.x < 0 || at.y >= p.num_partials) return;   // one part, the output itself; or past the plan, as reported
  const int here = min(row, valid - 1);
  const float* part = p.part_o + static_cast<size_t>(here) * kDim + el;
  const float* lse = p.part_lse + here;
  const size_t pitch = static_cast<size_t>(p.rows8) * kDim;
  float acc[8] = {}, sum = 0.f, top = -INFINITY;
  auto add = [&](float l) {   // (sums and accumulators move to the larger maximum)
    const float m = fmaxf(top, l), ref = m == -INFINITY ? 0.f : m;   // (a row that sees nothing of these parts)
    const float back = ex2_approx((top - ref) * 1.4426950408889634f), w = ex2_approx((l - ref) * 1.4426950408889634f);
    top = m;
    return make_float2(back, w);
  };
#pragma unroll 1
  for (int k = at.x + team; k <= at.y; k += kAhead * kTeams) {
    float o[kAhead][8], l[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const size_t slot = min(k + x * kTeams, at.y);
      l[x] = lse[slot * p.rows8];
      ld_global_f32x8(part + slot * pitch, o[x]);
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const float2 f = add(k + x * kTeams <= at.y ? l[x] : -INFINITY);
      sum = fmaf(sum, f.x, f.y);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(acc[i], f.x, f.y * o[x][i]);
    }
  }
  if constexpr (kTeams > 1) {
    if (team > 0) {
      float* mine = other[warp][lane];
#pragma unroll
      for (int i = 0; i < 8; ++i) mine[i] = acc[i];
      mine[8] = sum;
      mine[9] = top;
    }
    __syncthreads();
    if (team > 0) return;
#pragma unroll 1
    for (int x = 1; x < kTeams; ++x) {
      const float* theirs = other[warp + x][lane];
      const float2 f = add(theirs[9]);
      sum = fmaf(sum, f.x, f.y * theirs[8]);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(acc[i], f.x, f.y * theirs[i]);
    }
  }
  if (row >= valid) return;
  const size_t to = (static_cast<size_t>(b) * p.tokens + tg * p.unit_tokens + row / p.group) * p.heads + static_cast<size_t>(kvh) * p.group +
                    row % p.group;
  const float back = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] *= back;
  if (p.out_f32) {
    float* o = static_cast<float*>(p.out) + to * kDim + el;
    *reinterpret_cast<float4*>(o) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    *reinterpret_cast<float4*>(o + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[2 * k], acc[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&x);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + to * kDim + el) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (el == 0 && p.lse != nullptr) p.lse[to] = sum == 0.f ? -INFINITY : top + logf(sum);
}

cudaError_t launch_tree_combine(const BlockDecodeParams& p, int units, int ctas, int head_dim, cudaLaunchConfig_t cfg) {
  const int teams = ctas > 32 * units ? 8 : ctas > 4 * units ? 4 : 1, rows = 256 / head_dim * (8 / teams);   // by a unit's parts
  cfg.gridDim = dim3(static_cast<unsigned>(units), static_cast<unsigned>((p.rows8 + rows - 1) / rows), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = 0;
  BlockDecodeFn fn;
  if (head_dim == 256)
    fn = teams == 8   ? mfa_tree_combine_kernel<256, 8>
         : teams == 4 ? mfa_tree_combine_kernel<256, 4>
                      : mfa_tree_combine_kernel<256, 1>;
  else
    fn = teams == 8   ? mfa_tree_combine_kernel<128, 8>
         : teams == 4 ? mfa_tree_combine_kernel<128, 4>
                      : mfa_tree_combine_kernel<128, 1>;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

BlockDecodeFn tree_kernel(int head_dim) { return head_dim == 256 ? mfa_tree_decode_kernel<256> : mfa_tree_decode_kernel<128>; }
int tree_threads() { return kTThreads; }

}  // namespace mfa
