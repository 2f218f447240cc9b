// Norms of query heads and new key rows with their rotary positions in one pass, and the gradient
// (GB300, sm_103a).
//
// For each head x of d elements, with its side's weights w and R the rotation by the row's positions:
//     r = (sum x^2 / d + eps)^(-1/2),   y = R (x r w).
// Gradient, with g = R^T dy (R turns, so its transpose turns back), u = g w:
//     dx = r (u - x r^2 sum(u x) / d),   dw = sum over rows and heads of g x r.
//
// Every element is read once (in the gradient x and dy) and written once, with some ten operations for each:
// HBM-bound for a prompt or a training batch, launch-bound for a decode step.  A head's elements lie in
// the registers of a group of up to 32 lanes (a lane: 8 elements, under half pairing with their 8 partners, in
// vectors of 16 bytes), so that its sums are a few shuffles and nothing is read twice.
// A CTA turns all heads of a row: the row's angles are computed once and shared.  A group keeps to one
// side, q or k, and multiplies its weights with the angles' cosines and sines once a row in the forward
// pass.  All sums are fp32; outputs are rounded once.
//
// Measured in a graph of twelve calls over three states, bf16 unless said (the bytes at the copy rate of 6.7 TB/s in
// brackets):
//   8191 rows of 65 heads of 256, three axes: 85 us, 6.4 TB/s (82); 128 such rows 4.8 us, launch and one
//   chain of loads: positions and angles, the elements, two sums;
//   its gradient 151 us, 5.4 TB/s (122); that of 1021 rows of 68 heads of 128, fp32, 96 turned, 22 us (16),
//   4000 rows of 65 of 256 in fp32 90 us forward (80), 129 the gradient (120).
// What bounds the gradient: issue slots as much as memory, some 13 instructions an element beside the loads.
// The steps that carried it, the prompt / its gradient (replays of a graph of one call, some 3 us more each): plain loads, one
// CTA on an SM 188 / 272; arithmetic in pairs, two CTAs 108 / 240; copies ahead into shared memory, free of bank
// conflicts, 105 / 203; angles by a warp of their own 88 / -; values read from shared memory again in place of kept, and
// the CTA's meetings one in four rows, - / 156.  Asking L2 for the next rows gained nothing; three CTAs on an SM (fewer
// registers and copies ahead) 120 for the prompt.  fp32, a lane's two vectors side by side, so that each copy takes half of
// every sector: 115 and 193 for the 4000 rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "mfa.h"
#include "mfa_host.h"
#include "mfa_rope.cuh"
#include "ptx.cuh"

namespace mfa {

constexpr int kNormThreads = 288;        // of a CTA that have heads, at most; with a warp of angles two CTAs on an SM
// Wide path: where an element's partner in its pair lies.  In the same vector; in a vector of its own, which the same lane
// has; or anywhere in the head (half pairing of pairs that are no eights), read from the copies of the group's lanes, element by
// element, and with half as many elements a lane (65 heads of 256, fp32, gradient of 2000 rows: 70 us of 60, 288 on the
// path for any shape).
enum NormPairs { kPairsNext, kPairsVectors, kPairsFar };
constexpr int kNormAnyThreads = 256;     // of a CTA of the path for any shape
// The weights' gradient: where a thread's fp32 sum would have more terms than this, it is added to one in 64 bits and begins
// anew after so many, or after those of 36 rows, if they are more.  (One sum over all of a thread's rows is off by up to 2^-24
// a term: 2^21 equal rows, 6900 terms, by 9e-5 of itself.  65536 rows of 65 heads of 256 take 1136 us with, 1130 without; other
// widths and types 2 to 4% more.)
constexpr int kNormTerms = 256;
constexpr int kNormGradRows = 4;         // rows of a CTA from one meeting to the next, in the gradient on the wide path

struct NormSide {
  const void* x;
  const void* dy;       // gradient only
  void* out;            // y; gradient: dx
  const void* w;
  long long x_stride, dy_stride, out_stride;
  int heads, slots;     // slots: groups of lanes (any shape: warps) that share the heads
};

struct NormParams {
  NormSide q, k;
  const mfa_rope_pair* table;
  const int32_t* positions;
  int rows, axes, pairs, head_dim;
  int angles;           // pairs, and on the wide path what does not turn beside them
  int turned_vectors, units, log_lanes;   // wide path: vectors with partners (half pairing), a head's units, lanes of its group
  int half;                             // pairing, for any shape
  int w_f32;
  float eps, inv_dim;
  float* partial;                       // gradient: [CTAs][q, k][head_dim]
  float* dw[2];                         // gradient of the weights
  int parts;                            // CTAs that leave partial sums
  int fold;                             // rows (wide path: meetings) that a thread's sum goes over; 0: all
};

template <typename T>
__device__ __forceinline__ float norm_load(const void* p, int i) {
  if constexpr (sizeof(T) == 2)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else
    return static_cast<const float*>(p)[i];
}
template <typename T>
__device__ __forceinline__ void norm_store(T* p, float v) {
  if constexpr (sizeof(T) == 2)
    *p = __float2bfloat16_rn(v);
  else
    *p = v;
}
__device__ __forceinline__ float norm_weight(const NormParams& p, const NormSide& s, int i) {
  return p.w_f32 ? norm_load<float>(s.w, i) : norm_load<__nv_bfloat16>(s.w, i);
}

// Angles of row `row`, one pair a thread, into cs, pair i at place(i); kFar: one element a thread, its sine with the sign
// that its partner has in it.
template <bool kFar, typename Place>
__device__ __forceinline__ void row_angles(const NormParams& p, long long row, int tid, int threads, float (&cs)[2][kRopeMaxDim / 2],
                                           Place place) {
  int32_t pos[MFA_ROPE_MAX_AXES];
#pragma unroll
  for (int x = 0; x < MFA_ROPE_MAX_AXES; ++x) pos[x] = x < p.axes ? p.positions[static_cast<long long>(x) * p.rows + row] : 0;
  for (int i = tid; i < p.angles; i += threads) {
    float s = 0.f, c = 1.f;
    const bool second = kFar && i >= p.pairs;
    const int pair = second ? i - p.pairs : i;
    if (pair < p.pairs) rope_angle(p.table, pair, pos, s, c);
    cs[0][place(i)] = c;
    cs[1][place(i)] = kFar && !second ? -s : s;
  }
}

// Sums of N values over a head's group of 2^log_lanes lanes.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], unsigned mask, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    if (o >= lanes) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(mask, v[i], o);
  }
}

// A thread's place: its group's slot on one side, its unit of the head: one vector of 16 bytes, or two that lie as far
// apart as the units' vectors reach (fp32), so that neighbouring lanes' vectors are neighbours in memory; and under half
// pairing the partners of the vectors that turn.
template <typename T, bool kHalf>
struct NormPlace {
  static constexpr int kVectors = sizeof(T) / 2, kVec = 8 / kVectors;   // vectors of a unit, elements of one
  int u, a0, h0, step;
  int from[kVectors];   // elements from the first vector
  bool two[kVectors];   // it has a partner
  bool on_q, active;
  unsigned mask;
  __device__ __forceinline__ NormPlace(const NormParams& p) {
    const int lanes = 1 << p.log_lanes, slot = threadIdx.x >> p.log_lanes, lane = threadIdx.x & 31;
    u = threadIdx.x & (lanes - 1);
    on_q = slot < p.q.slots;
    active = u < p.units && slot < p.q.slots + p.k.slots;
    const int slots = on_q ? p.q.slots : p.k.slots;
    h0 = (on_q ? slot : slot - p.q.slots) + blockIdx.y * slots;
    step = slots * gridDim.y;
    mask = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1u) << (lane & ~(lanes - 1));
    a0 = start(p, u);
#pragma unroll
    for (int v = 0; v < kVectors; ++v) {
      from[v] = start(p, u + v * p.units) - a0;
      two[v] = kHalf && active && u + v * p.units < p.turned_vectors;
    }
  }
  // the first element of vector x
  static __device__ __forceinline__ int start(const NormParams& p, int x) {
    return kHalf && x >= p.turned_vectors ? 2 * p.pairs + kVec * (x - p.turned_vectors) : kVec * x;
  }
};

__device__ __forceinline__ uint64_t swap_f32x2(uint64_t v) {
  float lo, hi;
  unpack_f32x2(v, lo, hi);
  return pack_f32x2(hi, lo);
}
__device__ __forceinline__ uint64_t neg_f32x2(uint64_t v) { return v ^ 0x8000000080000000ull; }
__device__ __forceinline__ float sum_f32x2(uint64_t v) {
  float lo, hi;
  unpack_f32x2(v, lo, hi);
  return lo + hi;
}
// ------------------------------------------------------------------ forward and gradient
//
// A CTA takes rows blockIdx.x, + gridDim.x, ... (with few rows, of each the share blockIdx.y of its heads).  Each thread
// copies its elements of the next kDepth heads, of this row and those after it, into shared memory of its own ahead of
// their use, without registers and without a barrier; the CTA meets once in one or a few rows, whose angles a warp of its
// own has made.
// In the gradient a thread's sums of the weights' gradient stay in registers over its heads and rows (kNormTerms); each
// CTA leaves one partial sum a side and element, and a second kernel adds those in a fixed order.
template <typename T, NormPairs kPairs, bool kGrad>
struct NormRing {
  static constexpr bool kHalf = kPairs == kPairsVectors;
  static constexpr int kVectors = sizeof(T) / 2;                      // 16-byte vectors of 8 elements
  static constexpr int kParts = (kHalf ? 2 : 1) * (kGrad ? 2 : 1);    // x's first and second halves, dy's
  // rows from one meeting to the next (prompt of 8191 rows 86 us at 1, 93 at 4; its gradient 203 and 155)
  static constexpr int kAngleRows = kGrad ? kNormGradRows : 1;
  static constexpr int kDepth = 16 / (kVectors * (kGrad ? 4 : 2));    // heads ahead: up to 256 bytes a thread
  static constexpr int kVectorBytes = kNormThreads * 16;              // all threads' vector of one part
  static constexpr int kPartBytes = kVectors * kVectorBytes, kStageBytes = kParts * kPartBytes, kBytes = kDepth * kStageBytes;
};

// Eight floats of a lane, two conflict-free vectors `pitch` floats apart, packed in pairs.
__device__ __forceinline__ void load_pairs(const float* from, int pitch, uint64_t (&v)[4]) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(from), b = *reinterpret_cast<const ulonglong2*>(from + pitch);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// The same, read again where it is used again (values kept over a head's sums are registers that spill).
__device__ __forceinline__ void load_pairs_again(const float* from, int pitch, uint64_t (&v)[4]) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "r"(smem_u32(from)));
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[2]), "=l"(v[3]) : "r"(smem_u32(from + pitch)));
}

// kFold: the gradient with sums of many terms (instances of their own: their code costs the others registers).
template <typename T, NormPairs kPairs, bool kGrad, bool kFold>
__global__ void __launch_bounds__(kNormThreads + 32, 2) mfa_norm_rope_kernel(const __grid_constant__ NormParams p) {
  using Ring = NormRing<T, kPairs, kGrad>;
  constexpr bool kHalf = kPairs == kPairsVectors, kFar = kPairs == kPairsFar;
  constexpr int kDepth = Ring::kDepth, kParts = Ring::kParts, kVectors = Ring::kVectors, kAngleRows = Ring::kAngleRows;
  // a lane's four floats lie beside its neighbour's
  __shared__ __align__(16) float cs[2][kAngleRows][2][kRopeMaxDim / 2];
  __shared__ __align__(16) float sw[2][2][kRopeMaxDim / 2];   // [side][first half, second half][2 x 4 floats of a lane]
  extern __shared__ __align__(16) uint8_t ring[];             // stages; at the end the CTA's sums
  grid_dep_wait();
  if constexpr (!kGrad) grid_dep_launch();
  const NormPlace<T, kHalf> at(p);
  const int threads = blockDim.x, tid = threadIdx.x, lanes = 1 << p.log_lanes;
  const int step = at.step, d = p.head_dim;
  // (the last warp has angles in place of heads; what is left of a warp behind the slots has nothing)
  const bool angles = tid >= threads - 32;
  int heads = at.on_q ? p.q.heads : p.k.heads;
  if (angles || tid >= (p.q.slots + p.k.slots) << p.log_lanes || at.h0 >= heads) heads = 0;
  const bool two = kHalf && (at.two[0] || at.two[kVectors - 1]);

  // The head that is copied next; each thread goes over (row, head) by itself.
  const int head_step = step * d;
  long long in_row = blockIdx.x;
  int in_head = at.h0;
  const T* in_x;
  const T* in_dy;
  auto start = [&](long long row) {   // the row's first head of this thread
    const T* x = static_cast<const T*>(at.on_q ? p.q.x : p.k.x);
    in_x = x + row * (at.on_q ? p.q.x_stride : p.k.x_stride) + static_cast<long long>(at.h0) * d + at.a0;
    if constexpr (kGrad) {
      const T* dy = static_cast<const T*>(at.on_q ? p.q.dy : p.k.dy);
      in_dy = dy + row * (at.on_q ? p.q.dy_stride : p.k.dy_stride) + static_cast<long long>(at.h0) * d + at.a0;
    }
  };
  const uint32_t mine = smem_u32(ring) + tid * 16;
  uint32_t in_at = mine;
  const int second = p.pairs;   // from a vector to its partner
  auto copy = [&]() {
    if (in_row < p.rows && heads > 0 && at.active) {
#pragma unroll
      for (int v = 0; v < kVectors; ++v) {
        cp_async_16(in_at + v * Ring::kVectorBytes, in_x + at.from[v]);
        if constexpr (kGrad) cp_async_16(in_at + kParts / 2 * Ring::kPartBytes + v * Ring::kVectorBytes, in_dy + at.from[v]);
        if (at.two[v]) {
          cp_async_16(in_at + Ring::kPartBytes + v * Ring::kVectorBytes, in_x + second + at.from[v]);
          if constexpr (kGrad) cp_async_16(in_at + 3 * Ring::kPartBytes + v * Ring::kVectorBytes, in_dy + second + at.from[v]);
        }
      }
    }
    cp_async_commit();
    in_at = in_at == mine + (kDepth - 1) * Ring::kStageBytes ? mine : in_at + Ring::kStageBytes;
    in_head += step;
    in_x += head_step;
    if constexpr (kGrad) in_dy += head_step;
    if (in_head >= heads) {
      in_head = at.h0;
      in_row += gridDim.x;
      start(in_row);
    }
  };
  const uint8_t* out_at = ring + tid * 16;   // the stage that is used next
  const uint8_t* const out_end = out_at + Ring::kBytes;
  auto partner = [&](int part, int v) { return !(kHalf && part % 2 == 1) || at.two[v]; };
  auto fetch_again = [&](int part) {   // as load_pairs_again
    RopeVec<T, 8> r = {};
#pragma unroll
    for (int v = 0; v < kVectors; ++v) {
      if (!partner(part, v)) continue;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.w[4 * v]), "=r"(r.w[4 * v + 1]), "=r"(r.w[4 * v + 2]), "=r"(r.w[4 * v + 3])
                   : "r"(smem_u32(out_at) + part * Ring::kPartBytes + v * Ring::kVectorBytes));
    }
    return r;
  };
  auto fetch = [&](int part) {
    RopeVec<T, 8> r = {};
#pragma unroll
    for (int v = 0; v < kVectors; ++v) {
      if (!partner(part, v)) continue;
      const uint4 x = *reinterpret_cast<const uint4*>(out_at + part * Ring::kPartBytes + v * Ring::kVectorBytes);
      r.w[4 * v] = x.x, r.w[4 * v + 1] = x.y, r.w[4 * v + 2] = x.z, r.w[4 * v + 3] = x.w;
    }
    return r;
  };
  int far[8];   // of each element's partner, bytes from the group's first lane's
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = kFar ? at.a0 + (kVectors == 2 && i >= 4 ? at.from[kVectors - 1] : 0) + (kVectors == 2 ? i & 3 : i) : 0;
    const int x = e < p.pairs ? e + p.pairs : e < 2 * p.pairs ? e - p.pairs : e;
    const int v = kVectors == 2 && x / 4 >= p.units;
    far[i] = kVectors == 1 ? 2 * x : 4 * x - v * 16 * p.units + v * Ring::kVectorBytes;
  }
  auto fetch_far = [&](int part) {
    const uint8_t* base = out_at - 16 * at.u + part * Ring::kPartBytes;
    RopeVec<T, 8> r;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      if constexpr (kVectors == 1) {
        r.w[i / 2] = *reinterpret_cast<const uint16_t*>(base + far[i]) |
                     static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(base + far[i + 1])) << 16;
      } else {
        r.w[i] = *reinterpret_cast<const uint32_t*>(base + far[i]);
        r.w[i + 1] = *reinterpret_cast<const uint32_t*>(base + far[i + 1]);
      }
    }
    return r;
  };
  if (heads > 0) {
    start(in_row);
#pragma unroll 1
    for (int i = 0; i < kDepth; ++i) copy();
  }
  for (int i = tid; i < 32 * lanes; i += threads) {   // side, half, vector, lane, element
    const int lane = i >> 2, vector = lane >> p.log_lanes;   // (vector: side, half, first or second four elements)
    const int on_k = vector >> 2, half = vector >> 1 & 1, u = lane & (lanes - 1), e = (vector & 1) * 4 + (i & 3);
    const NormSide& side = on_k ? p.k : p.q;
    const int x = kVectors == 2 ? u + (vector & 1) * p.units : u;
    const bool there = side.heads > 0 && u < p.units && (half == 0 || kFar || (kHalf && x < p.turned_vectors));
    int el = at.start(p, x) + (kVectors == 2 ? i & 3 : e);
    if (half) el = kFar && el >= p.pairs ? (el < 2 * p.pairs ? el - p.pairs : el) : el + p.pairs;   // the partner's
    sw[on_k][half][(e / 4 * lanes + u) * 4 + (e & 3)] = there ? norm_weight(p, side, el) : 0.f;
  }
  // half pairing: a lane's eight pairs (or elements) in two groups of four; adjacent: its four together
  auto place = [&](int i) {
    const int x = i / (kPairs != kPairsNext ? at.kVec : at.kVec / 2);   // the pair's vector
    const int v = kVectors == 2 && x >= p.units, u = x - v * p.units;
    if constexpr (kPairs != kPairsNext) return kVectors == 2 ? (v * lanes + u) * 4 + (i & 3) : ((i >> 2 & 1) * lanes + u) * 4 + (i & 3);
    return kVectors == 2 ? 4 * u + 2 * v + (i & 1) : i;
  };
  const long long chunk = static_cast<long long>(kAngleRows) * gridDim.x;
  auto make_angles = [&](long long row, int buffer, int from, int by) {
#pragma unroll 1
    for (int i = 0; i < kAngleRows && row < p.rows; ++i, row += gridDim.x) row_angles<kFar>(p, row, from, by, cs[buffer][i], place);
  };
  make_angles(blockIdx.x, 0, tid, threads);
  __syncthreads();
  const float* my_wa = &sw[at.on_q ? 0 : 1][0][4 * at.u];
  const float* my_wb = &sw[at.on_q ? 0 : 1][1][4 * at.u];
  uint64_t da[4] = {}, db[4] = {};   // the weights' gradient, of this thread's elements
  // Where they are many: the CTA's sums of both sides, in 64 bits, behind the ring.  A warp's threads add theirs to them, its
  // groups in turn, and begin anew; one warp between two meetings.
  double* const sums = reinterpret_cast<double*>(ring + Ring::kBytes);
  if constexpr (kFold) {
    for (int e = tid; e < 2 * d; e += threads) sums[e] = 0.;   // (before the first meeting)
  }
  auto fold = [&]() {
    double* const own = sums + (at.on_q ? 0 : d) + at.a0;
    const int here = (tid >> p.log_lanes) & ((32 >> p.log_lanes) - 1);
#pragma unroll 1
    for (int g = 0; g < 32 >> p.log_lanes; ++g) {
      if (g == here && at.active) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int v = kVectors == 2 ? j / 2 : 0;
          double* const to = own + at.from[v] + (kVectors == 2 ? 2 * (j & 1) : 2 * j);
          float lo, hi;
          unpack_f32x2(da[j], lo, hi);
          to[0] += lo, to[1] += hi;
          if (at.two[v]) {
            unpack_f32x2(db[j], lo, hi);
            to[second] += lo, to[second + 1] += hi;
          }
        }
      }
      __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) da[j] = db[j] = 0;
  };
  [[maybe_unused]] int turn = 0;   // the warp that folds next
  int buffer = 0;
  if (angles) {   // rows ahead, so that their loads' way is nobody's wait
#pragma unroll 1
    for (long long row = blockIdx.x; row < p.rows; row += chunk, buffer ^= 1) {
      make_angles(row + chunk, buffer ^ 1, tid & 31, 32);
      __syncthreads();
    }
  }
  int in_chunk = 0;
#pragma unroll 1
  for (long long row = blockIdx.x; row < p.rows && !angles; row += gridDim.x) {
    T* to = static_cast<T*>(at.on_q ? p.q.out : p.k.out) + row * (at.on_q ? p.q.out_stride : p.k.out_stride) +
            static_cast<long long>(at.h0) * d + at.a0;
    // Half pairing: c and s of the thread's eight pairs (or elements, s with its sign); adjacent: of its four, as (c, c) and (-s, s).
    uint64_t c[4], s[4];
    if constexpr (kPairs != kPairsNext) {
      load_pairs(&cs[buffer][in_chunk][0][4 * at.u], 4 * lanes, c);
      load_pairs(&cs[buffer][in_chunk][1][4 * at.u], 4 * lanes, s);
    } else {
      const float4 x = *reinterpret_cast<const float4*>(&cs[buffer][in_chunk][0][4 * at.u]);
      const float4 y = *reinterpret_cast<const float4*>(&cs[buffer][in_chunk][1][4 * at.u]);
      c[0] = pack_f32x2(x.x, x.x), c[1] = pack_f32x2(x.y, x.y), c[2] = pack_f32x2(x.z, x.z), c[3] = pack_f32x2(x.w, x.w);
      s[0] = pack_f32x2(-y.x, y.x), s[1] = pack_f32x2(-y.y, y.y), s[2] = pack_f32x2(-y.z, y.z), s[3] = pack_f32x2(-y.w, y.w);
    }
    // Forward: c and s times the weights.  Half pairing: y = r (a ac + b bs), r (b bc + a as), with bs negated;
    // else: y = r ((x0, x1) ac + (x0's partner, x1's) bs).
    uint64_t ac[4], as[4], bc[4], bs[4];
    if constexpr (!kGrad) {
      load_pairs(my_wa, 4 * lanes, ac);
      if constexpr (kPairs != kPairsNext) load_pairs(my_wb, 4 * lanes, bc);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kFar) {
          bs[j] = mul_f32x2(bc[j], s[j]);
        } else if constexpr (kHalf) {
          as[j] = mul_f32x2(ac[j], s[j]);
          bs[j] = neg_f32x2(mul_f32x2(bc[j], s[j]));
          bc[j] = mul_f32x2(bc[j], c[j]);
        } else {
          bs[j] = mul_f32x2(swap_f32x2(ac[j]), s[j]);
        }
        ac[j] = mul_f32x2(ac[j], c[j]);
      }
    }
    // Lanes with 8 bf16 elements of a head: two heads at a time, so that one's waits are the other's work (8191 rows of 68 heads
    // of 128, adjacent, 53 us in place of 63; with 16 elements 57 in place of 55).
    constexpr bool kTwo = !kGrad && !kHalf && kVectors == 1;
    if constexpr (kTwo) {
#pragma unroll 1
      for (int h = at.h0; h < heads; h += 2 * step, to += 2 * head_step) {
        cp_async_wait<kDepth - 2>();
        if constexpr (kFar) __syncwarp(at.mask);   // the group's copies
        const bool second_head = h + step < heads;
        const uint8_t* const first_at = out_at;
        RopeVec<T, 8> a[2], b[2];
        float sum[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {   // (a second head that is not there: the next row's, and nothing is written)
          if (k == 1) out_at = out_at + Ring::kStageBytes == out_end ? out_end - Ring::kBytes : out_at + Ring::kStageBytes;
          a[k] = fetch(0);
          if constexpr (kFar) b[k] = fetch_far(0);
          uint64_t sq = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) sq = fma_f32x2(a[k].pair(2 * j), a[k].pair(2 * j), sq);
          sum[k] = at.active ? sum_f32x2(sq) : 0.f;
        }
        group_sum<2>(sum, at.mask, lanes);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float r = rsqrtf(fmaf(sum[k], p.inv_dim, p.eps));
          const uint64_t r2 = pack_f32x2(r, r);
          RopeVec<T, 8> y;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t u = mul_f32x2(a[k].pair(2 * j), r2);
            y.set_pair(2 * j, fma_f32x2(u, ac[j], mul_f32x2(kFar ? mul_f32x2(b[k].pair(2 * j), r2) : swap_f32x2(u), bs[j])));
          }
          if (at.active && (k == 0 || second_head)) y.store_raw(to + k * head_step);
        }
        if constexpr (kFar) __syncwarp(at.mask);   // (read by all)
        copy();   // into the stages that were read
        if (second_head) {
          copy();
          out_at = out_at + Ring::kStageBytes == out_end ? out_end - Ring::kBytes : out_at + Ring::kStageBytes;
        } else {
          out_at = first_at + Ring::kStageBytes == out_end ? out_end - Ring::kBytes : first_at + Ring::kStageBytes;
        }
      }
    }
#pragma unroll 1
    for (int h = at.h0; !kTwo && h < heads; h += step, to += head_step) {
      cp_async_wait<kDepth - 1>();
      if constexpr (kFar) __syncwarp(at.mask);   // the group's copies
      const RopeVec<T, 8> a = fetch(0);
      RopeVec<T, 8> b = {};
      if (two) b = fetch(1);
      if constexpr (kFar && !kGrad) b = fetch_far(0);
      uint64_t sq = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sq = fma_f32x2(a.pair(2 * j), a.pair(2 * j), sq);
        if constexpr (kHalf) sq = fma_f32x2(b.pair(2 * j), b.pair(2 * j), sq);
      }
      RopeVec<T, 8> y, z;
      if constexpr (!kGrad) {
        float sum[1] = {at.active ? sum_f32x2(sq) : 0.f};
        group_sum<1>(sum, at.mask, lanes);
        const float r = rsqrtf(fmaf(sum[0], p.inv_dim, p.eps));
        const uint64_t r2 = pack_f32x2(r, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t u = mul_f32x2(a.pair(2 * j), r2);
          if constexpr (kHalf) {
            const uint64_t v = mul_f32x2(b.pair(2 * j), r2);
            y.set_pair(2 * j, fma_f32x2(u, ac[j], mul_f32x2(v, bs[j])));
            z.set_pair(2 * j, fma_f32x2(v, bc[j], mul_f32x2(u, as[j])));
          } else {
            y.set_pair(2 * j, fma_f32x2(u, ac[j], mul_f32x2(kFar ? mul_f32x2(b.pair(2 * j), r2) : swap_f32x2(u), bs[j])));
          }
        }
      } else {
        // g: dy turned back; sums of x^2 and, with u = g w, of u x
        uint64_t g[4], k[4], wa[4], wb[4], ux = 0;
        const RopeVec<T, 8> ga = fetch(kParts / 2);
        RopeVec<T, 8> gb = {};
        if (two) gb = fetch(kParts / 2 + 1);
        if constexpr (kFar) gb = fetch_far(kParts / 2);
        load_pairs(my_wa, 4 * lanes, wa);
        if constexpr (kHalf) load_pairs(my_wb, 4 * lanes, wb);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t x = ga.pair(2 * j);
          if constexpr (kHalf) {
            const uint64_t v = gb.pair(2 * j);
            g[j] = fma_f32x2(x, c[j], mul_f32x2(v, s[j]));
            k[j] = fma_f32x2(v, c[j], neg_f32x2(mul_f32x2(x, s[j])));
            ux = fma_f32x2(mul_f32x2(k[j], wb[j]), b.pair(2 * j), ux);
          } else {
            g[j] = fma_f32x2(x, c[j], neg_f32x2(mul_f32x2(kFar ? gb.pair(2 * j) : swap_f32x2(x), s[j])));
          }
          ux = fma_f32x2(mul_f32x2(g[j], wa[j]), a.pair(2 * j), ux);
        }
        float sum[2] = {at.active ? sum_f32x2(sq) : 0.f, at.active ? sum_f32x2(ux) : 0.f};
        group_sum<2>(sum, at.mask, lanes);
        const float r = rsqrtf(fmaf(sum[0], p.inv_dim, p.eps));
        const float m = r * (r * (r * (sum[1] * p.inv_dim)));   // dx = r u - x m
        const uint64_t r2 = pack_f32x2(r, r), m2 = pack_f32x2(-m, -m);
        const RopeVec<T, 8> a = fetch_again(0);
        RopeVec<T, 8> b = {};
        if (two) b = fetch_again(1);
        load_pairs_again(my_wa, 4 * lanes, wa);
        if constexpr (kHalf) load_pairs_again(my_wb, 4 * lanes, wb);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t x = a.pair(2 * j), gr = mul_f32x2(g[j], r2);
          y.set_pair(2 * j, fma_f32x2(gr, wa[j], mul_f32x2(x, m2)));
          da[j] = fma_f32x2(gr, x, da[j]);
          if constexpr (kHalf) {
            const uint64_t v = b.pair(2 * j), kr = mul_f32x2(k[j], r2);
            z.set_pair(2 * j, fma_f32x2(kr, wb[j], mul_f32x2(v, m2)));
            db[j] = fma_f32x2(kr, v, db[j]);
          }
        }
      }
      if (at.active) {
#pragma unroll
        for (int v = 0; v < kVectors; ++v) {
          *reinterpret_cast<uint4*>(to + at.from[v]) = make_uint4(y.w[4 * v], y.w[4 * v + 1], y.w[4 * v + 2], y.w[4 * v + 3]);
          if (at.two[v])
            *reinterpret_cast<uint4*>(to + second + at.from[v]) = make_uint4(z.w[4 * v], z.w[4 * v + 1], z.w[4 * v + 2], z.w[4 * v + 3]);
        }
      }
      if constexpr (kFar) __syncwarp(at.mask);   // (read by all)
      copy();   // into the stage that was read
      out_at = out_at + Ring::kStageBytes == out_end ? out_end - Ring::kBytes : out_at + Ring::kStageBytes;
    }
    if (++in_chunk == kAngleRows || row + gridDim.x >= p.rows) {
      __syncthreads();   // the next rows' angles are there, and these rows' may be written over
      in_chunk = 0;
      buffer ^= 1;
      if constexpr (kFold) {
        if (turn == tid >> 5) fold();
        if (++turn == p.fold) turn = 0;
      }
    }
  }
  if constexpr (kGrad) {
    grid_dep_launch();
    cp_async_wait<0>();   // (copies past the last row are empty)
    // the CTA's sums: over the slots of a side, in order
    float* red = reinterpret_cast<float*>(ring);
    float* own = red + (tid >> p.log_lanes) * d + at.a0;
    __syncthreads();
    if (at.active) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int v = kVectors == 2 ? j / 2 : 0;
        float* to = own + at.from[v] + (kVectors == 2 ? 2 * (j & 1) : 2 * j);
        *reinterpret_cast<uint64_t*>(to) = da[j];
        if (at.two[v]) *reinterpret_cast<uint64_t*>(to + second) = db[j];
      }
    }
    __syncthreads();
    for (int e = tid; e < 2 * d; e += threads) {
      const bool on_k = e >= d;
      const int from = on_k ? p.q.slots : 0, to = on_k ? p.q.slots + p.k.slots : p.q.slots;
      float v = 0.f;
      for (int x = from; x < to; ++x) v += red[x * d + (on_k ? e - d : e)];
      if constexpr (kFold) v = static_cast<float>(sums[e] + v);
      p.partial[(static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * d + e] = v;
    }
  }
}

// The weights' gradient: partial sums of the CTAs, 8 elements a CTA, 32 threads for each, in a fixed order.
__global__ void __launch_bounds__(256) mfa_norm_rope_weights_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[32][9];
  grid_dep_wait();
  grid_dep_launch();
  const int el = blockIdx.x * 8 + (threadIdx.x & 7), part = threadIdx.x >> 3;
  float of[MFA_NORM_ROPE_GRAD_PARTS / 32], v = 0.f;   // (all loads on their way at once)
#pragma unroll
  for (int k = 0; k < MFA_NORM_ROPE_GRAD_PARTS / 32; ++k) {
    const int i = part + 32 * k;
    of[k] = el < 2 * p.head_dim && i < p.parts ? p.partial[static_cast<size_t>(i) * 2 * p.head_dim + el] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < MFA_NORM_ROPE_GRAD_PARTS / 32; ++k) v += of[k];
  red[part][threadIdx.x & 7] = v;
  __syncthreads();
  if (part != 0 || el >= 2 * p.head_dim) return;
  float sum = 0.f;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) sum += red[i][threadIdx.x];
  float* to = p.dw[el >= p.head_dim];
  if (to != nullptr) to[el >= p.head_dim ? el - p.head_dim : el] = sum;
}

// ------------------------------------------------------------------ any shape
//
// Heads of odd sizes or too many units, unaligned rows: a warp a head, a lane its every 32nd element and that element's
// partner in the pair.  Bound by its loads' latency: 2000 rows of 26 heads of 256, 100 elements turned, half pairing,
// gradient: 72 us (184 with registers for heads of 512, one CTA on an SM; 31 on the wide path).
template <typename T, bool kGrad, bool kFold, int kEach>
__global__ void __launch_bounds__(kNormAnyThreads, kEach <= 8 ? 3 : 1) mfa_norm_rope_any_kernel(const __grid_constant__ NormParams p) {
  __shared__ __align__(16) float cs[2][2][kRopeMaxDim / 2];
  // gradient: [warps][head_dim], sums of many terms in 64 bits
  extern __shared__ __align__(16) uint8_t any_smem[];
  float* const red = reinterpret_cast<float*>(any_smem);
  const int pitch = kFold ? 2 * p.head_dim : p.head_dim;   // of red: a warp's sums lie where its 64 bits were
  grid_dep_wait();
  if constexpr (!kGrad) grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool on_q = warp < p.q.slots;
  const NormSide& side = on_q ? p.q : p.k;
  const int h0 = on_q ? warp : warp - p.q.slots, step = side.slots;
  const int r2 = 2 * p.pairs;
  float dw[kEach] = {};
  // where a thread's sums are many: the sum of them, in 64 bits, as on the wide path
  double* const sums = reinterpret_cast<double*>(any_smem) + warp * p.head_dim + lane;
  auto fold = [&](bool first) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (lane + 32 * i < p.head_dim) sums[32 * i] = first ? 0. : sums[32 * i] + dw[i];
      dw[i] = 0.f;
    }
  };
  if constexpr (kFold) fold(true);
  [[maybe_unused]] int to_fold = p.fold;
  int buffer = 0;
#pragma unroll 1
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, buffer ^= 1) {
    row_angles<false>(p, row, threadIdx.x, blockDim.x, cs[buffer], [](int i) { return i; });
    __syncthreads();
    const T* xs = static_cast<const T*>(side.x) + row * side.x_stride;
    const T* dys = static_cast<const T*>(side.dy) + row * side.dy_stride;
    T* dst = static_cast<T*>(side.out) + row * side.out_stride;
#pragma unroll 1
    for (long long h = h0; h < side.heads; h += step) {
      const T* x = xs + h * p.head_dim;
      float own[kEach], out[kEach], sum[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int e = lane + 32 * i;
        own[i] = out[i] = 0.f;
        if (e >= p.head_dim) continue;
        own[i] = norm_load<T>(x, e);
        sum[0] = fmaf(own[i], own[i], sum[0]);
        int other = e, pair = 0;
        float sign = 0.f;
        if (e < r2) {
          const bool first = p.half ? e < p.pairs : (e & 1) == 0;
          other = p.half ? (first ? e + p.pairs : e - p.pairs) : e ^ 1;
          pair = p.half ? (first ? e : e - p.pairs) : e >> 1;
          sign = first ? -1.f : 1.f;
        }
        const float c = e < r2 ? cs[buffer][0][pair] : 1.f, s = e < r2 ? cs[buffer][1][pair] * sign : 0.f;
        if constexpr (kGrad) {   // g, the turn back
          const T* dy = dys + h * p.head_dim;
          out[i] = norm_load<T>(dy, e) * c - norm_load<T>(dy, other) * s;
          sum[1] = fmaf(out[i] * norm_weight(p, side, e), own[i], sum[1]);
        } else {
          out[i] = own[i] * norm_weight(p, side, e) * c + norm_load<T>(x, other) * norm_weight(p, side, other) * s;
        }
      }
      group_sum<2>(sum, 0xffffffffu, 32);
      __syncwarp();   // in place: every lane has read its elements and their partners before any is written
      const float r = rsqrtf(fmaf(sum[0], p.inv_dim, p.eps)), m = r * r * sum[1] * p.inv_dim;
      T* to = dst + h * p.head_dim;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int e = lane + 32 * i;
        if (e >= p.head_dim) continue;
        if constexpr (kGrad) {
          norm_store(to + e, r * (out[i] * norm_weight(p, side, e) - own[i] * m));
          dw[i] = fmaf(out[i], own[i] * r, dw[i]);
        } else {
          norm_store(to + e, r * out[i]);
        }
      }
    }
    if constexpr (kFold) {
      if (--to_fold == 0) {
        fold(false);
        to_fold = p.fold;
      }
    }
  }
  if constexpr (kGrad) {
    grid_dep_launch();
    if constexpr (kFold) {
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (lane + 32 * i < p.head_dim) dw[i] = static_cast<float>(sums[32 * i] + dw[i]);
      __syncwarp();   // every lane has read its sums
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = lane + 32 * i;
      if (e < p.head_dim) red[warp * pitch + e] = dw[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * p.head_dim; e += blockDim.x) {
      const bool on_k = e >= p.head_dim;
      const int from = on_k ? p.q.slots : 0, to = on_k ? p.q.slots + p.k.slots : p.q.slots;
      float v = 0.f;
      for (int x = from; x < to; ++x) v += red[x * pitch + (on_k ? e - p.head_dim : e)];
      p.partial[static_cast<size_t>(blockIdx.x) * 2 * p.head_dim + e] = v;
    }
  }
}

// ------------------------------------------------------------------ host side

// One side's rows as both calls take them (dy null: the forward pass).
static mfa_status check_norm_side(const NormSide& s, const mfa_rope_config* c, int rows, int esz, bool grad) {
  if (s.heads < 0 || s.heads > INT_MAX / 4 / kRopeMaxDim) return MFA_ERR_INVALID_ARG;
  if (s.heads == 0 || rows == 0) return MFA_OK;
  if (s.x == nullptr || s.out == nullptr || s.w == nullptr || (grad && s.dy == nullptr)) return MFA_ERR_INVALID_ARG;
  if (!aligned(s.x, esz) || !aligned(s.out, esz) || (grad && !aligned(s.dy, esz))) return MFA_ERR_INVALID_ARG;
  const int64_t least = static_cast<int64_t>(s.heads) * c->head_dim;
  const int64_t most = (int64_t{1} << 58) / rows;   // rows * stride * size stays inside 64 bits
  if (s.x_stride < least || s.out_stride < least || s.x_stride > most || s.out_stride > most) return MFA_ERR_INVALID_ARG;
  if (grad && (s.dy_stride < least || s.dy_stride > most)) return MFA_ERR_INVALID_ARG;
  // what is written is an input's own rows, or shares nothing with it
  auto clear = [&](const void* in, int64_t stride) {
    if (in == s.out) return stride == s.out_stride;
    return !rows_share(in, stride, least, s.out, s.out_stride, least, rows, esz);
  };
  return clear(s.x, s.x_stride) && (!grad || clear(s.dy, s.dy_stride)) ? MFA_OK : MFA_ERR_INVALID_ARG;
}

static bool wide_norm_side(const NormSide& s, bool grad) {
  return s.heads == 0 || (aligned(s.x, 16) && aligned(s.out, 16) && s.x_stride % 8 == 0 && s.out_stride % 8 == 0 &&
                          (!grad || (aligned(s.dy, 16) && s.dy_stride % 8 == 0)));
}

// Groups of lanes (or warps) for the sides' heads: one each, or, of what a CTA has room for, a share by their heads.
// (Fewer, with four heads each, leave CTAs of 17 groups of 8 lanes: 8191 rows of 68 heads of 128 66 us against 55, their
// gradient 121 against 96.)
static void norm_slots(NormParams& p, int room) {
  const int hq = p.q.heads, hk = p.k.heads;
  int nq = hq, nk = hk;
  if (nq + nk > room) {
    nk = hk == 0 ? 0 : std::max(1, static_cast<int>(static_cast<long long>(room) * hk / (hq + hk)));
    nk = hq == 0 ? room : std::min(nk, room - 1);
    nq = room - nk;
    // no more than the rounds need
    if (nq > 0) nq = (hq + (hq + nq - 1) / nq - 1) / ((hq + nq - 1) / nq);
    if (nk > 0) nk = (hk + (hk + nk - 1) / nk - 1) / ((hk + nk - 1) / nk);
  }
  p.q.slots = nq;
  p.k.slots = nk;
}

// The wide path's kernel, and its shared memory in cfg.
template <typename T, NormPairs kPairs>
static void (*wide_norm(const NormParams& p, bool grad, cudaLaunchConfig_t& cfg))(NormParams) {
  cfg.dynamicSmemBytes = grad ? NormRing<T, kPairs, true>::kBytes : NormRing<T, kPairs, false>::kBytes;
  if (p.fold > 0) cfg.dynamicSmemBytes += 16 * static_cast<size_t>(p.head_dim);
  return p.fold > 0 ? mfa_norm_rope_kernel<T, kPairs, true, true>
         : grad     ? mfa_norm_rope_kernel<T, kPairs, true, false>
                    : mfa_norm_rope_kernel<T, kPairs, false, false>;
}
template <typename T>
static void (*wide_norm(NormPairs pairs, const NormParams& p, bool grad, cudaLaunchConfig_t& cfg))(NormParams) {
  return pairs == kPairsNext      ? wide_norm<T, kPairsNext>(p, grad, cfg)
         : pairs == kPairsVectors ? wide_norm<T, kPairsVectors>(p, grad, cfg)
                                  : wide_norm<T, kPairsFar>(p, grad, cfg);
}

// The kernel for any shape: a lane's elements of a head (up to 256: fewer registers, three CTAs on an SM).
template <typename T, int kEach>
static void (*any_norm(bool grad, bool fold))(NormParams) {
  return fold   ? mfa_norm_rope_any_kernel<T, true, true, kEach>
         : grad ? mfa_norm_rope_any_kernel<T, true, false, kEach>
                : mfa_norm_rope_any_kernel<T, false, false, kEach>;
}
template <typename T>
static void (*any_norm(const NormParams& p, bool grad))(NormParams) {
  return p.head_dim <= 256 ? any_norm<T, 8>(grad, p.fold > 0) : any_norm<T, 16>(grad, p.fold > 0);
}

// cudaFuncSetAttribute for a wide kernel's dynamic shared memory, once per device and kernel.
static mfa_status ensure_norm_smem(int i, const void* fn, int dev) {
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> done[18][kMaxDevices];
  const bool cacheable = dev >= 0 && dev < kMaxDevices;
  if (cacheable && done[i][dev].load(std::memory_order_acquire)) return MFA_OK;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormThreads * 256 + 16 * kRopeMaxDim);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  if (cacheable) done[i][dev].store(true, std::memory_order_release);
  return MFA_OK;
}

static mfa_status launch_norm(const mfa_rope_config* c, const mfa_rope_pair* table, const int32_t* positions, int32_t num_rows,
                              int32_t dtype, const mfa_norm* norm, NormSide q, NormSide k, bool grad, float* const (&dw)[2],
                              void* workspace, uint64_t workspace_bytes, void* stream) {
  mfa_status st = check_rope(c);
  if (st != MFA_OK) return st;
  if (num_rows < 0 || (dtype != MFA_OUT_BF16 && dtype != MFA_OUT_FP32) || norm == nullptr) return MFA_ERR_INVALID_ARG;
  if (!(std::isfinite(norm->eps) && norm->eps > 0.f)) return MFA_ERR_INVALID_ARG;
  if (norm->weight_dtype != MFA_OUT_BF16 && norm->weight_dtype != MFA_OUT_FP32) return MFA_ERR_INVALID_ARG;
  const int esz = dtype == MFA_OUT_BF16 ? 2 : 4, wsz = norm->weight_dtype == MFA_OUT_BF16 ? 2 : 4;
  q.w = norm->q_weight;
  k.w = norm->k_weight;
  if ((st = check_norm_side(q, c, num_rows, esz, grad)) != MFA_OK || (st = check_norm_side(k, c, num_rows, esz, grad)) != MFA_OK)
    return st;
  if ((q.w && !aligned(q.w, wsz)) || (k.w && !aligned(k.w, wsz))) return MFA_ERR_INVALID_ARG;
  const long long heads = static_cast<long long>(q.heads) + k.heads;
  const bool run = num_rows > 0 && heads > 0;
  if (run && q.heads > 0 && k.heads > 0) {   // what one side writes is neither read nor written by the other
    const int64_t nq = static_cast<int64_t>(q.heads) * c->head_dim, nk = static_cast<int64_t>(k.heads) * c->head_dim;
    auto meet = [&](const void* a, int64_t sa, int64_t na, const void* b, int64_t sb, int64_t nb) {
      return rows_share(a, sa, na, b, sb, nb, num_rows, esz);
    };
    if (meet(q.out, q.out_stride, nq, k.x, k.x_stride, nk) || meet(q.out, q.out_stride, nq, k.out, k.out_stride, nk) ||
        meet(q.x, q.x_stride, nq, k.out, k.out_stride, nk))
      return MFA_ERR_INVALID_ARG;
    if (grad && (meet(q.out, q.out_stride, nq, k.dy, k.dy_stride, nk) || meet(q.dy, q.dy_stride, nq, k.out, k.out_stride, nk)))
      return MFA_ERR_INVALID_ARG;
  }
  if (run && (table == nullptr || positions == nullptr || !aligned(table, 16) || !aligned(positions, 4))) return MFA_ERR_INVALID_ARG;
  if (grad) {
    if ((dw[0] && !aligned(dw[0], 4)) || (dw[1] && !aligned(dw[1], 4)) || (dw[0] && dw[0] == dw[1])) return MFA_ERR_INVALID_ARG;
    if (run && (workspace == nullptr || !aligned(workspace, 16))) return MFA_ERR_INVALID_ARG;
    if (run && workspace_bytes < MFA_NORM_ROPE_GRAD_BYTES(c->head_dim)) return MFA_ERR_WORKSPACE;
  }
  if (!run && !(grad && (dw[0] || dw[1]))) return MFA_OK;
  const bool half = c->pairing == MFA_ROPE_HALF;
  NormParams p = {};
  p.q = q;
  p.k = k;
  p.table = table;
  p.positions = positions;
  p.rows = num_rows;
  p.axes = c->num_axes;
  p.pairs = c->rotary_dim / 2;
  p.head_dim = c->head_dim;
  p.half = half;
  p.w_f32 = wsz == 4;
  p.eps = norm->eps;
  p.inv_dim = 1.f / static_cast<float>(c->head_dim);
  p.partial = static_cast<float*>(workspace);
  p.dw[0] = dw[0];
  p.dw[1] = dw[1];
  const NormPairs pairs = !half ? kPairsNext : c->rotary_dim % 16 == 0 ? kPairsVectors : kPairsFar;
  p.turned_vectors = pairs == kPairsVectors ? p.pairs / (16 / esz) : 0;
  p.units = (c->head_dim - (pairs == kPairsVectors ? p.pairs : 0)) / 8;
  while ((1 << p.log_lanes) < p.units) ++p.log_lanes;
  // (what is left of the last turned vector turns by nothing)
  const bool wide = c->head_dim % 8 == 0 && p.log_lanes <= 5 && wide_norm_side(q, grad) && wide_norm_side(k, grad);
  p.angles = wide ? (half ? 8 : 4) * p.units : p.pairs;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  const bool bf16 = dtype == MFA_OUT_BF16;
  if (run) {
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return cuda_fail(e, "cudaDeviceGetAttribute");
    int ctas = std::min({num_rows, 2 * sms, MFA_NORM_ROPE_GRAD_PARTS});
    int shares = 1;
    void (*fn)(NormParams);
    // Where a thread's sum of the weights' gradient would have too many terms: the times between two folds of a warp's sums,
    // each time after so many rows, and at least so many times (for as many warps to take turns).
    auto set_fold = [&](int rows_at_once, int least) {
      auto each = [&](int heads, int slots) { return slots > 0 ? (heads + slots * shares - 1) / (slots * shares) : 0; };
      const int row = std::max(each(q.heads, p.q.slots), each(k.heads, p.k.slots));   // a row's terms
      if (grad && (static_cast<long long>(num_rows) + ctas - 1) / ctas * row > kNormTerms)
        p.fold = std::max(least, kNormTerms / row / rows_at_once);
    };
    if (wide) {
      norm_slots(p, kNormThreads >> p.log_lanes);
      // few rows: a row's heads shared by CTAs, as far as there is room and each slot has a head
      const int rounds = std::max(p.q.slots ? (q.heads + p.q.slots - 1) / p.q.slots : 1,
                                  p.k.slots ? (k.heads + p.k.slots - 1) / p.k.slots : 1);
      shares = std::max(1, std::min({rounds, std::min(2 * sms, MFA_NORM_ROPE_GRAD_PARTS) / ctas, 65535}));
      cfg.blockDim = dim3(static_cast<unsigned>((((p.q.slots + p.k.slots) << p.log_lanes) + 31) / 32 * 32 + 32), 1, 1);
      set_fold(kNormGradRows, static_cast<int>(cfg.blockDim.x) / 32 - 1);
      fn = bf16 ? wide_norm<__nv_bfloat16>(pairs, p, grad, cfg) : wide_norm<float>(pairs, p, grad, cfg);
      st = ensure_norm_smem((bf16 ? 0 : 9) + 3 * pairs + grad + (p.fold > 0), reinterpret_cast<const void*>(fn), dev);
      if (st != MFA_OK) return st;
    } else {
      norm_slots(p, kNormAnyThreads / 32);
      cfg.blockDim = dim3(static_cast<unsigned>((p.q.slots + p.k.slots) * 32), 1, 1);
      ctas = std::min(num_rows, grad ? std::min(3 * sms, MFA_NORM_ROPE_GRAD_PARTS) : 6 * sms);
      set_fold(1, 1);
      fn = bf16 ? any_norm<__nv_bfloat16>(p, grad) : any_norm<float>(p, grad);
      if (grad)   // (8 warps x 512 at most: 32 KB beside the kernel's own 4)
        cfg.dynamicSmemBytes = static_cast<size_t>(p.q.slots + p.k.slots) * p.head_dim * (p.fold > 0 ? 8 : 4);
    }
    p.parts = grad ? ctas * shares : 0;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(shares), 1);
    if ((e = cudaLaunchKernelEx(&cfg, fn, p)) != cudaSuccess) return cuda_fail(e, "norm rope launch");
  }
  if (grad && (dw[0] || dw[1])) {
    cfg.gridDim = dim3(static_cast<unsigned>((2 * p.head_dim + 7) / 8), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    if ((e = cudaLaunchKernelEx(&cfg, mfa_norm_rope_weights_kernel, p)) != cudaSuccess) return cuda_fail(e, "norm rope weights launch");
  }
  return MFA_OK;
}

}  // namespace mfa

using namespace mfa;

extern "C" mfa_status mfa_norm_rope_run(const mfa_rope_config* c, const mfa_rope_pair* table, const int32_t* positions,
                                        int32_t num_rows, int32_t dtype, const mfa_norm* norm, const mfa_rope_rows* q,
                                        const mfa_rope_rows* k, void* stream) {
  auto side = [](const mfa_rope_rows* s) {
    NormSide r = {};
    if (s != nullptr) {
      r.x = s->in, r.out = s->out, r.x_stride = s->in_stride, r.out_stride = s->out_stride, r.heads = s->heads;
    }
    return r;
  };
  float* const none[2] = {nullptr, nullptr};
  return launch_norm(c, table, positions, num_rows, dtype, norm, side(q), side(k), false, none, nullptr, 0, stream);
}

extern "C" mfa_status mfa_norm_rope_grad_run(const mfa_rope_config* c, const mfa_rope_pair* table, const int32_t* positions,
                                             int32_t num_rows, int32_t dtype, const mfa_norm* norm, const mfa_norm_grad_rows* q,
                                             const mfa_norm_grad_rows* k, float* q_weight_grad, float* k_weight_grad,
                                             void* workspace, uint64_t workspace_bytes, void* stream) {
  auto side = [](const mfa_norm_grad_rows* s) {
    NormSide r = {};
    if (s != nullptr) {
      r.x = s->x, r.dy = s->dy, r.out = s->dx;
      r.x_stride = s->x_stride, r.dy_stride = s->dy_stride, r.out_stride = s->dx_stride, r.heads = s->heads;
    }
    return r;
  };
  float* const dw[2] = {q_weight_grad, k_weight_grad};
  return launch_norm(c, table, positions, num_rows, dtype, norm, side(q), side(k), true, dw, workspace, workspace_bytes, stream);
}
