// Rotary positions with several axes for query heads and new key rows (GB300, sm_103a).
//
// Pair i of a head turns by the angle position[axis(i)] * frequency(i):
//     a' = a cos - b sin,   b' = b cos + a sin.
// Angles: the table holds each frequency as a 64-bit fraction of a turn, rounded to nearest, and
// position times fraction modulo 2^64 is the angle modulo one turn in two integer multiplies, off by
// 2^-34 of a turn at most at any 32-bit position; sincospif of its top 32 bits (2^-32 of a turn)
// gives cos and sin to fp32.  (A product in fp32 is off by 2^-24 of the whole angle, 0.008 rad at
// position 131072; a table made in doubles by 2^-20 of a turn at 2^31, stretched 16 times.)
//
// Every element is read once and written once, with some 3 operations for each: HBM-bound for
// a prompt, launch-bound for a decode step.  A CTA turns all heads of one row, so that the
// row's angles are computed once, by as many threads as there are pairs, and shared; each
// thread owns one place in a head (8 elements of a pair's first half and 8 of its second) and
// keeps its 8 cosines and sines in registers over its heads.  The loads of all its heads go
// out before the angles are computed.
//
// Measured: 8191 rows of 64 + 1 heads of 256 (545 MB) 79 us, 6.9 TB/s, the copy rate; 4097 rows of
// 64 + 4 heads of 128, 96 of them turned, adjacent pairs (143 MB) 24.5 us, 5.8 TB/s; a decode step's
// 128 rows 2.6 us, of which the copy would take 1.3.  (Loads widened to fp32 as they came took twice
// the registers and 212 us for the first of these.)  In fp32, with two heads a thread in place of
// four: 210 us (5.2 TB/s), 50 us (5.7 TB/s) and 6.7 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "mfa.h"
#include "mfa_host.h"
#include "ptx.cuh"

namespace mfa {

constexpr int kRopeMaxDim = 512;
// heads a thread turns, all loaded before the first is used
template <typename T>
constexpr int kRopeHeads = sizeof(T) == 2 ? 4 : 2;
constexpr int kRopeMaxThreads = 512;

struct RopeSide {
  const void* in;
  void* out;
  long long in_stride, out_stride;
  int heads;
};

struct RopeParams {
  RopeSide q, k;
  const mfa_rope_pair* table;
  const int32_t* positions;
  int rows, axes, pairs, head_dim;
  int turned_units, units;   // a head's units: turned ones first, then (out of place) copied ones
  int inverse;
};

// kVec elements as they lie in memory (widened when they are used: a thread holds its heads'
// loads in half the registers)
template <typename T, int kVec>
struct RopeVec {
  static constexpr int kWords = kVec == 8 ? kVec * sizeof(T) / 4 : kVec;
  uint32_t w[kWords];   // kVec = 1: one element in the low bits
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kVec == 8) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
        w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
      }
    } else if constexpr (sizeof(T) == 2) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  }
  __device__ __forceinline__ void store_raw(T* p) const {
    if constexpr (kVec == 8) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
    } else {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(w[i]);
    else
      return __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  // the pair of values i, i + 1 (kVec = 1: lo alone)
  __device__ __forceinline__ void set(int i, float lo, float hi) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(lo);
      if constexpr (kVec > 1) w[i + 1] = __float_as_uint(hi);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
      w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};

// kVec = 8: a unit is 8 elements of the first half and the 8 of the second that pair with them
// (half pairing), or 8 elements of 4 adjacent pairs; kVec = 1: one pair.  threadIdx.x is the
// unit, threadIdx.y and blockIdx.y the heads, blockIdx.x the row.
template <typename T, int kVec, bool kHalf>
__global__ void __launch_bounds__(kRopeMaxThreads) mfa_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr bool kTwo = kHalf || kVec == 1;            // a unit is two vectors, else one
  constexpr int kPairs = kTwo ? kVec : kVec / 2;       // pairs of a unit
  __shared__ __align__(16) float cs[2][kRopeMaxDim / 2];
  grid_dep_wait();
  grid_dep_launch();
  const int u = threadIdx.x;
  const bool turned = u < p.turned_units;
  const long long row = blockIdx.x;
  // offset of the unit's first and second vector in its head
  int a0, b0;
  if (turned) {
    a0 = kHalf ? kVec * u : (kVec == 1 ? 2 * u : kVec * u);
    b0 = kHalf ? a0 + p.pairs : a0 + 1;
  } else {
    a0 = 2 * p.pairs + (u - p.turned_units) * kVec;
    b0 = a0;
  }
  constexpr int kN = kRopeHeads<T>;
  RopeVec<T, kVec> a[kN], b[kN];
  const int heads = p.q.heads + p.k.heads;
  const int h0 = blockIdx.y * (blockDim.y * kN) + threadIdx.y;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int h = h0 + i * blockDim.y;
    if (h < heads) {
      const bool is_q = h < p.q.heads;
      const T* src = static_cast<const T*>(is_q ? p.q.in : p.k.in) + row * (is_q ? p.q.in_stride : p.k.in_stride) +
                     static_cast<long long>(is_q ? h : h - p.q.heads) * p.head_dim;
      a[i].load(src + a0);
      if (kTwo && turned) b[i].load(src + b0);
    }
  }
  {
    int32_t pos[MFA_ROPE_MAX_AXES];
#pragma unroll
    for (int x = 0; x < MFA_ROPE_MAX_AXES; ++x)
      pos[x] = x < p.axes ? p.positions[static_cast<long long>(x) * p.rows + row] : 0;
    for (int i = threadIdx.y * blockDim.x + u; i < p.pairs; i += blockDim.x * blockDim.y) {
      const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(p.table + i);
      const int axis = static_cast<int>(e.y & 3u);
      const int32_t at = axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
      const uint64_t turn = e.x * static_cast<uint64_t>(static_cast<int64_t>(at));
      // the top 32 bits as a signed fraction in [-1/2, 1/2) turns; 2^-31 of it is half turns
      const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;
      float s, c;
      sincospif(half_turns, &s, &c);
      cs[0][i] = c;
      cs[1][i] = p.inverse ? -s : s;
    }
  }
  __syncthreads();
  float c[kPairs], s[kPairs];
  if (turned) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      c[i] = cs[0][kPairs * u + i];
      s[i] = cs[1][kPairs * u + i];
    }
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int h = h0 + i * blockDim.y;
    if (h >= heads) continue;
    const bool is_q = h < p.q.heads;
    T* dst = static_cast<T*>(is_q ? p.q.out : p.k.out) + row * (is_q ? p.q.out_stride : p.k.out_stride) +
             static_cast<long long>(is_q ? h : h - p.q.heads) * p.head_dim;
    if (!turned) {
      a[i].store_raw(dst + a0);
      continue;
    }
    RopeVec<T, kVec> u, v;
    if constexpr (kVec == 1) {
      const float x = a[i].get(0), y = b[i].get(0);
      u.set(0, x * c[0] - y * s[0], 0.f);
      v.set(0, y * c[0] + x * s[0], 0.f);
    } else if constexpr (kTwo) {
#pragma unroll
      for (int j = 0; j < kVec; j += 2) {
        const float x0 = a[i].get(j), y0 = b[i].get(j), x1 = a[i].get(j + 1), y1 = b[i].get(j + 1);
        u.set(j, x0 * c[j] - y0 * s[j], x1 * c[j + 1] - y1 * s[j + 1]);
        v.set(j, y0 * c[j] + x0 * s[j], y1 * c[j + 1] + x1 * s[j + 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const float x = a[i].get(2 * j), y = a[i].get(2 * j + 1);
        u.set(2 * j, x * c[j] - y * s[j], y * c[j] + x * s[j]);
      }
    }
    u.store_raw(dst + a0);
    if constexpr (kTwo) v.store_raw(dst + b0);
  }
}

static mfa_status check_rope(const mfa_rope_config* c) {
  if (c == nullptr) return MFA_ERR_INVALID_ARG;
  if (c->head_dim < 1 || c->rotary_dim < 2 || (c->rotary_dim & 1) || c->rotary_dim > c->head_dim)
    return MFA_ERR_INVALID_ARG;
  if (c->head_dim > kRopeMaxDim) return MFA_ERR_UNSUPPORTED;
  if (c->num_axes < 1 || c->num_axes > MFA_ROPE_MAX_AXES) return MFA_ERR_INVALID_ARG;
  long long sum = 0;
  for (int i = 0; i < MFA_ROPE_MAX_AXES; ++i) {
    if (c->sections[i] < 0 || (i >= c->num_axes && c->sections[i] != 0)) return MFA_ERR_INVALID_ARG;
    sum += c->sections[i];
  }
  if (2 * sum != c->rotary_dim) return MFA_ERR_INVALID_ARG;
  if (c->pairing != MFA_ROPE_HALF && c->pairing != MFA_ROPE_ADJACENT) return MFA_ERR_INVALID_ARG;
  if (c->flags & ~(MFA_ROPE_INTERLEAVED | MFA_ROPE_OWN_SPECTRUM)) return MFA_ERR_INVALID_ARG;
  if (!(std::isfinite(c->theta) && c->theta >= 1.0)) return MFA_ERR_INVALID_ARG;
  if (!(std::isfinite(c->position_scale) && c->position_scale > 0.0 && c->position_scale <= 16.0))
    return MFA_ERR_INVALID_ARG;
  return MFA_OK;
}

// Whether two sets of rows share memory: `rows` rows of `len` elements each, `stride` apart.  Ranges that
// overlap are apart as columns of one wider row (q and k of one projection): equal strides, and the two
// column ranges apart.  (Different strides count as sharing.)
static bool share(const void* a, int64_t a_stride, int64_t a_len, const void* b, int64_t b_stride, int64_t b_len, int rows,
                  int esz) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uintptr_t a1 = a0 + ((rows - 1) * a_stride + a_len) * esz, b1 = b0 + ((rows - 1) * b_stride + b_len) * esz;
  if (a0 >= b1 || b0 >= a1) return false;
  if (rows == 1 || a_stride != b_stride) return true;
  const uintptr_t stride = static_cast<uintptr_t>(a_stride) * esz;
  const uintptr_t apart = (b0 >= a0 ? b0 - a0 : stride - (a0 - b0) % stride) % stride;   // b's columns past a's
  return apart < static_cast<uintptr_t>(a_len) * esz || stride - apart < static_cast<uintptr_t>(b_len) * esz;
}

static mfa_status check_side(const mfa_rope_rows* s, const mfa_rope_config* c, int rows, int esz) {
  if (s == nullptr || s->heads == 0) return MFA_OK;
  if (s->heads < 0 || s->heads > INT_MAX / 4 / kRopeMaxDim) return MFA_ERR_INVALID_ARG;
  if (rows == 0) return MFA_OK;
  if (s->in == nullptr || s->out == nullptr || !aligned(s->in, esz) || !aligned(s->out, esz)) return MFA_ERR_INVALID_ARG;
  const int64_t least = static_cast<int64_t>(s->heads) * c->head_dim;
  const int64_t most = (int64_t{1} << 58) / rows;   // rows * stride * size stays inside 64 bits
  if (s->in_stride < least || s->out_stride < least || s->in_stride > most || s->out_stride > most)
    return MFA_ERR_INVALID_ARG;
  // in place means the same rows; anything between would be read after it is written
  if (s->in == s->out) return s->in_stride == s->out_stride ? MFA_OK : MFA_ERR_INVALID_ARG;
  return share(s->in, s->in_stride, least, s->out, s->out_stride, least, rows, esz) ? MFA_ERR_INVALID_ARG : MFA_OK;
}

// The wide path needs 16-byte aligned vectors of 8 elements everywhere.
static bool wide_side(const mfa_rope_rows* s) {
  return s == nullptr || s->heads == 0 ||
         (aligned(s->in, 16) && aligned(s->out, 16) && s->in_stride % 8 == 0 && s->out_stride % 8 == 0);
}

static RopeSide side_of(const mfa_rope_rows* s) {
  RopeSide r = {};
  if (s != nullptr && s->heads > 0) r = {s->in, s->out, s->in_stride, s->out_stride, s->heads};
  return r;
}

template <typename T>
static void (*rope_kernel(bool wide, bool half))(RopeParams) {
  if (wide) return half ? mfa_rope_kernel<T, 8, true> : mfa_rope_kernel<T, 8, false>;
  return half ? mfa_rope_kernel<T, 1, true> : mfa_rope_kernel<T, 1, false>;
}

// ------------------------------------------------------------------ frequencies, on the host
//
// Sums of two doubles, hi + lo with |lo| at most half a step of hi: some 100 bits, by error-free sums and
// products (Dekker's; the products by fma).
struct Twofold {
  double hi, lo;
};
static Twofold two_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
static Twofold add(Twofold a, Twofold b) {
  const Twofold s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, s.lo + (a.lo + b.lo));
}
static Twofold mul(Twofold a, Twofold b) {
  const double p = a.hi * b.hi;
  return two_sum(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
static Twofold ratio(double a, double b) {   // of two whole numbers
  const double q = a / b;
  return two_sum(q, std::fma(-q, b, a) / b);
}
constexpr Twofold kLn2 = {0x1.62e42fefa39efp-1, 0x1.abc9e3b39803fp-56};
constexpr Twofold kInv2Pi = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};

// e^x, |x| < 745: x = k ln 2 + 512 r, e^r - 1 by its series, then nine times s -> 2 s + s^2.
static Twofold exp_of(Twofold x) {
  const double k = std::nearbyint(x.hi / kLn2.hi);
  Twofold r = add(x, mul({-k, 0.0}, kLn2));
  r = {std::ldexp(r.hi, -9), std::ldexp(r.lo, -9)};
  Twofold s = ratio(1.0, 10.0);   // s = r (1 + r / 2 (1 + r / 3 (...))), |r| < 7e-4
  s = mul(s, r);
  for (int n = 9; n >= 1; --n) s = mul(mul(add(s, {1.0, 0.0}), r), ratio(1.0, n));
  for (int n = 0; n < 9; ++n) s = add({2.0 * s.hi, 2.0 * s.lo}, mul(s, s));
  s = add(s, {1.0, 0.0});
  return {std::ldexp(s.hi, static_cast<int>(k)), std::ldexp(s.lo, static_cast<int>(k))};
}
// ln x, x >= 1: of its fraction m in [1/2, 1) a double's logarithm y and one Newton step, y + (m e^-y - 1).
static Twofold log_of(double x) {
  int e;
  const double m = std::frexp(x, &e), y = std::log(m);
  const Twofold step = add(mul({m, 0.0}, exp_of({-y, 0.0})), {-1.0, 0.0});
  return add(mul({static_cast<double>(e), 0.0}, kLn2), add({y, 0.0}, step));
}
// t turns (t >= 0) in units of 2^-64, to nearest, modulo 2^64.
static uint64_t turn_fraction(Twofold t) {
  const double hi = std::ldexp(t.hi, 64), whole = std::floor(hi);
  const double rest = std::nearbyint((hi - whole) + std::ldexp(t.lo, 64));   // (|lo| < 2^13 there)
  return static_cast<uint64_t>(std::fmod(whole, 18446744073709551616.0)) + static_cast<uint64_t>(static_cast<int64_t>(rest));
}

}  // namespace mfa

using namespace mfa;

extern "C" mfa_status mfa_rope_table(const mfa_rope_config* c, mfa_rope_pair* table) {
  const mfa_status st = check_rope(c);
  if (st != MFA_OK) return st;
  if (table == nullptr) return MFA_ERR_INVALID_ARG;
  const int pairs = c->rotary_dim / 2;
  const Twofold log_theta = log_of(c->theta);
  int used[MFA_ROPE_MAX_AXES] = {0, 0, 0, 0};
  int axis = 0;
  for (int i = 0; i < pairs; ++i) {
    // the next pair's axis: the current run's, or the next in turn, skipping those that are full
    while (used[axis] == c->sections[axis]) axis = (axis + 1) % c->num_axes;
    const Twofold power = (c->flags & MFA_ROPE_OWN_SPECTRUM) ? ratio(used[axis], c->sections[axis])
                                                             : ratio(2.0 * i, c->rotary_dim);
    const Twofold frequency = exp_of(mul(mul(power, log_theta), {-1.0, 0.0}));
    table[i].turns = turn_fraction(mul(mul(frequency, kInv2Pi), {c->position_scale, 0.0}));
    table[i].axis = axis;
    table[i].reserved = 0;
    ++used[axis];
    if (c->flags & MFA_ROPE_INTERLEAVED) axis = (axis + 1) % c->num_axes;
  }
  return MFA_OK;
}

extern "C" mfa_status mfa_rope_run(const mfa_rope_config* c, const mfa_rope_pair* table, const int32_t* positions,
                                   int32_t num_rows, int32_t dtype, int32_t inverse, const mfa_rope_rows* q,
                                   const mfa_rope_rows* k, void* stream_ptr) {
  mfa_status st = check_rope(c);
  if (st != MFA_OK) return st;
  if (num_rows < 0 || (dtype != MFA_OUT_BF16 && dtype != MFA_OUT_FP32) || (inverse != 0 && inverse != 1))
    return MFA_ERR_INVALID_ARG;
  const int esz = dtype == MFA_OUT_BF16 ? 2 : 4;
  if ((st = check_side(q, c, num_rows, esz)) != MFA_OK || (st = check_side(k, c, num_rows, esz)) != MFA_OK) return st;
  RopeParams p = {};
  p.q = side_of(q);
  p.k = side_of(k);
  const long long heads = static_cast<long long>(p.q.heads) + p.k.heads;
  if (num_rows == 0 || heads == 0) return MFA_OK;
  if (p.q.heads > 0 && p.k.heads > 0) {   // what one side writes is neither read nor written by the other
    const int64_t nq = static_cast<int64_t>(p.q.heads) * c->head_dim, nk = static_cast<int64_t>(p.k.heads) * c->head_dim;
    if (share(p.q.out, p.q.out_stride, nq, p.k.in, p.k.in_stride, nk, num_rows, esz) ||
        share(p.q.out, p.q.out_stride, nq, p.k.out, p.k.out_stride, nk, num_rows, esz) ||
        share(p.q.in, p.q.in_stride, nq, p.k.out, p.k.out_stride, nk, num_rows, esz))
      return MFA_ERR_INVALID_ARG;
  }
  if (table == nullptr || positions == nullptr || !aligned(table, 16) || !aligned(positions, 4)) return MFA_ERR_INVALID_ARG;
  const bool half = c->pairing == MFA_ROPE_HALF;
  const bool wide = c->head_dim % 8 == 0 && c->rotary_dim % (half ? 16 : 8) == 0 && wide_side(q) && wide_side(k);
  const int vec = wide ? 8 : 1;
  p.table = table;
  p.positions = positions;
  p.rows = num_rows;
  p.axes = c->num_axes;
  p.pairs = c->rotary_dim / 2;
  p.head_dim = c->head_dim;
  p.turned_units = (half || !wide) ? p.pairs / vec : c->rotary_dim / vec;
  const bool in_place = (p.q.heads == 0 || p.q.in == p.q.out) && (p.k.heads == 0 || p.k.in == p.k.out);
  p.units = p.turned_units + (in_place ? 0 : (c->head_dim - c->rotary_dim) / vec);
  p.inverse = inverse;
  // threads: a head's units by as many heads as a CTA can take, each thread some of them
  const int most = std::max(1, kRopeMaxThreads / p.units);
  const int each = dtype == MFA_OUT_BF16 ? kRopeHeads<__nv_bfloat16> : kRopeHeads<float>;
  const int ny = static_cast<int>(std::min<long long>(most, (heads + each - 1) / each));
  const long long gy = (heads + static_cast<long long>(ny) * each - 1) / (static_cast<long long>(ny) * each);
  if (gy > 65535) return MFA_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_rows), static_cast<unsigned>(gy), 1);
  cfg.blockDim = dim3(static_cast<unsigned>(p.units), static_cast<unsigned>(ny), 1);
  cfg.stream = static_cast<cudaStream_t>(stream_ptr);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, dtype == MFA_OUT_BF16 ? rope_kernel<__nv_bfloat16>(wide, half)
                                                                       : rope_kernel<float>(wide, half), p);
  if (e != cudaSuccess) return cuda_fail(e, "rope launch");
  return MFA_OK;
}
