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
// the registers of a group of up to 32 lanes (a lane: 8 elements of a pair's first half and the 8 of
// its second, as they lie in memory), so that its sums are a few shuffles and nothing is read twice.
// A CTA turns all heads of a row: the row's angles are computed once and shared.  A group keeps to one
// side, q or k, so that a lane's weights stay in its registers, multiplied with the angles' cosines and
// sines in the forward pass.  All sums are fp32; outputs are rounded once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "mfa.h"
#include "mfa_host.h"
#include "mfa_rope.cuh"
#include "ptx.cuh"

namespace mfa {

constexpr int kNormThreads = 512;        // of a CTA, at most
constexpr int kNormAnyThreads = 256;     // of a CTA of the path for any shape
constexpr int kNormAnyEach = kRopeMaxDim / 32;   // its elements a lane

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
  int turned_units, units, log_lanes;   // wide path: a head's units, lanes of its group
  int half;                             // pairing, for any shape
  int w_f32;
  float eps, inv_dim;
  float* partial;                       // gradient: [CTAs][q, k][head_dim]
  float* dw[2];                         // gradient of the weights
  int parts;                            // CTAs that leave partial sums
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

// Angles of row `row`, one pair a thread, into cs.
__device__ __forceinline__ void row_angles(const NormParams& p, long long row, int tid, int threads, float (&cs)[2][kRopeMaxDim / 2]) {
  int32_t pos[MFA_ROPE_MAX_AXES];
#pragma unroll
  for (int x = 0; x < MFA_ROPE_MAX_AXES; ++x) pos[x] = x < p.axes ? p.positions[static_cast<long long>(x) * p.rows + row] : 0;
  for (int i = tid; i < p.pairs; i += threads) {
    float s, c;
    rope_angle(p.table, i, pos, s, c);
    cs[0][i] = c;
    cs[1][i] = s;
  }
}

// Sums of N values over a head's group of 2^log_lanes lanes.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], unsigned mask, int lanes) {
#pragma unroll 1
  for (int o = lanes / 2; o > 0; o /= 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(mask, v[i], o);
  }
}

// A thread's place: its group's slot on one side, its unit of the head.
template <bool kHalf>
struct NormPlace {
  int u, a0, b0, h0, step;
  bool on_q, active, turned;
  unsigned mask;
  __device__ __forceinline__ NormPlace(const NormParams& p) {
    const int lanes = 1 << p.log_lanes, slot = threadIdx.x >> p.log_lanes, lane = threadIdx.x & 31;
    u = threadIdx.x & (lanes - 1);
    active = u < p.units;
    turned = u < p.turned_units;
    on_q = slot < p.q.slots;
    h0 = on_q ? slot : slot - p.q.slots;
    step = on_q ? p.q.slots : p.k.slots;
    mask = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1u) << (lane & ~(lanes - 1));
    a0 = turned ? 8 * u : 2 * p.pairs + 8 * (u - p.turned_units);
    b0 = kHalf && turned ? a0 + p.pairs : a0;
  }
};

// ------------------------------------------------------------------ forward
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kNormThreads) mfa_norm_rope_kernel(const __grid_constant__ NormParams p) {
  constexpr int kN = sizeof(T) == 2 ? 4 : 2;   // heads a thread has at a time
  constexpr int kPairs = kHalf ? 8 : 4;
  __shared__ __align__(16) float cs[2][kRopeMaxDim / 2];
  grid_dep_wait();
  grid_dep_launch();
  const NormPlace<kHalf> at(p);
  const NormSide& side = at.on_q ? p.q : p.k;
  const long long row = blockIdx.x;
  const T* src = static_cast<const T*>(side.x) + row * side.x_stride;
  T* dst = static_cast<T*>(side.out) + row * side.out_stride;
  RopeVec<T, 8> a[kN], b[kN];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int hi = h + i * at.step;
      if (hi < side.heads && at.active) {
        a[i].load(src + static_cast<long long>(hi) * p.head_dim + at.a0);
        if (kHalf && at.turned) b[i].load(src + static_cast<long long>(hi) * p.head_dim + at.b0);
      }
    }
  };
  load(at.h0);
  // weights times cosines and sines: y = r (a ac - b bs), r (b bc + a as)
  float ac[kPairs], as[kPairs], bc[kPairs], bs[kPairs];
  if (at.active) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      ac[i] = norm_weight(p, side, at.a0 + (kHalf ? i : 2 * i));
      bc[i] = norm_weight(p, side, kHalf ? at.b0 + i : at.a0 + 2 * i + 1);
    }
  }
  row_angles(p, row, threadIdx.x, blockDim.x, cs);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const float c = at.turned ? cs[0][kPairs * at.u + i] : 1.f, s = at.turned ? cs[1][kPairs * at.u + i] : 0.f;
    as[i] = ac[i] * s;
    ac[i] *= c;
    bs[i] = bc[i] * s;
    bc[i] *= c;
  }
#pragma unroll 1
  for (int h = at.h0; h < side.heads; h += kN * at.step) {
    if (h != at.h0) load(h);
    float sum[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      sum[i] = 0.f;
      if (h + i * at.step < side.heads && at.active) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[i] = fmaf(a[i].get(j), a[i].get(j), sum[i]);
        if (kHalf && at.turned) {
#pragma unroll
          for (int j = 0; j < 8; ++j) sum[i] = fmaf(b[i].get(j), b[i].get(j), sum[i]);
        }
      }
    }
    group_sum<kN>(sum, at.mask, 1 << p.log_lanes);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int hi = h + i * at.step;
      if (hi >= side.heads || !at.active) continue;
      const float r = rsqrtf(fmaf(sum[i], p.inv_dim, p.eps));
      T* to = dst + static_cast<long long>(hi) * p.head_dim;
      RopeVec<T, 8> y, z;
      if constexpr (kHalf) {
        if (at.turned) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const float a0 = a[i].get(j), b0 = b[i].get(j), a1 = a[i].get(j + 1), b1 = b[i].get(j + 1);
            y.set(j, r * (a0 * ac[j] - b0 * bs[j]), r * (a1 * ac[j + 1] - b1 * bs[j + 1]));
            z.set(j, r * (b0 * bc[j] + a0 * as[j]), r * (b1 * bc[j + 1] + a1 * as[j + 1]));
          }
          z.store_raw(to + at.b0);
        } else {
#pragma unroll
          for (int j = 0; j < 8; j += 2) y.set(j, r * (a[i].get(j) * ac[j]), r * (a[i].get(j + 1) * ac[j + 1]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = a[i].get(2 * j), x1 = a[i].get(2 * j + 1);
          y.set(2 * j, r * (x0 * ac[j] - x1 * bs[j]), r * (x1 * bc[j] + x0 * as[j]));
        }
      }
      y.store_raw(to + at.a0);
    }
  }
}

// ------------------------------------------------------------------ gradient
//
// CTAs loop over rows, so that the sums of the weights' gradient stay in registers; each CTA leaves one
// partial sum a side and element, and a second kernel adds those in a fixed order.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kNormThreads) mfa_norm_rope_grad_kernel(const __grid_constant__ NormParams p) {
  constexpr int kN = sizeof(T) == 2 ? 2 : 1;
  constexpr int kPairs = kHalf ? 8 : 4;
  __shared__ __align__(16) float cs[2][2][kRopeMaxDim / 2];
  extern __shared__ float red[];   // [slots][head_dim]
  grid_dep_wait();
  const NormPlace<kHalf> at(p);
  const NormSide& side = at.on_q ? p.q : p.k;
  float wa[8], wb[8], da[8] = {}, db[8] = {};   // weights and their gradients' sums, of a lane's elements
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    wa[j] = at.active ? norm_weight(p, side, at.a0 + j) : 0.f;
    wb[j] = kHalf && at.turned ? norm_weight(p, side, at.b0 + j) : 0.f;
  }
  int buffer = 0;
#pragma unroll 1
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, buffer ^= 1) {
    const T* xs = static_cast<const T*>(side.x) + row * side.x_stride;
    const T* dys = static_cast<const T*>(side.dy) + row * side.dy_stride;
    T* dst = static_cast<T*>(side.out) + row * side.out_stride;
    RopeVec<T, 8> a[kN], b[kN], ga[kN], gb[kN];
    auto load = [&](int h) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const long long hi = h + i * at.step;
        if (hi < side.heads && at.active) {
          a[i].load(xs + hi * p.head_dim + at.a0);
          ga[i].load(dys + hi * p.head_dim + at.a0);
          if (kHalf && at.turned) {
            b[i].load(xs + hi * p.head_dim + at.b0);
            gb[i].load(dys + hi * p.head_dim + at.b0);
          }
        }
      }
    };
    load(at.h0);
    row_angles(p, row, threadIdx.x, blockDim.x, cs[buffer]);
    __syncthreads();   // (the other buffer's readers are behind this barrier before it is written again)
    float c[kPairs], s[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      c[i] = at.turned ? cs[buffer][0][kPairs * at.u + i] : 1.f;
      s[i] = at.turned ? cs[buffer][1][kPairs * at.u + i] : 0.f;
    }
#pragma unroll 1
    for (int h = at.h0; h < side.heads; h += kN * at.step) {
      if (h != at.h0) load(h);
      // g of a lane's elements: dy turned back
      auto turn_back = [&](int i, float (&g)[8], float (&k)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (kHalf) {
            const float x = ga[i].get(j), y = at.turned ? gb[i].get(j) : 0.f;
            g[j] = x * c[j] + y * s[j];
            k[j] = y * c[j] - x * s[j];
          } else {
            const float x = ga[i].get(j & ~1), y = ga[i].get(j | 1);
            g[j] = (j & 1) ? y * c[j / 2] - x * s[j / 2] : x * c[j / 2] + y * s[j / 2];
          }
        }
      };
      float sum[2 * kN];   // sum x^2, sum u x
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        sum[2 * i] = sum[2 * i + 1] = 0.f;
        if (h + i * at.step < side.heads && at.active) {
          float g[8], k[8];
          turn_back(i, g, k);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sum[2 * i] = fmaf(a[i].get(j), a[i].get(j), sum[2 * i]);
            sum[2 * i + 1] = fmaf(g[j] * wa[j], a[i].get(j), sum[2 * i + 1]);
          }
          if (kHalf && at.turned) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              sum[2 * i] = fmaf(b[i].get(j), b[i].get(j), sum[2 * i]);
              sum[2 * i + 1] = fmaf(k[j] * wb[j], b[i].get(j), sum[2 * i + 1]);
            }
          }
        }
      }
      group_sum<2 * kN>(sum, at.mask, 1 << p.log_lanes);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const long long hi = h + i * at.step;
        if (hi >= side.heads || !at.active) continue;
        const float r = rsqrtf(fmaf(sum[2 * i], p.inv_dim, p.eps));
        const float m = r * r * sum[2 * i + 1] * p.inv_dim;   // dx = r (u - x m)
        float g[8], k[8];
        turn_back(i, g, k);
        T* to = dst + hi * p.head_dim;
        RopeVec<T, 8> y;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float x0 = a[i].get(j), x1 = a[i].get(j + 1);
          y.set(j, r * (g[j] * wa[j] - x0 * m), r * (g[j + 1] * wa[j + 1] - x1 * m));
          da[j] = fmaf(g[j], x0 * r, da[j]);
          da[j + 1] = fmaf(g[j + 1], x1 * r, da[j + 1]);
        }
        y.store_raw(to + at.a0);
        if (kHalf && at.turned) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const float x0 = b[i].get(j), x1 = b[i].get(j + 1);
            y.set(j, r * (k[j] * wb[j] - x0 * m), r * (k[j + 1] * wb[j + 1] - x1 * m));
            db[j] = fmaf(k[j], x0 * r, db[j]);
            db[j + 1] = fmaf(k[j + 1], x1 * r, db[j + 1]);
          }
          y.store_raw(to + at.b0);
        }
      }
    }
  }
  grid_dep_launch();
  // the CTA's sums: over the slots of a side, in order
  float* mine = red + (threadIdx.x >> p.log_lanes) * p.head_dim;
  if (at.active) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mine[at.a0 + j] = da[j];
      if (kHalf && at.turned) mine[at.b0 + j] = db[j];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * p.head_dim; e += blockDim.x) {
    const bool on_k = e >= p.head_dim;
    const int from = on_k ? p.q.slots : 0, to = on_k ? p.q.slots + p.k.slots : p.q.slots;
    float v = 0.f;
    for (int x = from; x < to; ++x) v += red[x * p.head_dim + (on_k ? e - p.head_dim : e)];
    p.partial[static_cast<size_t>(blockIdx.x) * 2 * p.head_dim + e] = v;
  }
}

// The weights' gradient: partial sums of the CTAs, 8 elements a CTA, 32 threads for each, in a fixed order.
__global__ void __launch_bounds__(256) mfa_norm_rope_weights_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[32][9];
  grid_dep_wait();
  grid_dep_launch();
  const int el = blockIdx.x * 8 + (threadIdx.x & 7), part = threadIdx.x >> 3;
  float v = 0.f;
  if (el < 2 * p.head_dim)
    for (int i = part; i < p.parts; i += 32) v += p.partial[static_cast<size_t>(i) * 2 * p.head_dim + el];
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
// Heads of odd sizes, unaligned rows: a warp a head, a lane its every 32nd element and that element's
// partner in the pair.
template <typename T, bool kGrad>
__global__ void __launch_bounds__(kNormAnyThreads) mfa_norm_rope_any_kernel(const __grid_constant__ NormParams p) {
  __shared__ __align__(16) float cs[2][2][kRopeMaxDim / 2];
  extern __shared__ float red[];   // gradient: [warps][head_dim]
  grid_dep_wait();
  if constexpr (!kGrad) grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool on_q = warp < p.q.slots;
  const NormSide& side = on_q ? p.q : p.k;
  const int h0 = on_q ? warp : warp - p.q.slots, step = side.slots;
  const int r2 = 2 * p.pairs;
  float dw[kNormAnyEach] = {};
  int buffer = 0;
#pragma unroll 1
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, buffer ^= 1) {
    row_angles(p, row, threadIdx.x, blockDim.x, cs[buffer]);
    __syncthreads();
    const T* xs = static_cast<const T*>(side.x) + row * side.x_stride;
    const T* dys = static_cast<const T*>(side.dy) + row * side.dy_stride;
    T* dst = static_cast<T*>(side.out) + row * side.out_stride;
#pragma unroll 1
    for (long long h = h0; h < side.heads; h += step) {
      const T* x = xs + h * p.head_dim;
      float own[kNormAnyEach], out[kNormAnyEach], sum[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kNormAnyEach; ++i) {
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
      for (int i = 0; i < kNormAnyEach; ++i) {
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
  }
  if constexpr (kGrad) {
    grid_dep_launch();
#pragma unroll
    for (int i = 0; i < kNormAnyEach; ++i) {
      const int e = lane + 32 * i;
      if (e < p.head_dim) red[warp * p.head_dim + e] = dw[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * p.head_dim; e += blockDim.x) {
      const bool on_k = e >= p.head_dim;
      const int from = on_k ? p.q.slots : 0, to = on_k ? p.q.slots + p.k.slots : p.q.slots;
      float v = 0.f;
      for (int x = from; x < to; ++x) v += red[x * p.head_dim + (on_k ? e - p.head_dim : e)];
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

// Groups of lanes (or warps) for the sides' heads: as many as heads of `each` a time fill, or, of what a CTA
// has room for, a share by their heads.
static void norm_slots(NormParams& p, int room, int each) {
  const int hq = p.q.heads, hk = p.k.heads;
  int nq = (hq + each - 1) / each, nk = (hk + each - 1) / each;
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
    if (run && workspace_bytes < MFA_NORM_ROPE_GRAD_BYTES(num_rows, c->head_dim)) return MFA_ERR_WORKSPACE;
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
  p.turned_units = (half ? p.pairs : c->rotary_dim) / 8;
  p.units = p.turned_units + (c->head_dim - c->rotary_dim) / 8;
  while ((1 << p.log_lanes) < p.units) ++p.log_lanes;
  const bool wide = c->head_dim % 8 == 0 && c->rotary_dim % (half ? 16 : 8) == 0 && p.log_lanes <= 5 && wide_norm_side(q, grad) &&
                    wide_norm_side(k, grad);
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
    int ctas = num_rows;
    if (grad) {
      int dev = 0, sms = 0;
      if ((e = cudaGetDevice(&dev)) != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
      if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return cuda_fail(e, "cudaDeviceGetAttribute");
      ctas = std::min({num_rows, 2 * sms, MFA_NORM_ROPE_GRAD_PARTS});
    }
    p.parts = grad ? ctas : 0;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    void (*fn)(NormParams);
    if (wide) {
      norm_slots(p, kNormThreads >> p.log_lanes, bf16 ? 4 : 2);
      cfg.blockDim = dim3(static_cast<unsigned>((p.q.slots + p.k.slots) << p.log_lanes), 1, 1);
      if (grad) {
        if (bf16) fn = half ? mfa_norm_rope_grad_kernel<__nv_bfloat16, true> : mfa_norm_rope_grad_kernel<__nv_bfloat16, false>;
        else fn = half ? mfa_norm_rope_grad_kernel<float, true> : mfa_norm_rope_grad_kernel<float, false>;
      } else {
        if (bf16) fn = half ? mfa_norm_rope_kernel<__nv_bfloat16, true> : mfa_norm_rope_kernel<__nv_bfloat16, false>;
        else fn = half ? mfa_norm_rope_kernel<float, true> : mfa_norm_rope_kernel<float, false>;
      }
    } else {
      norm_slots(p, kNormAnyThreads / 32, 1);
      cfg.blockDim = dim3(static_cast<unsigned>((p.q.slots + p.k.slots) * 32), 1, 1);
      if (grad) fn = bf16 ? mfa_norm_rope_any_kernel<__nv_bfloat16, true> : mfa_norm_rope_any_kernel<float, true>;
      else fn = bf16 ? mfa_norm_rope_any_kernel<__nv_bfloat16, false> : mfa_norm_rope_any_kernel<float, false>;
    }
    // a slot's sums of the weights' gradient: at most 512 threads x 16 elements, or 8 warps x 512
    if (grad) cfg.dynamicSmemBytes = static_cast<size_t>(p.q.slots + p.k.slots) * p.head_dim * 4;
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
