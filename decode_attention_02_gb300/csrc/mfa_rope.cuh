// Pieces shared by the kernels that turn rows by their positions: elements as vectors, and angles.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "mfa.h"
#include "ptx.cuh"

namespace mfa {

constexpr int kRopeMaxDim = 512;

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
  // values i and i + 1 (i even, kVec > 1), packed
  __device__ __forceinline__ uint64_t pair(int i) const { return pack_f32x2(get(i), get(i + 1)); }
  __device__ __forceinline__ void set_pair(int i, uint64_t v) {
    float lo, hi;
    unpack_f32x2(v, lo, hi);
    set(i, lo, hi);
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

// sin and cos of pair i of a row at positions pos: position times the table's fraction modulo one turn.
__device__ __forceinline__ void rope_angle(const mfa_rope_pair* table, int i, const int32_t (&pos)[MFA_ROPE_MAX_AXES], float& s,
                                           float& c) {
  const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(table + i);
  const int axis = static_cast<int>(e.y & 3u);
  const int32_t at = axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
  const uint64_t turn = e.x * static_cast<uint64_t>(static_cast<int64_t>(at));
  // the top 32 bits as a signed fraction in [-1/2, 1/2) turns; 2^-31 of it is half turns
  const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;
  sincospif(half_turns, &s, &c);
}

}  // namespace mfa
