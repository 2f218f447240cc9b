// Device helpers shared by the decode kernels: bounded waits, tcgen05 descriptors, block scans
// and the e4m3 split of q.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx.cuh"

namespace mfa {

constexpr uint64_t kWaitLimitNs = 1000000000ull;  // 1 s per pipeline wait
constexpr uint64_t kDrainLimitNs = 100000000ull;  // 0.1 s for drains after an abort

// tcgen05 shared-memory matrix descriptor: start, leading/stride byte offsets,
// descriptor version 1 (bits 46..47), 128-byte swizzle (bits 61..63 = 2).
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// The same with the 64-byte swizzle (layout code 4): 64-byte rows, 8-row atoms of 512 bytes,
// 16-byte chunk c of row r stored at chunk c ^ ((r >> 1) & 3).
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (4ull << 61);
}

// tcgen05 instruction descriptor for kind::f16: fp32 D, bf16 or f16 A/B,
// K-major (0) or MN-major (1) operands, N>>3 at bit 17, M>>4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, bool a_mn, bool b_mn, int m, int n) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// tcgen05 instruction descriptor for kind::f8f6f4 with e4m3 A and B (format code 0),
// fp32 D, K-major (0) or MN-major (1) operands.
__host__ __device__ constexpr uint32_t idesc_e4m3(bool a_mn, bool b_mn, int m, int n) {
  return (1u << 4) | (0u << 7) | (0u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ int clamp_len(int L, int cap, bool& bad) {
  if (L < 0) { bad = true; return 0; }
  if (L > cap) { bad = true; return cap; }
  return L;
}

// Bounded wait on an mbarrier phase.  Returns false after kWaitLimitNs, or at
// once when another role has raised the CTA's abort flag.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                       uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (abort_flag != nullptr && *abort_flag) return false;
    if (global_timer_ns() - t0 > limit_ns) return false;
  }
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const bool ok = wait_slow(bar, parity, abort_flag, kWaitLimitNs);
  if (!ok && abort_flag != nullptr) *abort_flag = 1;
  return ok;
}

// Bounded wait until a monotonic shared-memory count reaches target (see the ring-order
// counts in the kernel); sets the abort flag when it gives up.
__device__ __forceinline__ bool wait_count(const int* count, int target, volatile int* abort_flag) {
  if (ld_acquire_cta(count) >= target) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    __nanosleep(32);
    if (ld_acquire_cta(count) >= target) return true;
    if (abort_flag != nullptr && *abort_flag) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      if (abort_flag != nullptr) *abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_count_warp(const int* count, int target, volatile int* abort_flag) {
  const bool ok = wait_count(count, target, abort_flag);
  return __all_sync(0xffffffffu, ok);
}

// Block-wide (kThreads threads) inclusive scan of one value per thread; also returns the total.
template <int kThreads, typename V = int>
__device__ __forceinline__ V block_incl_scan(V v, V* scratch, V& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  V before = 0, tot = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const V x = scratch[w];
    before += (w < warp) ? x : 0;
    tot += x;
  }
  __syncthreads();
  total = tot;
  return v + before;
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Warp-uniform bounded wait (all lanes poll; the warp agrees on the outcome).
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const bool ok = wait_bar(bar, parity, abort_flag);
  return __all_sync(0xffffffffu, ok);
}

// Two floats to two e4m3 codes (round to nearest even, saturating); lo in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3_sat(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Split two scaled q values x into e4m3 pairs hi + lo with hi = e4m3(x) and lo = e4m3(x - hi).
// x is a bf16 value times a power of two (8 significant bits) and the largest |x| of the
// sequence lies in [64, 128).  x - hi is exact in fp32 and is k * ulp(x) with |k| <= 8, so
// it fits e4m3's 4 significant bits: hi + lo = x exactly when ulp(x) >= 2^-9 (the e4m3
// subnormal step), i.e. for |x| >= 2^-2, which covers every element at least 2^-9 of the
// largest.  Smaller elements err by at most 2^-10, under 2^-16 of the largest.
// (The hi part is read back exactly through the f16 conversion.  A bit-placement read-back,
// the 7 magnitude bits at bit 20 of an fp32 word times 2^120, gives the same bits, but the
// conversion measured faster end to end -- finishing a segment's q split earlier moves the
// CTAs' load streams into a worse phase.)
__device__ __forceinline__ void split_e4m3(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_e4m3_sat(x0, x1);
  uint32_t back;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(static_cast<uint16_t>(hi)));
  lo = pack_e4m3_sat(x0 - __half2float(__ushort_as_half(static_cast<unsigned short>(back))),
                     x1 - __half2float(__ushort_as_half(static_cast<unsigned short>(back >> 16))));
}

}  // namespace mfa
