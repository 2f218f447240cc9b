// KV append to a block-scaled 8-bit cache (GB300, sm_103a): new bf16 key and value rows are
// written as e4m3 codes under one fp32 scale for each block of tokens and head.
//
// For a block that gets rows, a = the largest finite |x| of its new rows (one head):
//     need = 2^e, the smallest power of two with a <= 448 * 2^e;
//     s    = need, or max(need, s_old) where the block holds older rows;
//     code = e4m3(x / s);  where s > s_old the older codes become e4m3(value * (s_old / s)).
// Powers of two: e4m3 has an exponent of its own, so that its precision does not depend on
// where in an octave the maximum falls, and a rise of the scale shifts the older codes'
// exponents without rounding them again (except below e4m3's smallest step).
//
// An item is one (block, head, K or V): its new rows are read once, into registers; their
// maximum gives the scale; the codes are written.  Items share nothing, so the work is one
// pass over the data with no atomics but error flags.  A thread holds up to 8 chunks of 8
// elements, all loads in flight together, and an item gets as many threads as that takes: a
// warp for the row of a decode step or a block of 16 x 128, a whole CTA for one of 64 x 256.
//
// HBM-bound for a prompt: 24 prompts of 700 to 8191 rows of 256 (164 MB) 30.2 us, 5.4 TB/s, 80% of
// the copy rate; 7 chunks behind 3001 tokens (blocks of 16, 4 heads of 128, 33 MB) 8.0 us.  A decode
// step's rows (128 sequences, 0.2 MB) are launch and latency, 2.6 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "mfa.h"
#include "mfa_host.h"
#include "ptx.cuh"
#include "mfa_append_row.cuh"

namespace mfa {

constexpr int kBlkPage = 64;
constexpr int kBlkThreads = 256;
constexpr int kChunks = 8;            // 8-element chunks a thread holds
static_assert(kChunks * kBlkThreads * 8 >= 64 * 256, "a CTA holds a whole block of 64 rows of 256");

struct BlockAppendParams {
  const uint4* k_new;        // bf16 [num_new, G, d] as 8-element chunks
  const uint4* v_new;
  const int32_t* offsets;    // may be null: `tokens` rows a sequence
  const int32_t* positions;
  const int32_t* block_table;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scale;
  float* v_scale;
  unsigned int* status;      // may be null
  int batch, tokens, num_new, max_new;
  int most_blocks;           // blocks a sequence's new rows can touch
  int heads;                 // G
  int log_chunks;            // log2(d / 8)
  int log_scale;             // log2(scale_tokens)
  int max_pages, num_blocks;
};

// The smallest power of two s = 2^e, e >= -126, with a <= 448 s (a finite, >= 0): with
// a = 2^E (1 + f), 448 = 1.75 * 2^8, so e = E - 8 while 1 + f <= 1.75, else E - 7.
__device__ __forceinline__ float pow2_scale(float a) {
  const uint32_t bits = __float_as_uint(a);
  int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  if (bits == 0u || e < -126) e = -126;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Eight bf16 values to eight e4m3 codes of x / s.  Where s is a power of two with a normal
// reciprocal the product with it is the quotient, exactly (a quotient below the normal range
// rounds to a zero code either way).
template <bool kProduct>
__device__ __forceinline__ uint2 encode_chunk(uint4 x, float s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = bf16_bits_lo(w[i]), hi = bf16_bits_hi(w[i]);
    c[i] = kProduct ? e4m3x2_rn_sat(lo * s, hi * s) : e4m3x2_rn_sat(__fdiv_rn(lo, s), __fdiv_rn(hi, s));
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
// (a scale of another kind is met where a begun block keeps the one it had: out of the way)
__device__ __noinline__ uint2 encode_chunk_by_division(uint4 x, float s) { return encode_chunk<false>(x, s); }

// The largest |x| of a chunk's bf16 values as bit patterns, pairwise: magnitudes order as integers,
// infinities and NaN above all finite ones.
__device__ __forceinline__ uint32_t max_bits(uint32_t m, uint4 x) {
  m = __vmaxu2(m, x.x & 0x7FFF7FFFu);
  m = __vmaxu2(m, x.y & 0x7FFF7FFFu);
  m = __vmaxu2(m, x.z & 0x7FFF7FFFu);
  return __vmaxu2(m, x.w & 0x7FFF7FFFu);
}
// The same with what is not finite left out (as zeros).
__device__ __noinline__ uint4 finite_only(uint4 x) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u;
    if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0x0000FFFFu;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Four e4m3 codes times r, rounded back to e4m3 (e4m3 values are exact in f16).
__device__ __forceinline__ uint32_t recode4(uint32_t codes, float r) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes >> (16 * i))));
    const __half2 h2 = *reinterpret_cast<const __half2*>(&h);
    out |= e4m3x2_rn_sat(__low2float(h2) * r, __high2float(h2) * r) << (16 * i);
  }
  return out;
}

// kItemThreads threads an item, 256 / kItemThreads items a CTA.
template <int kItemThreads>
__global__ void __launch_bounds__(kBlkThreads, 5) mfa_block_append_kernel(const __grid_constant__ BlockAppendParams p) {
  constexpr int kItems = kBlkThreads / kItemThreads;
  __shared__ float wmax[kBlkThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int it = threadIdx.x % kItemThreads;
  // item = ((sequence, touched block m), head, K or V)
  const long long items = static_cast<long long>(p.batch) * p.most_blocks * p.heads * 2;
  const long long item = static_cast<long long>(blockIdx.x) * kItems + threadIdx.x / kItemThreads;
  if (item >= items) return;   // (all of an item's threads leave together, here and below)
  const bool is_v = (item & 1) != 0;
  const long long bh = item >> 1;
  const int g = static_cast<int>(bh % p.heads);
  const int m = static_cast<int>((bh / p.heads) % p.most_blocks);
  const int b = static_cast<int>(bh / p.heads / p.most_blocks);
  const bool reporter = it == 0 && !is_v && g == 0 && p.status != nullptr;

  const int t0 = p.positions[b];
  int r0 = b * p.tokens, n = p.tokens;   // the sequence's rows r0 .. r0 + n - 1
  if (p.offsets != nullptr) {
    r0 = p.offsets[b];
    const int r1 = p.offsets[b + 1];
    if (r0 < 0 || r1 < r0 || r1 > p.num_new) {
      if (reporter && m == 0) atomicOr(p.status, MFA_DEV_BAD_LENGTH);
      return;
    }
    n = r1 - r0;
  }
  if (t0 < 0 || n == 0) return;
  const long long cap = static_cast<long long>(p.max_pages) * kBlkPage;
  const long long fit = cap > t0 ? cap - t0 : 0;
  if (n > p.max_new || n > fit) {
    if (reporter && m == 0) atomicOr(p.status, MFA_DEV_BAD_LENGTH);
    n = static_cast<int>(min(static_cast<long long>(min(n, p.max_new)), fit));
    if (n == 0) return;   // (t0 may lie far past the table)
  }
  const int bt = 1 << p.log_scale;
  const int first = ((t0 >> p.log_scale) + m) << p.log_scale;   // first token of this block
  if (first >= t0 + n) return;
  const int lo = max(t0, first), hi = min(t0 + n, first + bt);  // new tokens [lo, hi) of the block
  const int blk = p.block_table[static_cast<size_t>(b) * p.max_pages + first / kBlkPage];
  // the new rows, in registers; the loads go out before the page id is looked at
  // (a row's chunks divide the item's threads: a thread's chunks lie a fixed step apart)
  const int chunks = (hi - lo) << p.log_chunks;
  const uint4* src = (is_v ? p.v_new : p.k_new) +
                     ((static_cast<size_t>(r0 + (lo - t0) + (it >> p.log_chunks)) * p.heads + g) << p.log_chunks) +
                     (it & ((1 << p.log_chunks) - 1));
  const int step = kItemThreads * p.heads;
  uint4 x[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) x[i] = it + i * kItemThreads < chunks ? __ldg(src + i * step) : make_uint4(0u, 0u, 0u, 0u);
  if (blk < 0 || blk >= p.num_blocks) {
    if (reporter) atomicOr(p.status, MFA_DEV_BAD_BLOCK);
    return;
  }
  const size_t ph = static_cast<size_t>(blk) * p.heads + g;      // (page, head)
  float* scale = (is_v ? p.v_scale : p.k_scale) + (ph << (6 - p.log_scale)) + ((first % kBlkPage) >> p.log_scale);
  uint8_t* rows = (is_v ? p.v_cache : p.k_cache) + (((ph * kBlkPage) << p.log_chunks) << 3);
  const bool begun = lo > first;
  const float s_old = begun ? *scale : 0.f;

  uint32_t bits = 0;   // (zeros past the rows)
#pragma unroll
  for (int i = 0; i < kChunks; ++i) bits = max_bits(bits, x[i]);
  if (max(bits & 0xFFFFu, bits >> 16) >= 0x7F80u) {   // infinities or NaN: they do not count
    bits = 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) bits = max_bits(bits, finite_only(x[i]));
  }
  float a = __uint_as_float(max(bits & 0xFFFFu, bits >> 16) << 16);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if constexpr (kItemThreads > 32) {
    const int it_item = threadIdx.x / kItemThreads;
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = a;
    named_bar_sync(1 + it_item, kItemThreads);   // (and every thread of the item has read s_old)
#pragma unroll
    for (int w = 0; w < kItemThreads / 32; ++w) a = fmaxf(a, wmax[it_item * (kItemThreads / 32) + w]);
  } else {
    __syncwarp();   // (every lane has read s_old before the first writes it anew)
  }
  const float need = pow2_scale(a);
  const float s = begun ? fmaxf(s_old, need) : need;
  const uint32_t sb = __float_as_uint(s);
  const bool exact_inv = (sb & 0x7FFFFFu) == 0u && sb >= (1u << 23) && sb <= (253u << 23);
  const float inv = __uint_as_float((254u << 23) - sb);   // 1 / s there
  uint2* dst = reinterpret_cast<uint2*>(rows);
  const int at = ((lo % kBlkPage) << p.log_chunks);       // first new row's chunk in the page
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
    if (it + i * kItemThreads < chunks)
      dst[at + it + i * kItemThreads] = exact_inv ? encode_chunk<true>(x[i], inv) : encode_chunk_by_division(x[i], s);
  if (begun && s > s_old) {
    const float r = __fdiv_rn(s_old, s);
    const int from = (first % kBlkPage) << p.log_chunks;
    for (int c = from + it; c < at; c += kItemThreads) {
      const uint2 old = dst[c];
      dst[c] = make_uint2(recode4(old.x, r), recode4(old.y, r));
    }
  }
  if (it == 0 && !(begun && s == s_old)) *scale = s;
}

mfa_status check_block_problem(const mfa_problem* pr, int scale_tokens) {
  if (pr == nullptr) return MFA_ERR_INVALID_ARG;
  if (pr->batch < 0 || pr->max_pages_per_seq < 1 || pr->num_blocks < 1) return MFA_ERR_INVALID_ARG;
  if (pr->tokens_per_seq < 1 || pr->tokens_per_seq > 4) return MFA_ERR_INVALID_ARG;
  if (pr->num_q_heads < 1 || pr->num_kv_heads < 1 || pr->head_dim < 1 || pr->page_size < 1 || scale_tokens < 1)
    return MFA_ERR_INVALID_ARG;
  if (pr->kv_dtype != MFA_KV_BF16 && pr->kv_dtype != MFA_KV_FP8_E4M3 && pr->kv_dtype != MFA_KV_MXFP4)
    return MFA_ERR_INVALID_ARG;
  if (pr->kv_shared != 0 && pr->kv_shared != 1) return MFA_ERR_INVALID_ARG;
  if (pr->out_dtype != MFA_OUT_BF16 && pr->out_dtype != MFA_OUT_FP32) return MFA_ERR_INVALID_ARG;
  if (!(pr->softmax_scale > 0.f && pr->softmax_scale <= 3.4028235e38f)) return MFA_ERR_INVALID_ARG;
  if (pr->num_q_heads % pr->num_kv_heads != 0) return MFA_ERR_INVALID_ARG;
  if (pr->kv_dtype != MFA_KV_FP8_E4M3 || pr->kv_shared != 0) return MFA_ERR_UNSUPPORTED;
  if (pr->page_size != kBlkPage || (pr->head_dim != 128 && pr->head_dim != 256)) return MFA_ERR_UNSUPPORTED;
  if (scale_tokens != 16 && scale_tokens != 32 && scale_tokens != 64) return MFA_ERR_UNSUPPORTED;
  if (pr->num_q_heads / pr->num_kv_heads > 64 || pr->num_kv_heads > 65536) return MFA_ERR_UNSUPPORTED;
  // sizes that 32-bit indices of tokens, rows and (page, head) pairs reach
  if (static_cast<long long>(pr->max_pages_per_seq) * kBlkPage > INT_MAX / 2) return MFA_ERR_INVALID_ARG;
  if (static_cast<long long>(pr->num_blocks) * pr->num_kv_heads > INT_MAX / 2) return MFA_ERR_INVALID_ARG;
  if (static_cast<long long>(pr->batch) * pr->tokens_per_seq > INT_MAX / 2 / pr->num_q_heads) return MFA_ERR_INVALID_ARG;
  return MFA_OK;
}

}  // namespace mfa

using namespace mfa;

extern "C" mfa_status mfa_block_kv_append(const mfa_problem* pr, int32_t scale_tokens, const void* k_new,
                                          const void* v_new, int32_t num_new, const int32_t* new_offsets,
                                          int32_t max_new, const int32_t* positions, const int32_t* block_table,
                                          void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                          uint32_t* device_status, void* stream_ptr) {
  const mfa_status st = check_block_problem(pr, scale_tokens);
  if (st != MFA_OK) return st;
  if (num_new < 0 || (device_status && !aligned(device_status, 4))) return MFA_ERR_INVALID_ARG;
  if (new_offsets == nullptr) {
    if (static_cast<long long>(pr->batch) * pr->tokens_per_seq != num_new) return MFA_ERR_INVALID_ARG;
    max_new = pr->tokens_per_seq;
  }
  if (pr->batch == 0 || num_new == 0) return MFA_OK;
  if (max_new < 1) return MFA_ERR_INVALID_ARG;
  if (!k_new || !v_new || !positions || !block_table || !k_cache || !v_cache || !k_scale || !v_scale)
    return MFA_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(k_scale, 16) || !aligned(v_scale, 16) || !aligned(positions, 4) || !aligned(block_table, 4) ||
      (new_offsets && !aligned(new_offsets, 4)))
    return MFA_ERR_INVALID_ARG;
  const int most_rows = std::min(max_new, num_new);
  // a run of n rows touches 1 + floor((n + scale_tokens - 2) / scale_tokens) blocks at most
  const long long most =
      std::min<long long>((static_cast<long long>(most_rows) + scale_tokens - 2) / scale_tokens + 1,
                          static_cast<long long>(pr->max_pages_per_seq) * (kBlkPage / scale_tokens));
  const long long items = pr->batch * most * pr->num_kv_heads * 2;
  // threads an item: kChunks chunks each of the rows that a block can get
  const int need = std::min(most_rows, static_cast<int>(scale_tokens)) * (pr->head_dim / 8) / kChunks;
  const int threads = need <= 32 ? 32 : need <= 64 ? 64 : need <= 128 ? 128 : 256;
  const long long ctas = (items * threads + kBlkThreads - 1) / kBlkThreads;
  if (ctas > INT_MAX) return MFA_ERR_INVALID_ARG;
  BlockAppendParams p;
  p.k_new = static_cast<const uint4*>(k_new);
  p.v_new = static_cast<const uint4*>(v_new);
  p.offsets = new_offsets;
  p.positions = positions;
  p.block_table = block_table;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.status = device_status;
  p.batch = pr->batch;
  p.tokens = pr->tokens_per_seq;
  p.num_new = num_new;
  p.max_new = most_rows;
  p.most_blocks = static_cast<int>(most);
  p.heads = pr->num_kv_heads;
  p.log_chunks = pr->head_dim == 256 ? 5 : 4;
  p.log_scale = scale_tokens == 64 ? 6 : scale_tokens == 32 ? 5 : 4;
  p.max_pages = pr->max_pages_per_seq;
  p.num_blocks = pr->num_blocks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(kBlkThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream_ptr);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void (*const fn)(BlockAppendParams) = threads == 32    ? mfa_block_append_kernel<32>
                                        : threads == 64  ? mfa_block_append_kernel<64>
                                        : threads == 128 ? mfa_block_append_kernel<128>
                                                         : mfa_block_append_kernel<256>;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
  if (e != cudaSuccess) return cuda_fail(e, "block append launch");
  return MFA_OK;
}
