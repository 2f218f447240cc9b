// Decode attention over a block-scaled 8-bit KV cache (GB300, sm_103a): e4m3 codes with one
// fp32 scale for each block of tokens and key/value head.
//
// For token i of sequence b and query head h, over the tokens t that it sees:
//     s_t = softmax_scale * sk_t * dot(q, k_t),  out = sum_t e^(s_t) sv_t v_t / sum_t e^(s_t),
//     lse = ln sum_t e^(s_t),
// k_t and v_t being the e4m3 codes' values and sk_t, sv_t their blocks' scales.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstring>
#include <vector>

#include "mfa.h"
#include "mfa_host.h"
#include "ptx.cuh"

namespace mfa {

constexpr int kBPage = 64;
constexpr int kBTile = 128;           // tokens of a tile (two pages)
constexpr int kBRows = 64;            // query rows (new tokens x heads of one group) a unit holds at most
constexpr int kBCostTile = 4;         // schedule: cost of a tile
constexpr int kBCostUnit = 6;         // and of a unit boundary inside a CTA's range
constexpr int kBMaxSeg = 256;         // units that one CTA can meet
constexpr uint64_t kBWsHeader = 256;

// The work of one problem: a unit is (sequence, key/value head, group of new tokens); its rows
// are the group's new tokens x the query heads that read that head.
struct BlockShape {
  int group;      // query heads of a key/value head
  int unit_tokens;   // new tokens of a unit
  int token_groups;  // units along the new tokens
  int readers;    // units of a sequence
  int rows;       // rows of a unit (its last token group may use fewer)
};

static BlockShape block_shape(const mfa_problem* pr) {
  BlockShape s;
  s.group = pr->num_q_heads / pr->num_kv_heads;
  s.unit_tokens = std::min(pr->tokens_per_seq, kBRows / s.group);
  s.token_groups = (pr->tokens_per_seq + s.unit_tokens - 1) / s.unit_tokens;
  s.readers = s.token_groups * pr->num_kv_heads;
  s.rows = s.group * s.unit_tokens;
  return s;
}

static uint64_t block_lse_offset(long long partials, int rows, int d) {
  const uint64_t x = kBWsHeader + static_cast<uint64_t>(partials) * rows * d * 4;
  return (x + 255) / 256 * 256;
}
static uint64_t block_workspace_bytes(long long partials, int rows, int d) {
  return (block_lse_offset(partials, rows, d) + static_cast<uint64_t>(partials) * rows * 4 + 255) / 256 * 256;
}

struct BlockDecodeParams {
  const __nv_bfloat16* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  void* out;
  float* lse;
  unsigned int* status;
  int batch, tokens, heads, kv_heads;
  int log_scale;       // log2(scale_tokens)
  int max_pages, num_blocks;
  float scale_log2;    // softmax_scale * log2(e)
  int out_f32;
};

// One CTA per (sequence, new token, query head); each warp walks every eighth token with a
// running maximum and sum, and the eight states are merged at the end.
template <int kDim>
__global__ void __launch_bounds__(256) mfa_block_decode_kernel(const __grid_constant__ BlockDecodeParams p) {
  constexpr int kPer = kDim / 32;
  __shared__ float sm[8], sl[8], so[8][kDim];
  grid_dep_wait();
  grid_dep_launch();
  const int x = blockIdx.x, h = blockIdx.y, b = x / p.tokens, i = x % p.tokens;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = h / (p.heads / p.kv_heads);
  int L = p.seq_lens[b];
  if (L < 0 || L > p.max_pages * kBPage) {
    if (threadIdx.x == 0) atomicOr(p.status, MFA_DEV_BAD_LENGTH);
    L = min(max(L, 0), p.max_pages * kBPage);
  }
  const int n = max(0, L - (p.tokens - 1) + i);
  const size_t row = static_cast<size_t>(x) * p.heads + h;
  float q[kPer], acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    q[e] = __bfloat162float(p.q[row * kDim + lane * kPer + e]);
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  auto load = [&](const uint8_t* base, float (&v)[kPer]) {
#pragma unroll
    for (int e = 0; e < kPer; e += 4) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(base + lane * kPer + e);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t f;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(static_cast<uint16_t>(w >> (16 * k))));
        const __half2 f2 = *reinterpret_cast<const __half2*>(&f);
        v[e + 2 * k] = __low2float(f2);
        v[e + 2 * k + 1] = __high2float(f2);
      }
    }
  };
  for (int t = warp; t < n; t += 8) {
    const int blk = p.block_table[static_cast<size_t>(b) * p.max_pages + t / kBPage];
    float kv[kPer], vv[kPer], sk = 0.f, sv = 0.f;
    if (blk >= 0 && blk < p.num_blocks) {
      const size_t ph = static_cast<size_t>(blk) * p.kv_heads + g;
      load(p.k_cache + (ph * kBPage + t % kBPage) * kDim, kv);
      load(p.v_cache + (ph * kBPage + t % kBPage) * kDim, vv);
      const size_t si = (ph << (6 - p.log_scale)) + ((t % kBPage) >> p.log_scale);
      sk = p.k_scale[si];
      sv = p.v_scale[si];
    } else {
      if (lane == 0) atomicOr(p.status, MFA_DEV_BAD_BLOCK);
#pragma unroll
      for (int e = 0; e < kPer; ++e) kv[e] = vv[e] = 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) s += q[e] * kv[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.scale_log2 * sk;
    const float mn = fmaxf(m, s), al = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * al + w;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = acc[e] * al + w * sv * vv[e];
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) so[warp][lane * kPer + e] = acc[e];
  __syncthreads();
  float M = -INFINITY, S = 0.f;
  for (int w = 0; w < 8; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < 8; ++w) S += sm[w] == -INFINITY ? 0.f : sl[w] * exp2f(sm[w] - M);
  for (int d = threadIdx.x; d < kDim; d += 256) {
    float o = 0.f;
    for (int w = 0; w < 8; ++w) o += sm[w] == -INFINITY ? 0.f : so[w][d] * exp2f(sm[w] - M);
    o = n > 0 ? o / S : 0.f;
    if (p.out_f32)
      static_cast<float*>(p.out)[row * kDim + d] = o;
    else
      static_cast<__nv_bfloat16*>(p.out)[row * kDim + d] = __float2bfloat16_rn(o);
  }
  if (threadIdx.x == 0 && p.lse != nullptr) p.lse[row] = n > 0 ? M * 0.6931471805599453f + logf(S) : -INFINITY;
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
  long long tiles = 0, nonempty = 0;   // of one reader of each sequence
  if (host_seq_lens != nullptr) {
    for (int b = 0; b < pr->batch; ++b) {
      if (host_seq_lens[b] < 0 || host_seq_lens[b] > cap) return MFA_ERR_INVALID_ARG;
      tiles += (host_seq_lens[b] + kBTile - 1) / kBTile;
      nonempty += host_seq_lens[b] > 0;
    }
  } else {
    if (max_seq_len < 0 || max_seq_len > cap) return MFA_ERR_INVALID_ARG;
    tiles = static_cast<long long>(pr->batch) * ((max_seq_len + kBTile - 1) / kBTile);
    nonempty = max_seq_len > 0 ? pr->batch : 0;
  }
  if (num_sms <= 0) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
  }
  const long long W = tiles * sh.readers, N = nonempty * sh.readers;
  const long long C = kBCostTile * W + kBCostUnit * std::max(N - 1, 0ll);
  // a CTA's share of at most ceil(C / G) holds that over (tile + boundary) whole units and two
  // parts of units
  const long long share = static_cast<long long>(kBMaxSeg - 2) * (kBCostTile + kBCostUnit);
  const long long least = std::max(1ll, (C + share - 1) / share);
  long long G = force_ctas > 0 ? force_ctas : std::max(std::min<long long>(W, num_sms), least);
  if (G < least) return MFA_ERR_INVALID_ARG;
  const long long partials = static_cast<long long>(pr->batch) * sh.readers + G - 1;
  if (G > INT_MAX / 2 || partials > INT_MAX / 2 / sh.rows) return MFA_ERR_INVALID_ARG;
  std::memset(plan, 0, sizeof(*plan));
  plan->num_ctas = static_cast<int32_t>(G);
  plan->tile_tokens = kBTile;
  plan->max_tiles_per_cta = static_cast<int32_t>(std::min<long long>((C + G - 1) / G / kBCostTile + 1, std::max(W, 1ll)));
  plan->num_partials = static_cast<int32_t>(partials);
  plan->batch = pr->batch;
  plan->tokens_per_seq = pr->tokens_per_seq;
  plan->kv_dtype = pr->kv_dtype;
  plan->flags = flags;
  plan->num_sms = num_sms;
  plan->total_tiles = static_cast<uint64_t>(W);
  plan->workspace_bytes = block_workspace_bytes(partials, sh.rows, pr->head_dim);
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
  if (plan->batch != pr->batch || plan->kv_dtype != pr->kv_dtype || plan->tokens_per_seq != pr->tokens_per_seq ||
      plan->num_ctas < 1 || (plan->flags & ~(MFA_PLAN_CHECK | MFA_PLAN_EARLY_METADATA)) != 0 ||
      plan->num_partials != static_cast<long long>(pr->batch) * sh.readers + plan->num_ctas - 1 ||
      plan->workspace_bytes != block_workspace_bytes(plan->num_partials, sh.rows, pr->head_dim))
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
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = out;
  p.lse = lse;
  p.status = static_cast<unsigned int*>(workspace);
  p.batch = pr->batch;
  p.tokens = pr->tokens_per_seq;
  p.heads = pr->num_q_heads;
  p.kv_heads = pr->num_kv_heads;
  p.log_scale = scale_tokens == 64 ? 6 : scale_tokens == 32 ? 5 : 4;
  p.max_pages = pr->max_pages_per_seq;
  p.num_blocks = pr->num_blocks;
  p.scale_log2 = static_cast<float>(static_cast<double>(pr->softmax_scale) * 1.4426950408889634);
  p.out_f32 = pr->out_dtype == MFA_OUT_FP32 ? 1 : 0;
  const bool check = (plan->flags & MFA_PLAN_CHECK) != 0;
  cudaError_t e = cudaSuccess;
  if (check && (e = cudaMemsetAsync(workspace, 0, 4, stream)) != cudaSuccess) return cuda_fail(e, "memset");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pr->batch) * pr->tokens_per_seq, static_cast<unsigned>(pr->num_q_heads), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = pr->head_dim == 256 ? cudaLaunchKernelEx(&cfg, mfa_block_decode_kernel<256>, p)
                          : cudaLaunchKernelEx(&cfg, mfa_block_decode_kernel<128>, p);
  if (e != cudaSuccess) return cuda_fail(e, "block decode launch");
  if (check) {
    uint32_t word = 0;
    if ((e = cudaMemcpyAsync(&word, workspace, 4, cudaMemcpyDeviceToHost, stream)) != cudaSuccess)
      return cuda_fail(e, "copy");
    if ((e = cudaStreamSynchronize(stream)) != cudaSuccess) return cuda_fail(e, "sync");
    if (word != 0) return MFA_ERR_DEVICE_CHECK;
  }
  return MFA_OK;
}
