// extend.cuh -- parameters of the calls that take new tokens: the rotary cache writer and
// the attention of new tokens over the paged cache.
#pragma once

#include "common.cuh"

namespace ekv {

// The cache, and the new tokens of its sequences.
struct CacheView {
  const __half* k_pages;
  const uint8_t* v_pages;
  long long v_page_stride;
  int num_pages;
  const float* v_scales;
  int scale_mode;
  const uint8_t* page_mode;
  int uniform_mode;
  const int32_t* block_table;
  int bt_stride;
  const int32_t* seq_lens;  // [batch], the new tokens included
  const int32_t* cu_q;      // [batch + 1]
  int batch;
  int total_q;
  int Hq, Hkv, D;
  int* err;
};

struct RopeAppendParams {
  CacheView c;              // (the kernel writes its pools)
  const __half* q;          // null: no queries
  const __half* k_new;
  const __half* v_new;
  long long q_stride, k_stride, v_stride;
  const float* rope;        // [rope_len][rope_dim]
  int rope_len, rope_dim, rope_style;
  __half* q_out;
};

// Pages of a sequence at most (2^21 tokens): keeps the block counts of the plan in 32 bits.
constexpr int kMaxExtendPages = 1 << 17;

struct ExtendParams {
  CacheView c;
  const __half* q;
  __half* out;
  float* lse;
  int G;
  int max_q;
  int window;               // 0x7fffffff: none
  float qscale;             // sm_scale * log2(e)
  int tile_tokens;          // tokens of a query tile
};

// The least b in [0, batch] with cu[b + 1] > i (batch: i lies behind the last sequence), found by
// the whole warp: 32 probes a step, so one step for a batch of 32 and three for 4,096.
__device__ __forceinline__ int warp_find_sequence(const int32_t* cu, int batch, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = batch;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int b = lo + (lane + 1) * step - 1;      // the last sequence of this lane's piece
    const bool before = b < hi && __ldg(cu + b + 1) <= i;
    const int pieces = __popc(__ballot_sync(0xffffffffu, before));
    lo += pieces * step;
    if (step == 1) return min(lo, hi);
    hi = min(hi, lo + step - 1);                   // the answer lies in [lo, lo + step - 1]
  }
  return lo;
}

cudaError_t launch_rope_append(const RopeAppendParams& p, int num_sms, cudaStream_t st);

}  // namespace ekv
