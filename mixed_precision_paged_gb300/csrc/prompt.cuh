// prompt.cuh -- parameters of the attention of packed prompts (prompt_tc05.cu).
#pragma once

#include "common.cuh"

namespace ekv {

constexpr int kMaxPromptRows = 1 << 24;     // rows of a call: keeps the item counts in 32 bits

struct PromptParams {
  const __half* q;                          // rows of [Hq][D], q_stride values apart; k and v likewise
  const __half* k;
  const __half* v;
  long long q_stride, k_stride, v_stride;
  const int32_t* cu;                        // [n + 1]
  __half* out;                              // [total][Hq][D]
  float* lse;                               // [total][Hq] or null
  int n, total, Hq, Hkv, G;
  int heads;                                // query heads that a tile packs: 1 or G
  int tile_tokens;                          // 128 / heads
  int window;                               // 0x7fffffff: none
  float qscale;                             // sm_scale * log2(e)
  int* err;
#ifdef EKV_TEST_WAIT_TIMEOUT
  int inject_timeout;                       // test build only: the wait of CTA 0 that runs out, see the kernel; 0: none
#endif
};

cudaError_t launch_prompt_tc05(PromptParams p, int D, int num_sms, cudaStream_t st);

}  // namespace ekv
