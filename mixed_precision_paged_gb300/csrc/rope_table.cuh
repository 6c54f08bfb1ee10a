// rope_table.cuh -- parameters of the rotary table (rope_table.cu).
#pragma once

#include "common.cuh"

namespace ekv {

constexpr int kMaxRopePairs = 64;           // rope_dim / 2 at D = 128

struct RopeTableParams {
  float* table;                             // [rows][2 * half]
  int first, rows, half;
  float magnitude;
  uint64_t turns[kMaxRopePairs];            // of each pair, a position, in 2^-64 turns
};

// The turns of each pair under a configuration (already checked).
void rope_turns(uint64_t* turns, int rope_dim, const ekv_rope_config& c);
cudaError_t launch_rope_table(const RopeTableParams& p, int num_sms, cudaStream_t st);

}  // namespace ekv
