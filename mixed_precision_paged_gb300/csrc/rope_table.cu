// rope_table.cu -- cosines and sines of rotary positions, for the rotary cache writers.
//
// Angle of pair i at position t: 2 pi t w_i, w_i the turns a position (include/ekv.h: the frequencies of
// theta, divided where a context is stretched). Only the fraction of t w_i counts, and fp32 loses it: at
// t = 10^6 an angle of 10^6 radians has a step of 1/16. Here w_i is a 64-bit fixed-point fraction of a turn, so that t w_i
// wraps by itself: exact up to t 2^-65 turns, and the next row of a thread is one addition away. What
// lies beyond the nearest quarter turn goes to fp32 with all its bits, and the quarter is put back by swaps and signs.
// Writes 4 rope_dim bytes a position and reads nothing, so the floor is those bytes at HBM rate.
#include <math.h>

#include "rope_table.cuh"

namespace ekv {

namespace {

constexpr int kTableThreads = 256;

// cos and sin of a / 2^64 turns, times m.
__device__ __forceinline__ void cos_sin(uint64_t a, float m, float& c, float& s) {
  const uint32_t q = (uint32_t)((a + (1ull << 61)) >> 62);             // the nearest quarter
  const float x = __ll2float_rn((long long)(a - ((uint64_t)q << 62))) * 0x1p-63f;   // half turns, within 1/4
  float u, v;
  sincospif(x, &u, &v);
  const float cc = (q & 1u) ? u : v, ss = (q & 1u) ? v : u;
  c = ((q + 1u) & 2u) ? -m * cc : m * cc;
  s = (q & 2u) ? -m * ss : m * ss;
}

// A thread takes four pairs of a row, and every `step`-th row.
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const __grid_constant__ RopeTableParams p) {
  const int quads = p.half / 4, per_block = kTableThreads / quads;
  const int quad = (int)threadIdx.x % quads, lane = (int)threadIdx.x / quads;
  if (lane >= per_block) return;
  const int step = (int)gridDim.x * per_block;
  long long row = (int)blockIdx.x * per_block + lane;
  uint64_t a[4], d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t w = p.turns[4 * quad + i];
    a[i] = w * (uint64_t)(p.first + row);
    d[i] = w * (uint64_t)step;
  }
  float* out = p.table + (size_t)row * (2 * p.half) + 4 * quad;
  for (; row < p.rows; row += step) {
    float4 c, s;
    cos_sin(a[0], p.magnitude, c.x, s.x);
    cos_sin(a[1], p.magnitude, c.y, s.y);
    cos_sin(a[2], p.magnitude, c.z, s.z);
    cos_sin(a[3], p.magnitude, c.w, s.w);
    *reinterpret_cast<float4*>(out) = c;
    *reinterpret_cast<float4*>(out + p.half) = s;
    out += (size_t)step * (2 * p.half);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] += d[i];
  }
}

}  // namespace

void rope_turns(uint64_t* turns, int rope_dim, const ekv_rope_config& c) {
  const int half = rope_dim / 2;
  const double two_pi = 6.283185307179586476925;
  int lo = 0, hi = 0;
  if (c.scaling == EKV_ROPE_BY_DIMS) {
    // the pair that makes r turns over the original context, as a real number
    const double fast = rope_dim * log(c.original_len / (c.fast * two_pi)) / (2 * log(c.theta));
    const double slow = rope_dim * log(c.original_len / (c.slow * two_pi)) / (2 * log(c.theta));
    lo = (int)fmin(fmax(floor(fast), 0.0), rope_dim);
    hi = (int)fmax(fmin(ceil(slow), rope_dim - 1.0), -1.0);
  }
  for (int i = 0; i < half; ++i) {
    double w = pow(c.theta, -2.0 * i / rope_dim) / two_pi;
    double kept = 1.0;                                                 // the part of w that is not divided
    if (c.scaling == EKV_ROPE_LINEAR) kept = 0.0;
    if (c.scaling == EKV_ROPE_BY_TURNS) kept = (c.original_len * w - c.slow) / (c.fast - c.slow);
    if (c.scaling == EKV_ROPE_BY_DIMS) kept = hi > lo ? (double)(hi - i) / (hi - lo) : i <= lo ? 1.0 : 0.0;
    kept = fmin(1.0, fmax(0.0, kept));
    if (c.scaling != EKV_ROPE_PLAIN) w = w * kept + w / c.factor * (1.0 - kept);
    turns[i] = (uint64_t)ldexp(w, 64);                                 // w < 1/6: below 2^62
  }
}

cudaError_t launch_rope_table(const RopeTableParams& p, int num_sms, cudaStream_t st) {
  const int per_block = kTableThreads / (p.half / 4);
  const long long blocks = ((long long)p.rows + per_block - 1) / per_block, most = (long long)num_sms * 8;
  rope_table_kernel<<<(int)(blocks < most ? blocks : most), kTableThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace ekv
