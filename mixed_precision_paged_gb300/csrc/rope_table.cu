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

// a / 2^64 turns as half turns x within a quarter of zero, and the quarters q that were taken off. The 45 bits that
// follow the sign become fp32 in two steps without a conversion (an integer of 23 bits is the fraction of a float whose
// unit is 1); where they begin with 19 zeros or ones, the conversion keeps what lies further down.
__device__ __forceinline__ float half_turns(uint64_t a, uint32_t& q) {
  const uint32_t top = (uint32_t)(a >> 32);
  q = (top + 0x20000000u) >> 30;
  const int hi = (int)(top - (q << 30));
  const int x = hi >> 8;                                               // bits 40 .. 61 and the sign
  const uint32_t y = __funnelshift_l((uint32_t)a, (uint32_t)hi, 15) & 0x7fffffu;   // bits 17 .. 39
  if ((uint32_t)(x + 8) < 16u) return __ll2float_rn((long long)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)a)) * 0x1p-63f;
  const float fx = __int_as_float(0x4b400000 + x) - 12582912.f, fy = __uint_as_float(0x4b000000u | y) - 8388608.f;
  return fmaf(fx, 0x1p-23f, fy * 0x1p-46f);
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t x, y, z;
  float2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(x) : "l"(y), "l"(z));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(x));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// cos and sin of two angles a / 2^64 turns, times m. Taylor's series of sin(pi x) and cos(pi x) about 0, up to x^9 and
// x^10: what is left out is below 2^-28 of the value at |x| = 1/4. pi is taken in two parts, so that a sine is off by its
// argument's rounding, one of the sum and a little more.
__device__ __forceinline__ void cos_sin(uint64_t a, uint64_t b, float m, float2& c, float2& s) {
  constexpr double pi = 3.14159265358979323846, p2 = pi * pi;
  constexpr float hi = (float)pi, lo = (float)(pi - (double)hi);
  uint32_t q, r;
  float2 x;
  x.x = half_turns(a, q);
  x.y = half_turns(b, r);
  const float2 z = fma2(x, x, both(0.f));
  float2 u = fma2(z, both((float)(p2 * p2 * p2 * p2 * pi / 362880)), both((float)(-p2 * p2 * p2 * pi / 5040)));
  u = fma2(z, u, both((float)(p2 * p2 * pi / 120)));
  u = fma2(z, u, both((float)(-p2 * pi / 6)));
  u = fma2(z, u, both(lo));
  u = fma2(x, both(hi), fma2(x, u, both(0.f)));
  float2 v = fma2(z, both((float)(-p2 * p2 * p2 * p2 * p2 / 3628800)), both((float)(p2 * p2 * p2 * p2 / 40320)));
  v = fma2(z, v, both((float)(-p2 * p2 * p2 / 720)));
  v = fma2(z, v, both((float)(p2 * p2 / 24)));
  v = fma2(z, v, both((float)(-p2 / 2)));
  v = fma2(z, v, both(1.f));
  // the quarters: cos, sin of x + q / 2 half turns
  c.x = (q & 1u) ? u.x : v.x;
  s.x = (q & 1u) ? v.x : u.x;
  c.y = (r & 1u) ? u.y : v.y;
  s.y = (r & 1u) ? v.y : u.y;
  c.x *= __uint_as_float(__float_as_uint(m) ^ (((q + 1u) & 2u) << 30));
  s.x *= __uint_as_float(__float_as_uint(m) ^ ((q & 2u) << 30));
  c.y *= __uint_as_float(__float_as_uint(m) ^ (((r + 1u) & 2u) << 30));
  s.y *= __uint_as_float(__float_as_uint(m) ^ ((r & 2u) << 30));
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
    float2 c0, c1, s0, s1;
    cos_sin(a[0], a[1], p.magnitude, c0, s0);
    cos_sin(a[2], a[3], p.magnitude, c1, s1);
    *reinterpret_cast<float4*>(out) = make_float4(c0.x, c0.y, c1.x, c1.y);
    *reinterpret_cast<float4*>(out + p.half) = make_float4(s0.x, s0.y, s1.x, s1.y);
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
