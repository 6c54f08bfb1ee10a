// rope_table.cu -- cosines and sines of rotary positions, for the rotary cache writers.
//
// Angle of pair i at position t: 2 pi t w_i, w_i the turns a position (include/ekv.h: the frequencies of
// theta, divided where a context is stretched). Only the fraction of t w_i counts, and fp32 loses it: at
// t = 10^6 an angle of 10^6 radians has a step of 1/16. Here w_i is a 64-bit fixed-point fraction of a turn, so that t w_i
// wraps by itself: off by at most t times w_i's error (a double's, and 2^-64), and the next row of a thread is one addition away. What
// lies beyond the nearest quarter turn goes to fp32 with all its bits, and the quarter is put back by swaps and signs.
// Writes 4 rope_dim bytes a position and reads nothing, so the floor is those bytes at HBM rate: 131,072 positions of 128
// values 9.9 us. With sincospif and 64-bit conversions 31 us, with both replaced (below) 14.7: 35 instructions an angle, the
// integer ones of which (reduction, quarters) fill two thirds of the ALU pipe; the launch and the first angles take the rest.
#include <math.h>

#include "rope_table.cuh"

namespace ekv {

namespace {

constexpr int kTableThreads = 256;

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
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t x, y;
  float2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(y));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(x));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The rest of a / 2^64 turns beyond the nearest quarter, in half turns, where it is small. (It stands apart, or the compiler
// takes it every time and discards it: the 64-bit conversion goes to the fp64 pipe, which then bounds the kernel.)
__device__ __noinline__ float near_quarter(uint64_t a) {
  return __ll2float_rn((long long)(a - ((a + (1ull << 61)) & (3ull << 62)))) * 0x1p-63f;
}

// The rest of a / 2^64 turns beyond the nearest quarter as half turns, of two angles; `near`: one lies near its quarter, and
// near_quarter has to take its place. With t = a's upper word + 2^29, t's upper two bits are the nearest quarter and the
// others, with 2^29 taken off and the 15 bits that follow, the rest: 45 bits, which become fp32 in two pieces without a
// conversion (an integer below 2^23 is the fraction of a float whose unit is 1) and one rounding of their sum; where they begin
// with 18 zeros or ones, near_quarter keeps what lies further down.
__device__ __forceinline__ float2 half_turns(uint64_t a, uint64_t b, bool& near) {
  constexpr float unit = 8388608.f + 2097152.f + 1.f;      // the floats' bases, and the 1 by which y's counts too much
  const uint32_t t = (uint32_t)(a >> 32) + 0x20000000u, r = (uint32_t)(b >> 32) + 0x20000000u;
  const float2 f = make_float2(__uint_as_float(((t >> 8) & 0x3fffffu) | 0x4b000000u) - unit,
                               __uint_as_float(((r >> 8) & 0x3fffffu) | 0x4b000000u) - unit);
  const float2 y = make_float2(__uint_as_float((__funnelshift_l((uint32_t)a, t, 15) & 0x7fffffu) | 0x4b000000u),
                               __uint_as_float((__funnelshift_l((uint32_t)b, r, 15) & 0x7fffffu) | 0x4b000000u));
  near = near || fminf(fabsf(f.x), fabsf(f.y)) < 9.f;
  return fma2(y, both(0x1p-46f), mul2(f, both(0x1p-23f)));
}

// cos and sin of two angles a, b / 2^64 turns, x beyond the nearest quarter, times m (of two equal halves): Taylor's series of
// sin(pi x) and cos(pi x) about 0, up to x^9 and x^10: what is left out is below 2^-28 of the value at |x| = 1/4. pi is taken in
// two parts, so that a sine is off by its argument's rounding, one of the sum and a little more.
__device__ __forceinline__ void cos_sin(uint64_t a, uint64_t b, float2 x, float2 m, float2& c, float2& s) {
  constexpr double pi = 3.14159265358979323846, p2 = pi * pi;
  constexpr float hi = (float)pi, lo = (float)(pi - (double)hi);
  const uint32_t t = (uint32_t)(a >> 32) + 0x20000000u, r = (uint32_t)(b >> 32) + 0x20000000u;
  const float2 z = mul2(x, x);
  float2 u = fma2(z, both((float)(p2 * p2 * p2 * p2 * pi / 362880)), both((float)(-p2 * p2 * p2 * pi / 5040)));
  u = fma2(z, u, both((float)(p2 * p2 * pi / 120)));
  u = fma2(z, u, both((float)(-p2 * pi / 6)));
  u = fma2(z, u, both(lo));
  u = mul2(fma2(x, both(hi), mul2(x, u)), m);
  float2 v = fma2(z, both((float)(-p2 * p2 * p2 * p2 * p2 / 3628800)), both((float)(p2 * p2 * p2 * p2 / 40320)));
  v = fma2(z, v, both((float)(-p2 * p2 * p2 / 720)));
  v = fma2(z, v, both((float)(p2 * p2 / 24)));
  v = fma2(z, v, both((float)(-p2 / 2)));
  v = mul2(fma2(z, v, both(1.f)), m);
  // the quarters: an odd one exchanges the two, the upper half turn changes both signs, the second and third quarter the cosine's
  auto put = [](uint32_t q, float uu, float vv, float& cc, float& ss) {
    const bool odd = q & 0x40000000u;
    cc = __uint_as_float(__float_as_uint(odd ? uu : vv) ^ ((q ^ (q << 1)) & 0x80000000u));
    ss = __uint_as_float(__float_as_uint(odd ? vv : uu) ^ (q & 0x80000000u));
  };
  put(t, u.x, v.x, c.x, s.x);
  put(r, u.y, v.y, c.y, s.y);
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
  const float2 m = both(p.magnitude);
  float* out = p.table + (size_t)row * (2 * p.half) + 4 * quad;
  for (; row < p.rows; row += step) {
    float2 c0, c1, s0, s1;
    bool near = false;
    float2 x0 = half_turns(a[0], a[1], near), x1 = half_turns(a[2], a[3], near);
    if (near) {
      x0 = make_float2(near_quarter(a[0]), near_quarter(a[1]));
      x1 = make_float2(near_quarter(a[2]), near_quarter(a[3]));
    }
    cos_sin(a[0], a[1], x0, m, c0, s0);
    cos_sin(a[2], a[3], x1, m, c1, s1);
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
