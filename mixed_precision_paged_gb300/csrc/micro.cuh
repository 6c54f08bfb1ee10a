// micro.cuh -- the microscaled FP4 value form (EKV_MODE_MICRO_FP4): its place in a page and
// its conversions.
//
// A block of 32 values of a token's head row shares a scale 2^k; a value is an E2M1 code
// (sign, 2 exponent bits, 1 fraction bit: 0, .5, 1, 1.5, 2, 3, 4, 6) times it. k is the
// least that keeps the block's largest magnitude a <= 6 * 2^k, so nothing saturates and
// the error of a value is at most half a step: 2^k (between 4 and 6 times 2^k), a fifth
// of a at worst (a = 5 * 2^k). k stays in [-24, 13]: below, fp16 has no finer values; above,
// 4 * 2^14 would leave fp16's range (a block whose maximum is over 49152 saturates there, 65504 by
// a quarter). So every code times its scale is an fp16 value, and the product with the attention
// weights needs no further rounding. (Under 2^-24 the codes .5 and 1.5 are not: fp16 values need none of
// them, and micro_decode8 rounds foreign ones to 0 and 2^-23.)
#pragma once

#include <cuda_fp4.h>

#include "common.cuh"

namespace ekv {

constexpr int kMicroBlock = 32;                    // values that share a scale
constexpr int kMicroKMin = -24, kMicroKMax = 13;   // scale exponents

// One KV head's slice of a page: 16 rows of D / 2 code bytes, then 16 rows of D / 32 scale bytes.
__host__ __device__ constexpr int micro_head_bytes(int D) { return kPage * (D / 2 + D / kMicroBlock); }
__host__ __device__ constexpr int micro_scale_off(int D) { return kPage * (D / 2); }

__device__ __forceinline__ bool micro_scale_ok(uint32_t byte) {
  return byte - (uint32_t)(127 + kMicroKMin) <= (uint32_t)(kMicroKMax - kMicroKMin);
}

// k of a block whose largest fp16 magnitude has the bits `mag` (sign cleared):
// 6 * 2^k = 1.5 * 2^(k + 2), so k + 2 is the exponent of a, one more if its fraction is over a half.
__device__ __forceinline__ int micro_exponent(uint32_t mag) {
  const uint32_t f = __float_as_uint(__half2float(__ushort_as_half((unsigned short)mag)));
  const int k = (int)(f >> 23) - 129 + ((f & 0x7fffffu) > 0x400000u ? 1 : 0);
  return max(kMicroKMin, min(kMicroKMax, k));
}

__device__ __forceinline__ float exp2_int(int k) { return __uint_as_float((uint32_t)(127 + k) << 23); }

// The codes of 8 fp16 values (two a register, the first low) under the scale 2^k: one
// byte for each two, the first value in its low half. The quotient by 2^k is exact in fp32.
__device__ __forceinline__ uint32_t micro_encode8(const uint4& x, int k) {
  const float inv = exp2_int(-k);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f.x *= inv;
    f.y *= inv;
    out |= (uint32_t)__nv_cvt_float2_to_fp4x2(f, __NV_E2M1, cudaRoundNearest) << (8 * i);
  }
  return out;
}

// fp16 2^k as a pair, k in [-24, 13] (below -14 a subnormal).
__device__ __forceinline__ __half2 micro_scale_h2(uint32_t byte) {
  return __float2half2_rn(__uint_as_float(byte << 23));
}

// The values of 8 codes (4 bytes) under a scale, as 4 registers of two fp16 each (exact, but .5 and
// 1.5 under 2^-24).
__device__ __forceinline__ uint4 micro_decode8(uint32_t codes, __half2 scale) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw r = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((codes >> (8 * i)) & 0xffu), __NV_E2M1);
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&r), scale);
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace ekv
