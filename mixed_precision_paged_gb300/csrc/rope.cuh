// rope.cuh -- what the rotary cache writers share: the value row of a token in the form of its page.
#pragma once

#include "extend.cuh"
#include "micro.cuh"

namespace ekv {

__device__ __forceinline__ float2 word_values(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint32_t word_of(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 8 fp16 values as E4M3 codes of the IEEE quotient by s.
__device__ __forceinline__ uint2 e4m3_encode8(const uint4& x, float s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t out[2];
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w[i + 1]));
    out[i / 2] = (uint32_t)float2_to_e4m3x2(__fdiv_rn(a.x, s), __fdiv_rn(a.y, s)) |
                 ((uint32_t)float2_to_e4m3x2(__fdiv_rn(b.x, s), __fdiv_rn(b.y, s)) << 16);
  }
  return make_uint2(out[0], out[1]);
}

// The same out of line, for a loop that seldom needs it and is cold when it starts. (A call costs append_rope.cu's loop
// its registers: 65,536 tokens 291 against 250 us.)
static __device__ __noinline__ uint2 e4m3_encode8_apart(const uint4 x, float s) { return e4m3_encode8(x, s); }

// 16 values as E4M3 codes of the IEEE quotient by s; plain: they are finite and s is far from the ends of fp32's
// range, r = 1 / s, and the quotient takes three operations.
__device__ __forceinline__ bool far_from_ends(float s) { return s > 0x1p-64f && s < 0x1p64f; }
template <bool APART>
__device__ __forceinline__ uint4 e4m3_encode16(const uint4& a, const uint4& b, float s, float r, bool plain) {
  if (!plain) {
    const uint2 lo = APART ? e4m3_encode8_apart(a, s) : e4m3_encode8(a, s);
    const uint2 hi = APART ? e4m3_encode8_apart(b, s) : e4m3_encode8(b, s);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 x = word_values(w[i]), y = word_values(w[i + 1]);
    o[i / 2] = (uint32_t)float2_to_e4m3x2(div_by_scale(x.x, s, r), div_by_scale(x.y, s, r)) |
               ((uint32_t)float2_to_e4m3x2(div_by_scale(y.x, s, r), div_by_scale(y.y, s, r)) << 16);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The largest magnitude of 16 fp16 values, as bits, in either half of the result.
__device__ __forceinline__ uint32_t max_mag16(const uint4& a, const uint4& b) {
  return __vmaxu2(__vmaxu2(__vmaxu2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu), __vmaxu2(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu)),
                  __vmaxu2(__vmaxu2(b.x & 0x7fff7fffu, b.y & 0x7fff7fffu), __vmaxu2(b.z & 0x7fff7fffu, b.w & 0x7fff7fffu)));
}

// Unit u (16 values, a0 and a1) of row `trow` and KV head h of a page, in the page's form. mx2: the
// largest magnitude of the unit and its neighbour, which share a block of a microscaled row.
template <int D, bool APART>
__device__ __forceinline__ void store_value(const CacheView& c, int page, int mode, int trow, int h, int u, const uint4& a0,
                                            const uint4& a1, uint32_t mx2, int b) {
  uint8_t* vpage = const_cast<uint8_t*>(c.v_pages) + (size_t)page * c.v_page_stride;
  const int e0 = (trow * c.Hkv + h) * D + 16 * u;     // the unit's first element of the page
  if (mode == EKV_MODE_TARGET_FP16) {
    uint4* dst = reinterpret_cast<uint4*>(vpage + 2 * e0);
    dst[0] = a0;
    dst[1] = a1;
  } else if (mode == EKV_MODE_BASE) {
    *reinterpret_cast<uint4*>(vpage + e0) =
        make_uint4(__byte_perm(a0.x, a0.y, 0x7531), __byte_perm(a0.z, a0.w, 0x7531), __byte_perm(a1.x, a1.y, 0x7531),
                   __byte_perm(a1.z, a1.w, 0x7531));
  } else if (mode == EKV_MODE_COMPACT_E4M3) {
    const float s = !c.v_scales ? 0.f
                    : __ldg(c.v_scales + (c.scale_mode == EKV_SCALE_PER_TENSOR ? 0 : (size_t)page * c.Hkv + h));
    if (!scale_ok(s)) {
      report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SCALE, b);
      return;
    }
    const bool plain = max(mx2 & 0xffffu, mx2 >> 16) < 0x7c00u && far_from_ends(s);
    *reinterpret_cast<uint4*>(vpage + e0) = e4m3_encode16<APART>(a0, a1, s, __frcp_rn(s), plain);
  } else {
    const int k = micro_exponent(max(mx2 & 0xffffu, mx2 >> 16));
    uint8_t* slice = vpage + h * micro_head_bytes(D);
    *reinterpret_cast<uint2*>(slice + (trow * D + 16 * u) / 2) = make_uint2(micro_encode8(a0, k), micro_encode8(a1, k));
    if ((u & 1) == 0) slice[micro_scale_off(D) + (trow * D + 16 * u) / kMicroBlock] = (uint8_t)(127 + k);
  }
}

}  // namespace ekv
