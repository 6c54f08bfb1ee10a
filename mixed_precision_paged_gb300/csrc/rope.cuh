// rope.cuh -- what the rotary cache writers share: norm and rotation of a head row's values, and the value
// row of a token in the form of its page.
#pragma once

#include "extend.cuh"
#include "micro.cuh"

namespace ekv {

// 8 pairs (lo[j], hi[j]) turned by (c[j], s[j]).
__device__ __forceinline__ void rotate8(uint4& lo, uint4& hi, const float (&c)[8], const float (&s)[8]) {
  uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&a[i]));
    const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&b[i]));
    const __half2 x = __floats2half2_rn(u.x * c[2 * i] - w.x * s[2 * i], u.y * c[2 * i + 1] - w.y * s[2 * i + 1]);
    const __half2 y = __floats2half2_rn(w.x * c[2 * i] + u.x * s[2 * i], w.y * c[2 * i + 1] + u.y * s[2 * i + 1]);
    a[i] = *reinterpret_cast<const uint32_t*>(&x);
    b[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  lo = make_uint4(a[0], a[1], a[2], a[3]);
  hi = make_uint4(b[0], b[1], b[2], b[3]);
}

// 8 interleaved pairs over two vectors turned by (c[j], s[j]).
__device__ __forceinline__ void rotate_pairs(uint4& v, const float* c, const float* s) {
  uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&a[i]));
    const __half2 x = __floats2half2_rn(u.x * c[i] - u.y * s[i], u.y * c[i] + u.x * s[i]);
    a[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
  v = make_uint4(a[0], a[1], a[2], a[3]);
}

__device__ __forceinline__ float2 word_values(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint32_t word_of(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The sum of the squares of 8 values, added to s.
__device__ __forceinline__ float add_squares(const uint4& v, float s) {
  const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = word_values(a[i]);
    s = fmaf(x.x, x.x, fmaf(x.y, x.y, s));
  }
  return s;
}

// 16 values of a head row, lo and hi, times inv and their weights, then turned where `rot`: with `split` pairs
// (lo[j], hi[j]) by angle j, else neighbours, lo's by angles 0 .. 3 and hi's by 4 .. 7. fp32 up to the last step.
__device__ __forceinline__ void scale_and_turn(uint4& lo, uint4& hi, float inv, const uint4& wlo, const uint4& whi, bool rot,
                                               bool split, const float (&c)[8], const float (&s)[8]) {
  uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
  const uint32_t u[4] = {wlo.x, wlo.y, wlo.z, wlo.w}, w[4] = {whi.x, whi.y, whi.z, whi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x = word_values(a[i]), y = word_values(b[i]);
    const float2 wx = word_values(u[i]), wy = word_values(w[i]);
    x.x *= inv * wx.x;
    x.y *= inv * wx.y;
    y.x *= inv * wy.x;
    y.y *= inv * wy.y;
    if (rot) {
      const float2 f = x, g = y;
      if (split) {
        x = make_float2(f.x * c[2 * i] - g.x * s[2 * i], f.y * c[2 * i + 1] - g.y * s[2 * i + 1]);
        y = make_float2(g.x * c[2 * i] + f.x * s[2 * i], g.y * c[2 * i + 1] + f.y * s[2 * i + 1]);
      } else {
        x = make_float2(f.x * c[i] - f.y * s[i], f.y * c[i] + f.x * s[i]);
        y = make_float2(g.x * c[4 + i] - g.y * s[4 + i], g.y * c[4 + i] + g.x * s[4 + i]);
      }
    }
    a[i] = word_of(x.x, x.y);
    b[i] = word_of(y.x, y.y);
  }
  lo = make_uint4(a[0], a[1], a[2], a[3]);
  hi = make_uint4(b[0], b[1], b[2], b[3]);
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

// The largest magnitude of 16 fp16 values, as bits, in either half of the result.
__device__ __forceinline__ uint32_t max_mag16(const uint4& a, const uint4& b) {
  return __vmaxu2(__vmaxu2(__vmaxu2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu), __vmaxu2(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu)),
                  __vmaxu2(__vmaxu2(b.x & 0x7fff7fffu, b.y & 0x7fff7fffu), __vmaxu2(b.z & 0x7fff7fffu, b.w & 0x7fff7fffu)));
}

// Unit u (16 values, a0 and a1) of row `trow` and KV head h of a page, in the page's form. mx2: the
// largest magnitude of the unit and its neighbour, which share a block of a microscaled row.
template <int D>
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
    const uint2 lo = e4m3_encode8(a0, s), hi = e4m3_encode8(a1, s);
    *reinterpret_cast<uint4*>(vpage + e0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  } else {
    const int k = micro_exponent(max(mx2 & 0xffffu, mx2 >> 16));
    uint8_t* slice = vpage + h * micro_head_bytes(D);
    *reinterpret_cast<uint2*>(slice + (trow * D + 16 * u) / 2) = make_uint2(micro_encode8(a0, k), micro_encode8(a1, k));
    if ((u & 1) == 0) slice[micro_scale_off(D) + (trow * D + 16 * u) / kMicroBlock] = (uint8_t)(127 + k);
  }
}

}  // namespace ekv
