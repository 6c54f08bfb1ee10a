// extend.cu -- attention of new tokens over the paged cache.
#include "extend.cuh"
#include "micro.cuh"

namespace ekv {

// One warp per (new token, query head): one pass over the keys it sees with the running
// maximum and sum of the softmax, a lane holding D / 32 columns.
template <int D>
__global__ void __launch_bounds__(128)
extend_kernel(const ExtendParams p) {
  constexpr int C = D / 32;
  const CacheView& c = p.c;
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int i = (int)(item / c.Hq), hq = (int)(item % c.Hq);
  if (i >= c.total_q || i < __ldg(c.cu_q)) return;
  const int b = warp_find_sequence(c.cu_q, c.batch, i);
  if (b >= c.batch) return;
  const int q0 = __ldg(c.cu_q + b), q1 = __ldg(c.cu_q + b + 1), len = __ldg(c.seq_lens + b);
  const int h = hq / p.G, d0 = lane * C;
  bool bad = i < q0 || q1 - q0 > len || q1 - q0 > p.max_q || (long long)len > (long long)c.bt_stride * kPage;
  if (bad && lane == 0) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SEQ_LEN, b);
  const int t = len - (q1 - i);
  const int lo = max(0, t - p.window + 1);
  float q[C], acc[C], m = -INFINITY, l = 0.f;
  for (int x = 0; x < C; ++x) {
    q[x] = __half2float(p.q[((size_t)i * c.Hq + hq) * D + d0 + x]);
    acc[x] = 0.f;
  }
  int page = -1, mode = 0;
  float vs = 1.f;
  for (int k = lo; k <= t && !bad; ++k) {
    if (k == lo || k % kPage == 0) {
      page = __ldg(c.block_table + (size_t)b * c.bt_stride + k / kPage);
      int detail = page < 0 || page >= c.num_pages ? EKV_DETAIL_PAGE_ID : EKV_DETAIL_NONE;
      if (!detail) mode = c.page_mode ? (int)__ldg(c.page_mode + page) : c.uniform_mode;
      if (!detail && mode > EKV_MODE_MICRO_FP4) detail = EKV_DETAIL_PAGE_MODE;
      vs = 1.f;
      if (!detail && mode == EKV_MODE_COMPACT_E4M3) {
        vs = !c.v_scales ? 0.f : __ldg(c.v_scales + (c.scale_mode == EKV_SCALE_PER_TENSOR ? 0 : (size_t)page * c.Hkv + h));
        if (!scale_ok(vs)) detail = EKV_DETAIL_SCALE;
      }
      bad = detail != EKV_DETAIL_NONE;
      if (bad) {
        if (lane == 0) report_error(c.err, EKV_ERR_DEVICE_CHECK, detail, b);
        break;
      }
    }
    const int row = k % kPage;
    float s = 0.f;
    const __half* kr = c.k_pages + (((size_t)page * kPage + row) * c.Hkv + h) * D + d0;
    for (int x = 0; x < C; ++x) s = fmaf(q[x], __half2float(kr[x]), s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.qscale;
    const float mn = fmaxf(m, s), a = exp2f(m - mn), w = exp2f(s - mn);
    l = fmaf(l, a, w);
    m = mn;
    const uint8_t* vp = c.v_pages + (size_t)page * c.v_page_stride;
    const int e0 = (row * c.Hkv + h) * D + d0;
    float v[C];
    if (mode == EKV_MODE_MICRO_FP4) {
      const uint8_t* slice = vp + h * micro_head_bytes(D);
      const uint32_t sb = slice[micro_scale_off(D) + (row * D + d0) / kMicroBlock];
      if (!micro_scale_ok(sb)) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SCALE, b);
      for (int x = 0; x < C; x += 2) {
        const __half2_raw r = __nv_cvt_fp4x2_to_halfraw2(slice[(row * D + d0 + x) / 2], __NV_E2M1);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
        const float e = micro_scale_ok(sb) ? __uint_as_float(sb << 23) : 0.f;
        v[x] = f.x * e;
        v[x + 1] = f.y * e;
      }
    } else {
      for (int x = 0; x < C; ++x)
        v[x] = mode == EKV_MODE_TARGET_FP16 ? __half2float(reinterpret_cast<const __half*>(vp)[e0 + x])
               : mode == EKV_MODE_BASE ? __half2float(__ushort_as_half((unsigned short)(vp[e0 + x] << 8)))
                                       : e4m3x2_to_float2(vp[e0 + x]).x * vs;
    }
    for (int x = 0; x < C; ++x) acc[x] = fmaf(w, v[x], acc[x] * a);
  }
  const float inv = bad ? 0.f : 1.f / l;
  for (int x = 0; x < C; ++x) p.out[((size_t)i * c.Hq + hq) * D + d0 + x] = __float2half_rn(bad ? 0.f : acc[x] * inv);
  if (lane == 0 && p.lse) p.lse[(size_t)i * c.Hq + hq] = bad ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

cudaError_t launch_extend(const ExtendParams& p, int num_sms, cudaStream_t st) {
  const long long blocks = ((long long)p.c.total_q * p.c.Hq + 3) / 4;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (p.c.D == 128) extend_kernel<128><<<(int)blocks, 128, 0, st>>>(p);
  else extend_kernel<64><<<(int)blocks, 128, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace ekv
