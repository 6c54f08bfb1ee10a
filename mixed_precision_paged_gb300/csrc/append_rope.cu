// append_rope.cu -- the rotary cache writer: new tokens of a ragged batch, their queries
// and keys rotated by the position, keys and values written into the pages.
//
// Per pair (u, w) of a head at angle a: (u cos a - w sin a, w cos a + u sin a), in fp32 from
// the caller's table, rounded once to fp16. Pure streaming: every input value is read once and
// every output written once (per token 2 B in and out of each query, key and FP16 value), plus
// the table row, which all heads of a token share: the floor is those bytes at HBM rate. 65,536 tokens of
// 32 + 2 x 8 heads of 128, FP16 pages: 252 us, 6.4 TB/s. (Consecutive tokens a warp, which saves look-ups, 259 us.)
//
// One warp takes a token, or a share of its heads when tokens are few. A lane owns unit u of a
// head, 16 values: with half-split pairs the 8-value vectors u and u + rope_dim / 16, so that
// both ends of 8 pairs meet in one lane; with interleaved pairs, and past rope_dim, the vectors
// 2u and 2u + 1. Either way its angles are 8u .. 8u + 7, loaded once and used for every head
// the lane sees. The rows of q, k and v are loaded before the sequence of the token is known (their
// addresses need the token's index only, once the end of the last sequence is known), so the search and the
// page lookups hide behind them.
#include "extend.cuh"
#include "micro.cuh"

namespace ekv {

constexpr int kRopeThreads = 128;
// Head rows a lane has in flight, 2 x 16 B each. 65,536 tokens of 48 rows: 4 rows 260 us, 6 rows 247 us, 8 rows
// (fewer warps fit) 333 us.
constexpr int kRopeRows = 6;

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

template <int D>
__global__ void __launch_bounds__(kRopeThreads)
rope_append_kernel(const RopeAppendParams p, int parts, int part_rows) {
  constexpr int UN = D / 16;                       // units of a head
  constexpr int SLOTS = 32 / UN;                   // head rows a warp works on at a time
  const CacheView& c = p.c;
  const int lane = threadIdx.x & 31;
  const int u = lane % UN, slot = lane / UN;
  const int warps = (int)gridDim.x * (kRopeThreads / 32);
  const int warp = (int)blockIdx.x * (kRopeThreads / 32) + (int)(threadIdx.x >> 5);
  const int nq = p.q ? c.Hq : 0;
  const int rows = nq + 2 * c.Hkv;                 // q heads, then k heads, then v heads
  const bool rot = 16 * u < p.rope_dim;
  // the two 8-value vectors of unit u: the rotated units of half-split pairs take the vectors
  // below rope_dim / 8, and 2u of the first unit past them is rope_dim / 8
  const bool split = rot && p.rope_style == 0;
  const int v0 = split ? u : 2 * u, v1 = split ? u + p.rope_dim / 16 : 2 * u + 1;
  // Rows behind the last sequence are not touched: k_new and v_new may end there.
  const int end = min(c.total_q, __ldg(c.cu_q + c.batch));
  const long long items = (long long)end * parts;
  // a sequence of fewer than no new tokens has no row that would show it
  for (int b = (int)blockIdx.x * kRopeThreads + (int)threadIdx.x; b < c.batch; b += (int)gridDim.x * kRopeThreads)
    if (__ldg(c.cu_q + b + 1) < __ldg(c.cu_q + b)) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SEQ_LEN, b);
  for (long long it = warp; it < items; it += warps) {
    const int i = (int)(it / parts), part = (int)(it % parts);
    int b = -1, t = 0, page = -1, mode = 0;
    bool ok = false, page_ok = false;
    float cs[8], sn[8];
    const int x1 = min(rows, (part + 1) * part_rows);
    for (int x0 = part * part_rows; x0 < x1; x0 += SLOTS * kRopeRows) {
      uint4 a0[kRopeRows], a1[kRopeRows];
#pragma unroll
      for (int r = 0; r < kRopeRows; ++r) {
        const int x = x0 + r * SLOTS + slot;
        if (x >= x1) continue;
        const bool is_v = x >= nq + c.Hkv;
        const __half* src = x < nq ? p.q + (size_t)i * p.q_stride + x * D
                            : !is_v ? p.k_new + (size_t)i * p.k_stride + (x - nq) * D
                                    : p.v_new + (size_t)i * p.v_stride + (x - nq - c.Hkv) * D;
        a0[r] = __ldg(reinterpret_cast<const uint4*>(src) + (is_v ? 2 * u : v0));
        a1[r] = __ldg(reinterpret_cast<const uint4*>(src) + (is_v ? 2 * u + 1 : v1));
      }
      if (b < 0) {                                 // first rows of the token: where it goes
        b = i < __ldg(c.cu_q) ? c.batch : warp_find_sequence(c.cu_q, c.batch, i);
        if (b < c.batch) {
          const int q0 = __ldg(c.cu_q + b), q1 = __ldg(c.cu_q + b + 1), len = __ldg(c.seq_lens + b);
          t = len - (q1 - i);
          ok = q0 >= 0 && i >= q0 && q1 - q0 <= len && (long long)len <= (long long)c.bt_stride * kPage && (p.rope_dim == 0 || t < p.rope_len);
          if (!ok && lane == 0) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SEQ_LEN, b);
        }
        if (!ok) break;
        if (rot) {
          const float* row = p.rope + (size_t)t * p.rope_dim + 8 * u;
          const float4 c0 = __ldg(reinterpret_cast<const float4*>(row)), c1 = __ldg(reinterpret_cast<const float4*>(row) + 1);
          const float4 s0 = __ldg(reinterpret_cast<const float4*>(row + p.rope_dim / 2));
          const float4 s1 = __ldg(reinterpret_cast<const float4*>(row + p.rope_dim / 2) + 1);
          cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w; cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
          sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w; sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
        }
        page = __ldg(c.block_table + (size_t)b * c.bt_stride + t / kPage);
        page_ok = page >= 0 && page < c.num_pages;
        if (!page_ok && lane == 0) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_PAGE_ID, b);
        if (page_ok) {
          mode = c.page_mode ? (int)__ldg(c.page_mode + page) : c.uniform_mode;
          if (mode > EKV_MODE_MICRO_FP4) {
            page_ok = false;
            if (lane == 0) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_PAGE_MODE, b);
          }
        }
      }
      const int trow = t % kPage;
#pragma unroll
      for (int r = 0; r < kRopeRows; ++r) {
        const int x = x0 + r * SLOTS + slot;
        if (x < x1 && x < nq + c.Hkv) {            // q or k: turned
          if (rot) {
            if (split) {
              rotate8(a0[r], a1[r], cs, sn);
            } else {
              rotate_pairs(a0[r], cs, sn);
              rotate_pairs(a1[r], cs + 4, sn + 4);
            }
          }
          if (x < nq || page_ok) {
            __half* dst = x < nq ? p.q_out + ((size_t)i * c.Hq + x) * D
                                 : const_cast<__half*>(c.k_pages) + (((size_t)page * kPage + trow) * c.Hkv + (x - nq)) * D;
            reinterpret_cast<uint4*>(dst)[v0] = a0[r];
            reinterpret_cast<uint4*>(dst)[v1] = a1[r];
          }
        }
        // v: in the form of its page. The block of a microscaled row is two units, in two lanes.
        uint32_t mx2 = 0;
        const bool is_v = x >= nq + c.Hkv && x < x1;
        if (is_v)
          mx2 = __vmaxu2(__vmaxu2(__vmaxu2(a0[r].x & 0x7fff7fffu, a0[r].y & 0x7fff7fffu),
                                  __vmaxu2(a0[r].z & 0x7fff7fffu, a0[r].w & 0x7fff7fffu)),
                         __vmaxu2(__vmaxu2(a1[r].x & 0x7fff7fffu, a1[r].y & 0x7fff7fffu),
                                  __vmaxu2(a1[r].z & 0x7fff7fffu, a1[r].w & 0x7fff7fffu)));
        mx2 = __vmaxu2(mx2, __shfl_xor_sync(0xffffffffu, mx2, 1));
        if (!is_v || !page_ok) continue;
        const int h = x - nq - c.Hkv;
        uint8_t* vpage = const_cast<uint8_t*>(c.v_pages) + (size_t)page * c.v_page_stride;
        const int e0 = (trow * c.Hkv + h) * D + 16 * u;     // the unit's first element of the page
        if (mode == EKV_MODE_TARGET_FP16) {
          uint4* dst = reinterpret_cast<uint4*>(vpage + 2 * e0);
          dst[0] = a0[r];
          dst[1] = a1[r];
        } else if (mode == EKV_MODE_BASE) {
          *reinterpret_cast<uint4*>(vpage + e0) =
              make_uint4(__byte_perm(a0[r].x, a0[r].y, 0x7531), __byte_perm(a0[r].z, a0[r].w, 0x7531),
                         __byte_perm(a1[r].x, a1[r].y, 0x7531), __byte_perm(a1[r].z, a1[r].w, 0x7531));
        } else if (mode == EKV_MODE_COMPACT_E4M3) {
          const float s = !c.v_scales ? 0.f
                          : __ldg(c.v_scales + (c.scale_mode == EKV_SCALE_PER_TENSOR ? 0 : (size_t)page * c.Hkv + h));
          if (!scale_ok(s)) {
            report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SCALE, b);
            continue;
          }
          const uint2 lo = e4m3_encode8(a0[r], s), hi = e4m3_encode8(a1[r], s);
          *reinterpret_cast<uint4*>(vpage + e0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
          const int k = micro_exponent(max(mx2 & 0xffffu, mx2 >> 16));
          uint8_t* slice = vpage + h * micro_head_bytes(D);
          *reinterpret_cast<uint2*>(slice + (trow * D + 16 * u) / 2) =
              make_uint2(micro_encode8(a0[r], k), micro_encode8(a1[r], k));
          if ((u & 1) == 0) slice[micro_scale_off(D) + (trow * D + 16 * u) / kMicroBlock] = (uint8_t)(127 + k);
        }
      }
    }
  }
}

cudaError_t launch_rope_append(const RopeAppendParams& p, int num_sms, cudaStream_t st) {
  if (p.c.total_q <= 0 || p.c.batch <= 0) return cudaSuccess;
  const int slots = 512 / p.c.D;
  const int rows = (p.q ? p.c.Hq : 0) + 2 * p.c.Hkv;
  // A warp takes a part of a token's rows: what its lanes hold in flight at once; or, while that leaves warps
  // idle (16 a processor), two rows a lane (32 tokens: 8.3 -> 6.3 us). The parts of a token are of
  // one size, so that the grid ends together.
  const int fit = (rows + slots * kRopeRows - 1) / (slots * kRopeRows), fine = (rows + 2 * slots - 1) / (2 * slots);
  const int want = p.c.total_q * (long long)fine <= (long long)num_sms * 16 ? fine : fit;
  const int part_rows = (rows + want * slots - 1) / (want * slots) * slots;
  const int parts = (rows + part_rows - 1) / part_rows;
  const long long warps = (long long)p.c.total_q * parts;
  const long long most = (long long)num_sms * 8;
  long long grid = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (grid > most) grid = most;
  if (p.c.D == 128) rope_append_kernel<128><<<(int)grid, kRopeThreads, 0, st>>>(p, parts, part_rows);
  else rope_append_kernel<64><<<(int)grid, kRopeThreads, 0, st>>>(p, parts, part_rows);
  return cudaGetLastError();
}

}  // namespace ekv
