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
#include "rope.cuh"

namespace ekv {

constexpr int kRopeThreads = 128;
// Head rows a lane has in flight, 2 x 16 B each. 65,536 tokens of 48 rows: 4 rows 260 us, 6 rows 247 us, 8 rows
// (fewer warps fit) 333 us.
constexpr int kRopeRows = 6;
constexpr int kNormRows = 6, kNormBlocks = 4;   // the same with norms, and blocks that share a processor

// ------------------------------------------------------- E4M3 pages whose scales grow
// Values of one page and KV head by one warp: the rows that the call writes stay in registers while their largest
// magnitude a is found, so every value is read once and every code written once (3 bytes a value).
//   the call writes row 0:  s = max(a, 2^-24) / 448 (the scale of a demotion, of which one lies above zero)
//   else:                   s = s_old 2^k, k >= 0 the least with 448 s_old 2^k >= a; earlier rows' codes are
//                           divided by 2^k, which loses nothing but what falls below the format's least.
// Infinities count as fp16's largest value and saturate, NaN counts for nothing and keeps a code of its own.
__device__ __forceinline__ uint32_t finite_mag(uint32_t mag) {   // of two fp16 magnitudes
  return __vminu2(mag, 0x7bff7bffu) & ~__vcmpgtu2(mag, 0x7c007c00u);
}
__device__ __forceinline__ uint32_t finite_mag16(const uint4& a, const uint4& b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, finite_mag(w[i] & 0x7fff7fffu));
  return m;
}

// 16 values as E4M3 codes of the IEEE quotient by s; plain: they are finite and s is far from the ends of fp32's range, r = 1 / s.
__device__ __forceinline__ uint4 e4m3_encode16(const uint4& a, const uint4& b, float s, float r, bool plain) {
  if (!plain) {
    const uint2 lo = e4m3_encode8(a, s), hi = e4m3_encode8(b, s);
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

// 4 codes times f, rounded to codes again.
__device__ __forceinline__ uint32_t e4m3_rescale4(uint32_t codes, float f) {
  const float2 a = e4m3x2_to_float2((uint16_t)codes), b = e4m3x2_to_float2((uint16_t)(codes >> 16));
  return (uint32_t)float2_to_e4m3x2(a.x * f, a.y * f) | ((uint32_t)float2_to_e4m3x2(b.x * f, b.y * f) << 16);
}

// Warps `warp`, `warp + warps`, ... of the items (chunk of token rows, KV head). An item takes the pages whose first new
// row lies in its chunk: a page's rows may go on behind it.
template <int D>
__device__ __forceinline__ void grow_values(const RopeAppendParams& p, int warp, int warps, int chunk, int end) {
  constexpr int UN = D / 16, SLOTS = 32 / UN, NP = kPage / SLOTS;
  const CacheView& c = p.c;
  const int lane = threadIdx.x & 31, u = lane % UN, slot = lane / UN;
  const long long items = (long long)((end + chunk - 1) / chunk) * c.Hkv;
  const int start = __ldg(c.cu_q);
  for (long long it = warp; it < items; it += warps) {
    const int h = (int)(it % c.Hkv), i0 = (int)(it / c.Hkv) * chunk, i = i0 + lane;
    // a lane's row of the chunk: where it goes, and how many rows its page takes from it on
    int t = 0, rows = 0, page = 0, mode = 0, b = 0;
    const int b0 = i0 < start ? 0 : warp_find_sequence(c.cu_q, c.batch, i0);
    if (lane < chunk && i < end && i >= start) {
      int hi = c.batch;                                  // the least b with cu_q[b + 1] > i
      b = b0;
      if (b < hi && __ldg(c.cu_q + b + 1) <= i)
        while (b < hi) {
          const int mid = (b + hi) >> 1;
          if (__ldg(c.cu_q + mid + 1) <= i) b = mid + 1;
          else hi = mid;
        }
      if (b < c.batch) {
        const int q0 = __ldg(c.cu_q + b), q1 = __ldg(c.cu_q + b + 1), len = __ldg(c.seq_lens + b);
        t = len - (q1 - i);
        // (what fails is reported where queries and keys are written)
        if (q0 >= 0 && i >= q0 && q1 - q0 <= len && (long long)len <= (long long)c.bt_stride * kPage &&
            (i == q0 || t % kPage == 0)) {
          rows = min(kPage - t % kPage, min(q1, end) - i);
          if (p.rope_dim > 0) rows = min(rows, p.rope_len - t);
          if (rows > 0) {
            page = __ldg(c.block_table + (size_t)b * c.bt_stride + t / kPage);
            if (page < 0 || page >= c.num_pages) rows = 0;
            else mode = c.page_mode ? (int)__ldg(c.page_mode + page) : c.uniform_mode;
            if (mode > EKV_MODE_MICRO_FP4) rows = 0;
          }
        }
      }
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, rows > 0); left; left &= left - 1) {
      const int src = __ffs(left) - 1;
      const int r0 = __shfl_sync(0xffffffffu, t, src) % kPage, n = __shfl_sync(0xffffffffu, rows, src);
      const int pg = __shfl_sync(0xffffffffu, page, src), md = __shfl_sync(0xffffffffu, mode, src);
      const int sb = __shfl_sync(0xffffffffu, b, src);
      uint4 a0[NP], a1[NP];
#pragma unroll
      for (int x = 0; x < NP; ++x) {
        const int row = x * SLOTS + slot;                // of the rows from r0 on
        a0[x] = a1[x] = make_uint4(0u, 0u, 0u, 0u);
        if (row < n) {
          const uint4* v = reinterpret_cast<const uint4*>(p.v_new + (size_t)(i0 + src + row) * p.v_stride + h * D) + 2 * u;
          a0[x] = __ldg(v);
          a1[x] = __ldg(v + 1);
        }
      }
      if (md != EKV_MODE_COMPACT_E4M3) {
#pragma unroll
        for (int x = 0; x < NP; ++x) {
          uint32_t mx2 = max_mag16(a0[x], a1[x]);
          mx2 = __vmaxu2(mx2, __shfl_xor_sync(0xffffffffu, mx2, 1));
          const int row = x * SLOTS + slot;
          if (row < n) store_value<D>(c, pg, md, r0 + row, h, u, a0[x], a1[x], mx2, sb);
        }
        continue;
      }
      float* scale = const_cast<float*>(c.v_scales) + (size_t)pg * c.Hkv + h;
      float s = r0 > 0 ? *scale : 0.f;
      uint32_t m2 = 0;
#pragma unroll
      for (int x = 0; x < NP; ++x) m2 = __vmaxu2(m2, max_mag16(a0[x], a1[x]));
      uint32_t mag = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
      const bool finite = mag < 0x7c00u;
      if (!finite) {
        m2 = 0;
#pragma unroll
        for (int x = 0; x < NP; ++x) m2 = __vmaxu2(m2, finite_mag16(a0[x], a1[x]));
        mag = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
      }
      const float a = __half2float(__ushort_as_half((unsigned short)mag));
      uint8_t* base = const_cast<uint8_t*>(c.v_pages) + (size_t)pg * c.v_page_stride + h * D + 16 * u;
      if (r0 == 0) {
        s = __fdiv_rn(fmaxf(a, 0x1p-24f), 448.f);
        if (lane == 0) *scale = s;
      } else {
        if (!scale_ok(s)) {
          if (lane == 0) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SCALE, sb);
          continue;
        }
        const float top = __fmul_rn(s, 448.f);
        if (a > top) {
          int ea, et;
          const float ma = frexpf(a, &ea), mt = frexpf(top, &et);
          const int k = ea - et + (ma > mt ? 1 : 0);     // least k with top 2^k >= a
          const float f = k < 126 ? ldexpf(1.f, -k) : 0.f;   // (2^-126 of a code is zero)
          for (int row = slot; row < r0; row += SLOTS) {
            uint4* at = reinterpret_cast<uint4*>(base + (size_t)row * c.Hkv * D);
            uint4 q = *at;
            q = make_uint4(e4m3_rescale4(q.x, f), e4m3_rescale4(q.y, f), e4m3_rescale4(q.z, f), e4m3_rescale4(q.w, f));
            *at = q;
          }
          s = ldexpf(s, k);
          __syncwarp();                                  // every lane has read the scale before it changes
          if (lane == 0) *scale = s;
        }
      }
      const bool plain = finite && s > 1e-30f && s < 1e30f;
      const float r = __frcp_rn(s);
#pragma unroll
      for (int x = 0; x < NP; ++x) {
        const int row = x * SLOTS + slot;
        if (row < n) *reinterpret_cast<uint4*>(base + (size_t)(r0 + row) * c.Hkv * D) = e4m3_encode16(a0[x], a1[x], s, r, plain);
      }
    }
  }
}

// The rows of q, k and v by blocks 0 .. blocks - 1. NORM: the heads of q and k are normalised first (those with weights),
// keys also go to k_out, and where p.grow values are left to grow_values.
template <int D, bool NORM>
__device__ __forceinline__ void append_rows(const RopeAppendParams& p, int parts, int part_rows, int blocks) {
  constexpr int ROWS = NORM ? kNormRows : kRopeRows;
  constexpr int UN = D / 16;                       // units of a head
  constexpr int SLOTS = 32 / UN;                   // head rows a warp works on at a time
  const CacheView& c = p.c;
  const int lane = threadIdx.x & 31;
  const int u = lane % UN, slot = lane / UN;
  const int warps = blocks * (kRopeThreads / 32);
  const int warp = (int)blockIdx.x * (kRopeThreads / 32) + (int)(threadIdx.x >> 5);
  const int nq = p.q ? c.Hq : 0;
  const int rows = nq + (NORM && p.grow ? 1 : 2) * c.Hkv;   // q heads, then k heads, then v heads
  const bool rot = 16 * u < p.rope_dim;
  // the two 8-value vectors of unit u: the rotated units of half-split pairs take the vectors
  // below rope_dim / 8, and 2u of the first unit past them is rope_dim / 8
  const bool split = rot && p.rope_style == 0;
  const int v0 = split ? u : 2 * u, v1 = split ? u + p.rope_dim / 16 : 2 * u + 1;
  uint4 wq[2], wk[2];                              // this lane's weights; without weights ones, which change nothing
  if (NORM) {
    const uint4 one = make_uint4(0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u);
    wq[0] = p.q_weight ? __ldg(reinterpret_cast<const uint4*>(p.q_weight) + v0) : one;
    wq[1] = p.q_weight ? __ldg(reinterpret_cast<const uint4*>(p.q_weight) + v1) : one;
    wk[0] = p.k_weight ? __ldg(reinterpret_cast<const uint4*>(p.k_weight) + v0) : one;
    wk[1] = p.k_weight ? __ldg(reinterpret_cast<const uint4*>(p.k_weight) + v1) : one;
  }
  // Rows behind the last sequence are not touched: k_new and v_new may end there.
  const int end = min(c.total_q, __ldg(c.cu_q + c.batch));
  const long long items = (long long)end * parts;
  // a sequence of fewer than no new tokens has no row that would show it
  for (int b = (int)blockIdx.x * kRopeThreads + (int)threadIdx.x; b < c.batch; b += blocks * kRopeThreads)
    if (__ldg(c.cu_q + b + 1) < __ldg(c.cu_q + b)) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SEQ_LEN, b);
  for (long long it = warp; it < items; it += warps) {
    const int i = (int)(it / parts), part = (int)(it % parts);
    int b = -1, t = 0, page = -1, mode = 0;
    bool ok = false, page_ok = false;
    float cs[8], sn[8];
    const int x1 = min(rows, (part + 1) * part_rows);
    for (int x0 = part * part_rows; x0 < x1; x0 += SLOTS * ROWS) {
      uint4 a0[ROWS], a1[ROWS];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
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
      for (int r = 0; r < ROWS; ++r) {
        const int x = x0 + r * SLOTS + slot;
        float inv = 1.f;
        if (NORM) {                                // 1 / sqrt(mean of squares + eps), over the lanes of a row
          // (row after row: all rows' squares at once kept their values unpacked, 250 registers)
          inv = add_squares(a1[r], add_squares(a0[r], 0.f));
#pragma unroll
          for (int o = 1; o < UN; o <<= 1) inv += __shfl_xor_sync(0xffffffffu, inv, o);
          inv = rsqrtf(fmaf(inv, 1.f / D, p.eps));
        }
        if (x < x1 && x < nq + c.Hkv) {            // q or k: normalised, turned
          if (NORM) {
            const bool is_q = x < nq;
            const uint4 w0 = make_uint4(is_q ? wq[0].x : wk[0].x, is_q ? wq[0].y : wk[0].y, is_q ? wq[0].z : wk[0].z,
                                        is_q ? wq[0].w : wk[0].w);
            const uint4 w1 = make_uint4(is_q ? wq[1].x : wk[1].x, is_q ? wq[1].y : wk[1].y, is_q ? wq[1].z : wk[1].z,
                                        is_q ? wq[1].w : wk[1].w);
            scale_and_turn(a0[r], a1[r], (is_q ? p.q_weight : p.k_weight) ? inv : 1.f, w0, w1, rot, split, cs, sn);
          } else if (rot) {
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
          if (NORM && x >= nq && p.k_out) {
            uint4* dst = reinterpret_cast<uint4*>(p.k_out + ((size_t)i * c.Hkv + (x - nq)) * D);
            dst[v0] = a0[r];
            dst[v1] = a1[r];
          }
        }
        // v: in the form of its page. The block of a microscaled row is two units, in two lanes.
        const bool is_v = x >= nq + c.Hkv && x < x1;
        uint32_t mx2 = is_v ? max_mag16(a0[r], a1[r]) : 0u;
        mx2 = __vmaxu2(mx2, __shfl_xor_sync(0xffffffffu, mx2, 1));
        if (!is_v || !page_ok) continue;
        store_value<D>(c, page, mode, trow, x - nq - c.Hkv, u, a0[r], a1[r], mx2, b);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads)
rope_append_kernel(const RopeAppendParams p, int parts, int part_rows) {
  append_rows<D, false>(p, parts, part_rows, (int)gridDim.x);
}

// Blocks from row_blocks on write the values of pages whose scales grow, in chunks of `chunk` token rows.
template <int D>
__global__ void __launch_bounds__(kRopeThreads, kNormBlocks)
norm_append_kernel(const RopeAppendParams p, int parts, int part_rows, int row_blocks, int chunk) {
  if ((int)blockIdx.x < row_blocks) {
    append_rows<D, true>(p, parts, part_rows, row_blocks);
  } else {
    const int end = min(p.c.total_q, __ldg(p.c.cu_q + p.c.batch));
    grow_values<D>(p, ((int)blockIdx.x - row_blocks) * (kRopeThreads / 32) + (int)(threadIdx.x >> 5),
                   ((int)gridDim.x - row_blocks) * (kRopeThreads / 32), chunk, end);
  }
}

namespace {

struct RopeGrid {
  int parts, part_rows, grid;
};

// A warp takes a part of a token's rows: what its lanes hold in flight at once; or, while that leaves warps
// idle (16 a processor), two rows a lane (32 tokens: 8.3 -> 6.3 us). The parts of a token are of
// one size, so that the grid ends together.
RopeGrid rope_grid(const RopeAppendParams& p, int rows, int lane_rows, int num_sms) {
  const int slots = 512 / p.c.D;
  const int fit = (rows + slots * lane_rows - 1) / (slots * lane_rows), fine = (rows + 2 * slots - 1) / (2 * slots);
  const int want = p.c.total_q * (long long)fine <= (long long)num_sms * 16 ? fine : fit;
  RopeGrid g;
  g.part_rows = (rows + want * slots - 1) / (want * slots) * slots;
  g.parts = (rows + g.part_rows - 1) / g.part_rows;
  const long long warps = (long long)p.c.total_q * g.parts;
  const long long most = (long long)num_sms * 8;
  const long long grid = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  g.grid = (int)(grid > most ? most : grid);
  return g;
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams& p, int num_sms, cudaStream_t st) {
  if (p.c.total_q <= 0 || p.c.batch <= 0) return cudaSuccess;
  const RopeGrid g = rope_grid(p, (p.q ? p.c.Hq : 0) + 2 * p.c.Hkv, kRopeRows, num_sms);
  if (p.c.D == 128) rope_append_kernel<128><<<g.grid, kRopeThreads, 0, st>>>(p, g.parts, g.part_rows);
  else rope_append_kernel<64><<<g.grid, kRopeThreads, 0, st>>>(p, g.parts, g.part_rows);
  return cudaGetLastError();
}

cudaError_t launch_norm_append(const RopeAppendParams& p, int num_sms, cudaStream_t st) {
  if (p.c.total_q <= 0 || p.c.batch <= 0) return cudaSuccess;
  const RopeGrid g = rope_grid(p, (p.q ? p.c.Hq : 0) + (p.grow ? 1 : 2) * p.c.Hkv, kNormRows, num_sms);
  int chunk = 0, grow_blocks = 0;
  if (p.grow) {
    // a row an item while that leaves no warp a second item, so that pages are looked for in parallel; else 16
    // rows, of which one or two begin a page
    const long long most = (long long)num_sms * 8 * (kRopeThreads / 32);
    chunk = (long long)p.c.total_q * p.c.Hkv <= most ? 1 : kPage;
    long long warps = (long long)((p.c.total_q + chunk - 1) / chunk) * p.c.Hkv;
    if (warps > most) warps = most;
    grow_blocks = (int)((warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32));
  }
  const int grid = g.grid + grow_blocks;
  if (p.c.D == 128) norm_append_kernel<128><<<grid, kRopeThreads, 0, st>>>(p, g.parts, g.part_rows, g.grid, chunk);
  else norm_append_kernel<64><<<grid, kRopeThreads, 0, st>>>(p, g.parts, g.part_rows, g.grid, chunk);
  return cudaGetLastError();
}

}  // namespace ekv
