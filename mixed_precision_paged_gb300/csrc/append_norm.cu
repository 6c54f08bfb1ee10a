// append_norm.cu -- the rotary cache writer for models that normalise queries and keys per head, and the values of
// E4M3 pages whose scales the call makes.
//
//   x^_d = x_d / sqrt(mean x^2 + eps) * w_d, then the rotation of append_rope.cu, in fp32 and rounded once.
// Every value is read once and written once (keys twice with k_out): HBM-bound, the floor is those bytes.
// A norm needs a whole row before its first result. With the rows in registers, as append_rope.cu has them, loads
// stop while a warp computes (65,536 tokens of 32 + 2 x 8 heads of 128: 305 us, however rows and blocks are chosen). So they come
// by bulk copies into a ring of a warp's own in shared memory, a token's part (its rows of q, k and v and its angles) a stage,
// issued as many tokens ahead as there are stages. The sums and products are packed fp32 (two values an instruction).
// A decode step is a chain of loads that wait for one another (sequence, lengths, page and mode, then the copies): 32 tokens 10.1 us on the device,
// caches cold, on 8 blocks, where append_rope.cu, which loads its rows first and splits tokens finer, takes 8.6; 256 with
// growing scales 13.6. With D 128 and growing scales 128 registers do not hold everything (100 bytes of spills stored, 60 loaded).
#include "rope.cuh"

namespace ekv {

namespace {

// Two fp32 values as one operand of the packed instructions.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}

// 8 fp16 values as four pairs, and back.
__device__ __forceinline__ void unpack8(const uint4& v, uint64_t (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = word_values(w[i]);
    x[i] = pair(f.x, f.y);
  }
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = halves(x[i]);
    w[i] = word_of(f.x, f.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A head row of the norm: lo and hi (16 values of a lane) become their multiples by 1 / sqrt(mean square + eps) and the
// weights (fp32 pairs), turned where `rot`: with `split` pairs (lo[j], hi[j]) by angle j, else neighbours,
// lo's by angles 0 .. 3 and hi's by 4 .. 7 (c and s: the angles' cosines and sines, two a pair). fp32, two values
// an instruction, up to the last step. The UN lanes of the row share its sum; every lane of the warp takes part. Without
// `norm` the row is turned alone.
template <int UN>
__device__ __forceinline__ void norm_and_turn(uint4& lo, uint4& hi, bool norm, float eps, const uint64_t (&wlo)[4],
                                              const uint64_t (&whi)[4], bool rot, bool split, const uint64_t (&c)[4], const uint64_t (&s)[4]) {
  uint64_t x[4], y[4], q = 0;
  unpack8(lo, x);
  unpack8(hi, y);
#pragma unroll
  for (int i = 0; i < 4; ++i) q = fma2(y[i], y[i], fma2(x[i], x[i], q));
  const float2 qs = halves(q);
  float sum = qs.x + qs.y;
#pragma unroll
  for (int o = 1; o < UN; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = norm ? rsqrtf(fmaf(sum, 1.f / (16 * UN), eps)) : 1.f;
  const uint64_t inv2 = pair(inv, inv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = mul2(mul2(x[i], inv2), wlo[i]);
    y[i] = mul2(mul2(y[i], inv2), whi[i]);
  }
  if (rot) {
    if (split) {
      const uint64_t minus = pair(-1.f, -1.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t u = x[i];
        x[i] = fma2(mul2(y[i], minus), s[i], mul2(u, c[i]));
        y[i] = fma2(u, s[i], mul2(y[i], c[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {                  // (angle i is half i % 2 of pair i / 2)
        const float2 u = halves(x[i]), v = halves(y[i]);
        const float2 c0 = halves(c[i / 2]), s0 = halves(s[i / 2]), c1 = halves(c[2 + i / 2]), s1 = halves(s[2 + i / 2]);
        const float ca = i & 1 ? c0.y : c0.x, sa = i & 1 ? s0.y : s0.x, cb = i & 1 ? c1.y : c1.x, sb = i & 1 ? s1.y : s1.x;
        x[i] = fma2(pair(u.y, u.x), pair(-sa, sa), mul2(x[i], pair(ca, ca)));
        y[i] = fma2(pair(v.y, v.x), pair(-sb, sb), mul2(y[i], pair(cb, cb)));
      }
    }
  }
  lo = pack8(x);
  hi = pack8(y);
}

// The 8 fp32 values of vector v of a head's weights, as pairs: [2][D / 8] quarter vectors in shared memory, so that
// eight lanes read 128 bytes without a conflict.
template <int D>
__device__ __forceinline__ void load_weights(const float4* w, int v, uint64_t (&x)[4]) {
  const float4 a = w[v], b = w[D / 8 + v];
  x[0] = pair(a.x, a.y);
  x[1] = pair(a.z, a.w);
  x[2] = pair(b.x, b.y);
  x[3] = pair(b.z, b.w);
}
// Fills the weights of q and, behind them, of k; without weights ones, which change nothing. All threads.
template <int D>
__device__ __forceinline__ void fill_weights(const RopeAppendParams& p, float4* weights) {
  for (int x = threadIdx.x; x < 2 * D; x += blockDim.x) {
    const __half* w = x < D ? p.q_weight : p.k_weight;
    const int d = x % D;
    reinterpret_cast<float*>(weights)[x - d + ((d >> 2) & 1) * (D / 2) + (d >> 3) * 4 + (d & 3)] = w ? __half2float(w[d]) : 1.f;
  }
}

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

// 4 codes times f, rounded to codes again.
__device__ __forceinline__ uint32_t e4m3_rescale4(uint32_t codes, float f) {
  const float2 a = e4m3x2_to_float2((uint16_t)codes), b = e4m3x2_to_float2((uint16_t)(codes >> 16));
  return (uint32_t)float2_to_e4m3x2(a.x * f, a.y * f) | ((uint32_t)float2_to_e4m3x2(b.x * f, b.y * f) << 16);
}

// Warps `warp`, `warp + warps`, ... of the items (chunk of token rows, `heads` KV heads). An item takes the pages whose first
// new row lies in its chunk: a page's rows may go on behind it. A head's rows are loaded while the one before is worked on.
template <int D>
__device__ __forceinline__ void grow_values(const RopeAppendParams& p, int warp, int warps, int chunk, int heads, int start, int end) {
  constexpr int UN = D / 16, SLOTS = 32 / UN, NP = kPage / SLOTS;
  const CacheView& c = p.c;
  const int lane = threadIdx.x & 31, u = lane % UN, slot = lane / UN;
  const int groups = c.Hkv / heads;
  const long long items = (long long)((end + chunk - 1) / chunk) * groups;
  for (long long it = warp; it < items; it += warps) {
    const int h0 = (int)(it % groups) * heads, i0 = (int)(it / groups) * chunk, i = i0 + lane;
    // a lane's row of the chunk: where it goes, and how many rows its page takes from it on
    int t = 0, rows = 0, page = 0, mode = 0, b = 0;
    if (lane < chunk && i < end && i >= start) {
      b = lane_find_sequence(c.cu_q, c.batch, i, start, end);
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
      uint4 a0[NP], a1[NP], n0[NP], n1[NP];
      auto load = [&](int h, uint4 (&x0)[NP], uint4 (&x1)[NP]) {
#pragma unroll
        for (int x = 0; x < NP; ++x) {
          const int row = x * SLOTS + slot;              // of the rows from r0 on
          x0[x] = x1[x] = make_uint4(0u, 0u, 0u, 0u);
          if (row < n) {
            const uint4* v = reinterpret_cast<const uint4*>(p.v_new + (size_t)(i0 + src + row) * p.v_stride + h * D) + 2 * u;
            x0[x] = __ldg(v);
            x1[x] = __ldg(v + 1);
          }
        }
      };
      load(h0, n0, n1);
      for (int h = h0; h < h0 + heads; ++h) {
#pragma unroll
        for (int x = 0; x < NP; ++x) {
          a0[x] = n0[x];
          a1[x] = n1[x];
        }
        if (h + 1 < h0 + heads) load(h + 1, n0, n1);
        if (md != EKV_MODE_COMPACT_E4M3) {
#pragma unroll
          for (int x = 0; x < NP; ++x) {
            uint32_t mx2 = max_mag16(a0[x], a1[x]);
            mx2 = __vmaxu2(mx2, __shfl_xor_sync(0xffffffffu, mx2, 1));
            const int row = x * SLOTS + slot;
            if (row < n) store_value<D, true>(c, pg, md, r0 + row, h, u, a0[x], a1[x], mx2, sb);
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
        const bool plain = finite && far_from_ends(s);
        const float r = __frcp_rn(s);
#pragma unroll
        for (int x = 0; x < NP; ++x) {
          const int row = x * SLOTS + slot;
          if (row < n) *reinterpret_cast<uint4*>(base + (size_t)(r0 + row) * c.Hkv * D) = e4m3_encode16<true>(a0[x], a1[x], s, r, plain);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ the kernel
constexpr int kNormWarps = 8, kNormThreads = 32 * kNormWarps;
constexpr int kNormStages = 4;                     // of a warp, at most
constexpr int kNormSmem = 108 * 1024;              // two blocks a processor

// Blocks of the growing scales, as far as there are items for them: a quarter of the rows' blocks, and one round (two a
// processor) at least. Values are 12% of the call's bytes with 32/8 heads and packed keys, 27% with as many query heads as KV
// heads, 43% without queries; the share hardly matters to any of them (all / a half / a quarter / an eighth of the rows'
// blocks: 24 prompts of 700 to 4,000 tokens 242 / 242 / 244 / 242 us, with 8/8 heads 142 / 140 / 140 / 140, without queries
// 103 / 102 / 103 / 102).
constexpr int kGrowShare = 4;
struct NormShape {
  int nst, stage;                                  // stages of a warp, bytes of one
  int parts, part_rows;                            // of a token, a warp each: so many head rows
  int row_blocks, grow_blocks;                     // blocks of the rows, and of values whose scales grow
  int chunk, heads;                                // of the latter: token rows and KV heads of an item
};

// Head rows [xa, xb) of a kind (q or k) of one token, in shared memory at `tok`: normalised, turned and written to
// dst + x D, and to also + x D, where these are not null.
template <int D>
__device__ __forceinline__ void put_rows(const uint8_t* tok, int xa, int xb, bool norm, float eps, const float4* weights, int v0, int v1,
                                         bool rot, bool split, const uint64_t (&cs)[4], const uint64_t (&sn)[4], __half* dst,
                                         __half* also) {
  constexpr int UN = D / 16, SLOTS = 32 / UN;
  if (xa >= xb) return;
  const int slot = (threadIdx.x & 31) / UN;
  uint64_t wlo[4], whi[4];
  load_weights<D>(weights, v0, wlo);
  load_weights<D>(weights, v1, whi);
#pragma unroll 2
  for (int x0 = xa; x0 < xb; x0 += SLOTS) {
    const int x = x0 + slot;
    const uint4* row = reinterpret_cast<const uint4*>(tok + min(x, xb - 1) * (D * 2));
    uint4 lo = row[v0], hi = row[v1];
    norm_and_turn<UN>(lo, hi, norm, eps, wlo, whi, rot, split, cs, sn);
    if (x >= xb) continue;
    if (dst) {
      reinterpret_cast<uint4*>(dst + x * D)[v0] = lo;
      reinterpret_cast<uint4*>(dst + x * D)[v1] = hi;
    }
    if (also) {
      reinterpret_cast<uint4*>(also + x * D)[v0] = lo;
      reinterpret_cast<uint4*>(also + x * D)[v1] = hi;
    }
  }
}

template <int D, bool GROW>
__global__ void __launch_bounds__(kNormThreads, 2)
norm_append_kernel(const RopeAppendParams p, const NormShape sh) {
  constexpr int UN = D / 16, SLOTS = 32 / UN;
  extern __shared__ __align__(128) uint8_t ring[];         // [warps][nst][stage]
  __shared__ uint64_t full[kNormWarps * kNormStages];
  __shared__ float4 weights[D / 2];
  const CacheView& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Values whose scales grow have blocks of their own, spread among those of the rows: their longer way (a page's rows, their
  // maximum, the codes) runs beside the others' copies.
  int block = (int)blockIdx.x;
  const int start = __ldg(c.cu_q), end = min(c.total_q, __ldg(c.cu_q + c.batch));
  if (GROW) {
    const int before = block * sh.grow_blocks / (int)gridDim.x;          // blocks of values before this one
    if ((block + 1) * sh.grow_blocks / (int)gridDim.x > before) {
      grow_values<D>(p, before * kNormWarps + warp, sh.grow_blocks * kNormWarps, sh.chunk, sh.heads, start, end);
      return;
    }
    block -= before;
  }
  fill_weights<D>(p, weights);
  if ((int)threadIdx.x < kNormWarps * sh.nst) mbar_init(&full[threadIdx.x], 1);
  if (threadIdx.x == 0) fence_barrier_init();
  __syncthreads();
  // a sequence of fewer than no new tokens has no row that would show it
  for (int b = block * kNormThreads + (int)threadIdx.x; b < c.batch; b += sh.row_blocks * kNormThreads)
    if (__ldg(c.cu_q + b + 1) < __ldg(c.cu_q + b)) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SEQ_LEN, b);

  const int u = lane % UN, slot = lane / UN;
  const int nq = p.q ? c.Hq : 0, nk = nq + c.Hkv, rows = GROW ? nk : nk + c.Hkv;
  const bool rot = 16 * u < p.rope_dim, split = rot && p.rope_style == 0;
  const int v0 = split ? u : 2 * u, v1 = split ? u + p.rope_dim / 16 : 2 * u + 1;
  const int angles = sh.part_rows * D * 2;                 // where a stage's angles lie
  uint8_t* base = ring + (size_t)warp * sh.nst * sh.stage;
  uint64_t* bars = full + warp * sh.nst;
  // this warp's part of a token, [xa, xb), and its tokens first, first + stride, ...: neighbours go to neighbouring processors
  const int id = warp * sh.row_blocks + block, stride = kNormWarps * sh.row_blocks / sh.parts;
  const int xa = id % sh.parts * sh.part_rows, xb = min(rows, xa + sh.part_rows), first = id / sh.parts;
  const int n = first < min(end, stride) ? (end - 1 - first) / stride + 1 : 0;
  // where 32 tokens go, a token a lane: position, page (-1: it failed its checks), mode and sequence; t < 0: nothing to write
  auto look_up = [&](int k, int& t, int& page, int& mode, int& b) {
    t = page = -1;
    mode = b = 0;
    if (k + lane >= n) return;
    const int i = first + (k + lane) * stride;
    if (i < start) return;
    b = lane_find_sequence(c.cu_q, c.batch, i, start, end);
    if (b >= c.batch) return;
    const int q0 = __ldg(c.cu_q + b), q1 = __ldg(c.cu_q + b + 1), len = __ldg(c.seq_lens + b);
    const int at = len - (q1 - i);
    if (q0 < 0 || i < q0 || q1 - q0 > len || (long long)len > (long long)c.bt_stride * kPage || (p.rope_dim > 0 && at >= p.rope_len)) {
      report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SEQ_LEN, b);
      return;
    }
    t = at;
    page = __ldg(c.block_table + (size_t)b * c.bt_stride + t / kPage);
    if (page < 0 || page >= c.num_pages) {
      report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_PAGE_ID, b);
      page = -1;
      return;
    }
    mode = c.page_mode ? (int)__ldg(c.page_mode + page) : c.uniform_mode;
    if (mode > EKV_MODE_MICRO_FP4) {
      report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_PAGE_MODE, b);
      page = -1;
    }
  };
  int t0, page0, mode0, b0, t1 = -1, page1 = -1, mode1 = 0, b1 = 0;   // of this batch of 32 and of the next
  look_up(0, t0, page0, mode0, b0);
  // the copies of token k, whose batch has the positions tk: none for a token that is not written
  auto issue = [&](int k, int tk) {
    const int t = __shfl_sync(0xffffffffu, tk, k & 31);
    if (t < 0 || lane != 0) return;
    const long long i = first + k * stride;
    uint8_t* dst = base + (size_t)(k % sh.nst) * sh.stage;
    uint64_t* bar = bars + k % sh.nst;
    mbar_arrive_expect_tx(bar, (xb - xa) * D * 2 + p.rope_dim * 4);
    auto copy = [&](const __half* src, long long row_stride, int a, int b) {   // rows [a, b) of a kind that begins at row a0
      const int lo = max(a, xa), hi = min(b, xb);
      if (lo < hi) bulk_load(dst + (lo - xa) * D * 2, src + i * row_stride + (lo - a) * D, (hi - lo) * D * 2, bar);
    };
    copy(p.q, p.q_stride, 0, nq);
    copy(p.k_new, p.k_stride, nq, nk);
    if (!GROW) copy(p.v_new, p.v_stride, nk, rows);
    if (p.rope_dim > 0) bulk_load(dst + angles, p.rope + (size_t)t * p.rope_dim, p.rope_dim * 4, bar);
  };
#ifdef EKV_TEST_WAIT_TIMEOUT
  if (p.inject_timeout && block == 0 && warp == 0 && lane == 0) mbar_expect_tx(bars, 16);   // (no copy delivers them)
  __syncwarp();
#endif
  for (int k = 0; k < min(sh.nst, n); ++k) issue(k, t0);
  uint32_t phases = 0;                                     // bit per stage: the parity of its next phase
  int k = 0;
  bool ok = true;
  for (; k < n; ++k) {
    const int src = k & 31, st = k % sh.nst;
    const int t = __shfl_sync(0xffffffffu, t0, src), page = __shfl_sync(0xffffffffu, page0, src);
    const int mode = __shfl_sync(0xffffffffu, mode0, src), b = __shfl_sync(0xffffffffu, b0, src);
    if (t >= 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(bars + st, (phases >> st) & 1u));
      if (!ok) break;
      phases ^= 1u << st;
      const int i = first + k * stride;
      const uint8_t* tok = base + (size_t)st * sh.stage - xa * (D * 2);   // (row 0 of the token would lie here)
      uint64_t cs[4], sn[4];
      if (rot) {
        const uint64_t* a = reinterpret_cast<const uint64_t*>(base + (size_t)st * sh.stage + angles) + 4 * u;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          cs[x] = a[x];
          sn[x] = a[p.rope_dim / 4 + x];
        }
      }
      put_rows<D>(tok, xa, min(xb, nq), p.q_weight != nullptr, p.eps, weights, v0, v1, rot, split, cs, sn,
                  p.q_out + (size_t)i * c.Hq * D, nullptr);
      put_rows<D>(tok + nq * (D * 2), max(xa, nq) - nq, min(xb, nk) - nq, p.k_weight != nullptr, p.eps, weights + D / 4, v0, v1, rot, split,
                  cs, sn, page >= 0 ? const_cast<__half*>(c.k_pages) + ((size_t)page * kPage + t % kPage) * c.Hkv * D : nullptr,
                  p.k_out ? p.k_out + (size_t)i * c.Hkv * D : nullptr);
      if (!GROW) {
#pragma unroll 2
        for (int x0 = max(xa, nk); x0 < xb; x0 += SLOTS) {
          const int x = x0 + slot;
          const uint4* row = reinterpret_cast<const uint4*>(tok + min(x, xb - 1) * (D * 2));
          const uint4 lo = row[2 * u], hi = row[2 * u + 1];
          uint32_t mx2 = max_mag16(lo, hi);
          mx2 = __vmaxu2(mx2, __shfl_xor_sync(0xffffffffu, mx2, 1));
          if (x < xb && page >= 0) store_value<D, true>(c, page, mode, t % kPage, x - nk, u, lo, hi, mx2, b);
        }
      }
      fence_reads_before_refill();
      __syncwarp();
    }
    const int next = k + sh.nst;
    if ((next & 31) == 0 && next < n) look_up(next, t1, page1, mode1, b1);
    if (next < n) issue(next, (next >> 5) == (k >> 5) ? t0 : t1);
    if (src == 31) {
      t0 = t1;
      page0 = page1;
      mode0 = mode1;
      b0 = b1;
    }
  }
  if (!ok) {
    // the copies in flight land before the CTA can exit (a stage's next phase, where one was begun)
    if (lane == 0) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_TIMEOUT, -1);
    for (int x = k; x < min(k + sh.nst, n); ++x) {
      const int t = __shfl_sync(0xffffffffu, (x >> 5) == (k >> 5) ? t0 : t1, x & 31);
      if (t >= 0) mbar_wait(bars + x % sh.nst, (phases >> (x % sh.nst)) & 1u);
    }
  }
}

template <int D, bool GROW>
cudaError_t launch(const RopeAppendParams& p, const NormShape& sh, cudaStream_t st) {
  const cudaError_t e = set_smem_attr(reinterpret_cast<const void*>(norm_append_kernel<D, GROW>), kNormSmem);
  if (e != cudaSuccess) return e;
  norm_append_kernel<D, GROW><<<sh.row_blocks + sh.grow_blocks, kNormThreads, kNormWarps * sh.nst * sh.stage, st>>>(p, sh);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_append(const RopeAppendParams& p, int num_sms, cudaStream_t st) {
  if (p.c.total_q <= 0 || p.c.batch <= 0) return cudaSuccess;
  const int rows = (p.q ? p.c.Hq : 0) + (p.grow ? 1 : 2) * p.c.Hkv, slots = 512 / p.c.D;   // slots: rows of a pass
  NormShape sh;
  // As many parts of a token as let every warp have two stages in shared memory (a ring of whole tokens for half
  // the warps leaves these to set the pace).
  for (sh.parts = 1;; ++sh.parts) {
    sh.part_rows = ((rows + sh.parts - 1) / sh.parts + slots - 1) / slots * slots;
    sh.stage = (sh.part_rows * p.c.D * 2 + p.rope_dim * 4 + 127) & ~127;
    sh.nst = kNormSmem / (kNormWarps * sh.stage);
    if (sh.nst >= 2) break;
  }
  sh.parts = (rows + sh.part_rows - 1) / sh.part_rows;
  if (sh.nst > kNormStages) sh.nst = kNormStages;
  // Two blocks a processor, and up to eight rounds of them where each warp still has eight tokens' parts: processors differ in
  // speed (65,536 tokens, 1 / 2 / 4 / 6 / 8 rounds: 303 / 299 / 279 / 266 / 266 us; 18,285 tokens, 1 / 2 / 4: 70 / 76 / 82).
  const long long items = (long long)p.c.total_q * sh.parts, round = (long long)num_sms * 2;
  auto blocks_for = [&](long long n, long long each) {     // of n items, `each` at least a warp
    const long long most = round * 8, least = (n + kNormWarps - 1) / kNormWarps;
    const long long rounds = n / (round * kNormWarps * each);
    return (int)(least < round ? least : rounds < 1 ? round : rounds * round < most ? rounds * round : most);
  };
  sh.row_blocks = blocks_for(items, 8);
  if (sh.row_blocks * kNormWarps < sh.parts) sh.row_blocks = (sh.parts + kNormWarps - 1) / kNormWarps;
  sh.grow_blocks = sh.chunk = sh.heads = 0;
  if (p.grow) {
    // few values: a row and head an item, so that pages are looked for in parallel; else 16 rows, of which one or two begin
    // a page, and as many heads as leave every warp an item
    const long long warps = round * kNormWarps;
    sh.chunk = (long long)p.c.total_q * p.c.Hkv <= 2 * warps ? 1 : kPage;
    const long long chunks = (p.c.total_q + sh.chunk - 1) / sh.chunk;
    sh.heads = 1;
    while (sh.heads < p.c.Hkv && chunks * p.c.Hkv / (2 * sh.heads) >= warps) sh.heads *= 2;
    const long long n = chunks * (p.c.Hkv / sh.heads);
    const long long least = (n + kNormWarps - 1) / kNormWarps;
    const long long share = sh.row_blocks / kGrowShare > round ? sh.row_blocks / kGrowShare : round;
    sh.grow_blocks = (int)(least < share ? least : share);
  }
  if (p.c.D == 128) return p.grow ? launch<128, true>(p, sh, st) : launch<128, false>(p, sh, st);
  return p.grow ? launch<64, true>(p, sh, st) : launch<64, false>(p, sh, st);
}

}  // namespace ekv
