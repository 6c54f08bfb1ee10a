// extend_split.cuh -- attention of few new tokens per sequence over the paged cache (decode
// steps, draft verification): split over the cache's length, joined in the same kernel.
//
// With few query rows the cache is read once and everything else is small, so the kernel is a
// stream: 2 B a key value and 2, 1 or 17/32 B a value of V at HBM rate. The pages that any
// sequence has to read form one sequence of positions, cut into one contiguous range per
// warp stream as in the one-token decode (pipeline.cuh): warp w of CTA c works on KV head
// h = w mod H_kv and range c * NG + w / H_kv, with its own ring of TMA-filled slots, so no warp
// waits for another. What differs here:
//   * rows: the G query heads of all n_b new tokens are the N columns of the products, row
//     rho = r * G + g, in NT tiles of 8 (up to 32 rows; tiles past n_b * G are left out at run time);
//   * causal and window limits, applied only on pages that some row sees in part;
//   * four page forms. An E4M3 page's scale joins the exponent, p' = 2^(score + log2 scale - m)
//     with the running maximum m over the scaled scores, and the sum takes p' / scale: so codes
//     enter the product exactly as they are, and p' is rounded to fp16 once relative to the largest
//     contribution, whatever the scales are. A microscaled value is code * 2^k, exact in fp16.
//   * the rows d of the V^T fragments: m-tiles 2j and 2j+1 hold d = 32j + 4 r8 + {0, 1} and {2, 3}
//     in their rows r8 and r8 + 8, so a lane's values of one token are 4 neighbours in every form:
//     8 bytes of FP16, 4 of E4M3 or BASE, one 16-bit word of codes.
//
// Joining: a sequence inside one range is finished by its warp. Otherwise each range leaves a
// record (m, l, acc) per row, two slots a range (its first and its last segment), and the warp
// that takes the last ticket of a group merges it: up to kJoin records directly, and beyond that
// in two levels, groups of kJoin first, each merged by its own last warp, then the groups, so that
// a single long sequence over all SMs does not wait for one warp reading every record.
#pragma once

#include "extend.cuh"
#include "micro.cuh"
#include "pipeline.cuh"

namespace ekv {

enum ExtVMode { kXFP16 = 0, kXE4M3 = 1, kXMicro = 2, kXMixed = 3 };

constexpr int kXWarps = 8;
constexpr int kXThreads = 32 * kXWarps;
constexpr int kXRows = 32;                         // query rows of a KV head (n_b * G) at most
constexpr int kJoin = 16;                          // records merged by one warp at a time

struct ExtSplitParams {
  ExtendParams e;
  float* part_acc;        // [2 * ranges][Hkv][kXRows][D]
  float2* part_ml;        // [2 * ranges][Hkv][kXRows]  (m in log2 units, l)
  int* ticket;            // [max_batch][8] joins of whole sequences, then [2 * ranges][Hkv] of groups
  int* group_ticket;
  int NG;                 // page groups: 8 / Hkv
  int nsl;                // ring slots per warp
  int v_off, bar_off, cu_off, q_off;
};

template <int D, int VM>
struct ExtSlot {
  static constexpr int kK = kPage * D * 2;
  static constexpr int kV = VM == kXMicro ? micro_head_bytes(D) : VM == kXE4M3 ? kPage * D : kPage * D * 2;
};

namespace xs {

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t fp4_pair(uint32_t byte, uint32_t scale) {
  const __half2_raw r = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(byte & 0xffu), __NV_E2M1);
  return bits(__hmul2(*reinterpret_cast<const __half2*>(&r), *reinterpret_cast<const __half2*>(&scale)));
}

// One sequence's part in the plan.
struct Seq {
  int L, n, q0;            // tokens, new tokens, first row of q
  int p0;                  // first page that any of its queries sees
};

// Reads sequence b; false (nothing to attend) when it is empty or fails its checks.
__device__ __forceinline__ bool load_seq(const ExtendParams& e, int b, Seq& s) {
  const CacheView& c = e.c;
  s.q0 = __ldg(c.cu_q + b);
  s.n = __ldg(c.cu_q + b + 1) - s.q0;
  s.L = __ldg(c.seq_lens + b);
  s.p0 = s.L - s.n < e.window ? 0 : (s.L - s.n - e.window + 1) / kPage;
  return s.n != 0;
}
__device__ __forceinline__ bool seq_ok(const ExtendParams& e, const Seq& s) {
  return s.n > 0 && s.n <= s.L && s.n <= e.max_q && s.q0 >= 0 && (long long)s.q0 + s.n <= e.c.total_q &&
         (long long)s.L <= (long long)e.c.bt_stride * kPage;
}

// Zero rows and -inf lse of sequence b's new tokens.
__device__ __forceinline__ void zero_rows(const ExtendParams& e, const Seq& s) {
  const CacheView& c = e.c;
  const int r0 = max(s.q0, 0), r1 = (int)min((long long)s.q0 + s.n, (long long)c.total_q);
  const long long n = (long long)max(0, r1 - r0) * c.Hq;
  for (long long i = threadIdx.x; i < n * c.D; i += blockDim.x) e.out[(long long)r0 * c.Hq * c.D + i] = __float2half(0.f);
  if (e.lse)
    for (long long i = threadIdx.x; i < n; i += blockDim.x) e.lse[(long long)r0 * c.Hq + i] = -INFINITY;
}

// Block-wide prefix sum of the pages each sequence has to read into cu[0 .. batch]; returns their total.
// CTA 0 reports the sequences that fail their checks and zeroes their rows.
__device__ __forceinline__ int plan(const ExtendParams& e, int* cu, int* warp_tot) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, batch = e.c.batch;
  if (tid == 0) cu[0] = 0;
  int carry = 0;
  for (int base = 0; base < batch; base += kXThreads) {
    const int b = base + tid;
    int np = 0;
    bool fails = false;
    if (b < batch) {
      Seq s;
      if (load_seq(e, b, s)) {
        fails = !seq_ok(e, s);
        if (!fails) np = (s.L + kPage - 1) / kPage - s.p0;
      }
      if (fails && blockIdx.x == 0) report_error(e.c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SEQ_LEN, b);
    }
    int incl = np;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_tot[warp] = incl;
    const int any_fails = __syncthreads_or(fails);
    int woff = 0, chunk = 0;
#pragma unroll
    for (int w = 0; w < kXWarps; ++w) {
      const int t = warp_tot[w];
      woff += (w < warp) ? t : 0;
      chunk += t;
    }
    if (b < batch) cu[b + 1] = carry + woff + incl;
    carry += chunk;
    __syncthreads();
    if (any_fails && blockIdx.x == 0) {
      for (int x = base; x < min(batch, base + kXThreads); ++x) {
        Seq s;
        if (load_seq(e, x, s) && !seq_ok(e, s)) zero_rows(e, s);
      }
    }
  }
  return carry;
}

// ------------------------------------------------------------------ page metadata
// One page per lane for 32 consecutive pages of the warp's range.
struct Meta {
  int page, lp, b, flags;
  float lsc, ivs;          // log2 of an E4M3 page's scale, and its reciprocal
};
constexpr int kSkip = 1, kE4 = 2, kBs = 4, kMx = 8;

__device__ __forceinline__ void meta_ids(const ExtendParams& e, const int* cu, int start, int n_my, int k, Meta& m) {
  m.page = m.lp = 0;
  m.flags = kSkip;
  m.b = -1;
  m.lsc = 0.f;
  m.ivs = 1.f;
  if (k < n_my) {
    const int j = start + k;
    const int b = upper_bound_i(cu, e.c.batch + 1, j) - 1;
    int p0 = 0;
    if (e.window != 0x7fffffff) {
      Seq s;
      load_seq(e, b, s);
      p0 = s.p0;
    }
    m.b = b;
    m.lp = p0 + j - cu[b];
    m.page = __ldg(e.c.block_table + (size_t)b * e.c.bt_stride + m.lp);
    m.flags = 0;
  }
}

template <int VM>
__device__ __forceinline__ void meta_mode(const ExtendParams& e, int h, Meta& m) {
  if (m.b < 0) return;
  const CacheView& c = e.c;
  int detail = m.page < 0 || m.page >= c.num_pages ? EKV_DETAIL_PAGE_ID : EKV_DETAIL_NONE;
  if (!detail && VM != kXFP16 && VM != kXMicro) {
    int mode = EKV_MODE_COMPACT_E4M3;
    if (VM == kXMixed) mode = c.page_mode ? (int)__ldg(c.page_mode + m.page) : c.uniform_mode;
    if (mode > EKV_MODE_MICRO_FP4) {
      detail = EKV_DETAIL_PAGE_MODE;
    } else if (mode == EKV_MODE_COMPACT_E4M3) {
      const float s = !c.v_scales ? 0.f
                                  : __ldg(c.v_scales + (c.scale_mode == EKV_SCALE_PER_TENSOR ? 0 : (size_t)m.page * c.Hkv + h));
      if (!scale_ok(s)) detail = EKV_DETAIL_SCALE;
      m.flags = kE4;
      m.lsc = log2f(s);
      m.ivs = 1.f / s;
    } else {
      m.flags = mode == EKV_MODE_BASE ? kBs : mode == EKV_MODE_MICRO_FP4 ? kMx : 0;
    }
  }
  if (detail) {
    report_error(c.err, EKV_ERR_DEVICE_CHECK, detail, m.b);
    m.flags = kSkip;
  }
}

struct Ring {
  uint8_t* k;
  uint8_t* v;
  uint64_t* full;
  int nsl;
};

// Lane 0 fills slot s with the slice of (page, head h).
template <int D, int VM>
__device__ __forceinline__ void fill(const ExtendParams& e, const Ring& ring, int s, int h, int page, int flags,
                                     const CUtensorMap* tmK, const CUtensorMap* tmV8, const CUtensorMap* tmV16) {
  if ((threadIdx.x & 31) != 0) return;
  using S = ExtSlot<D, VM>;
  uint64_t* bar = &ring.full[s];
  if (flags & kSkip) {
    mbar_arrive(bar);
    return;
  }
  uint8_t* dk = ring.k + (size_t)s * S::kK;
  uint8_t* dv = ring.v + (size_t)s * S::kV;
  const bool micro = VM == kXMicro || (VM == kXMixed && (flags & kMx));
  const bool bytes = VM == kXE4M3 || (VM == kXMixed && (flags & (kE4 | kBs)));
  const int vb = micro ? micro_head_bytes(D) : bytes ? kPage * D : kPage * D * 2;
  mbar_arrive_expect_tx(bar, S::kK + vb);
  tma_load_5d(dk, tmK, 0, 0, 0, h, page, bar);
  if (micro)
    bulk_load(dv, e.c.v_pages + (size_t)page * e.c.v_page_stride + h * micro_head_bytes(D), vb, bar);
  else if (bytes)
    tma_load_4d(dv, tmV8, 0, h, 0, page, bar);
  else
    tma_load_5d(dv, tmV16, 0, 0, 0, h, page, bar);
}

// ---------------------------------------------------------------------- joining
// Merges `nrec` records of KV head h, rows < n_b * G: record 0 at `first`, record i at rec0 + i * step;
// to the record `dst`, or to the output when dst < 0.
//   M = max m_i,  L = sum l_i 2^(m_i - M),  out = sum acc_i 2^(m_i - M) / L,  lse = (M + log2 L) ln 2.
// One warp. Several rows at a time, as many as their records fit `buf` (its ring): the acc rows by 16-byte
// asynchronous copies and the (m, l) pairs by plain loads, all under way before any is used, so a
// wave costs one round trip to L2. A row of more records than fit is taken in pieces with a running maximum.
template <int D>
__device__ void join(const ExtSplitParams& p, int h, const Seq& s, int first, int rec0, int step, int nrec, int dst,
                     uint8_t* buf, int buf_bytes) {
  const ExtendParams& e = p.e;
  const int lane = threadIdx.x & 31;
  const int R = s.n * e.G;
  constexpr int kRowB = D * 4;
  constexpr int C = D / 32;                        // columns per lane
  const int cap = min(buf_bytes / (kRowB + 8), 64);
  float2* mls = reinterpret_cast<float2*>(buf + cap * kRowB);
  const int rows = max(1, cap / nrec);             // rows of a wave
  for (int row0 = 0; row0 < R; row0 += rows) {
    const int nr = min(rows, R - row0);
    float acc[C], M = -INFINITY, L = 0.f;
    bool bad = false;
    for (int i0 = 0; i0 < nrec; i0 += cap) {       // (one piece, except for a row of many records)
      const int ni = min(cap, nrec - i0), np = nr * ni;
      auto at = [&](int q) {
        const int i = i0 + q % ni;
        return ((size_t)(i == 0 ? first : rec0 + i * step) * e.c.Hkv + h) * kXRows + row0 + q / ni;
      };
      float2 v[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) v[y] = lane + 32 * y < np ? __ldcg(p.part_ml + at(lane + 32 * y)) : make_float2(0.f, 0.f);
      for (int o = lane; o < np * (kRowB / 16); o += 32)
        cp_async_16(buf + o * 16, reinterpret_cast<const uint8_t*>(p.part_acc + at(o / (kRowB / 16)) * D) + (o % (kRowB / 16)) * 16);
#pragma unroll
      for (int y = 0; y < 2; ++y)
        if (lane + 32 * y < np) mls[lane + 32 * y] = v[y];
      cp_async_wait_all();
      __syncwarp();
      for (int r = 0; r < nr; ++r) {
        if (i0 == 0) {
          M = -INFINITY;
          L = 0.f;
          bad = false;
#pragma unroll
          for (int x = 0; x < C; ++x) acc[x] = 0.f;
        }
        float Mn = M;
        for (int i = 0; i < ni; ++i) {
          const float2 ml = mls[r * ni + i];
          bad |= ml.y < 0.f;
          if (ml.y > 0.f) Mn = fmaxf(Mn, ml.x);
        }
        const float a = Mn == -INFINITY ? 1.f : exp2f(M - Mn);
        M = Mn;
        L *= a;
#pragma unroll
        for (int x = 0; x < C; ++x) acc[x] *= a;
        for (int i = 0; i < ni; ++i) {
          const float2 ml = mls[r * ni + i];
          if (!(ml.y > 0.f)) continue;             // (a record without keys holds no sums)
          const float w = exp2f(ml.x - M);
          L = fmaf(w, ml.y, L);
          const float* src = reinterpret_cast<const float*>(buf + (r * ni + i) * kRowB) + lane * C;
#pragma unroll
          for (int x = 0; x < C; ++x) acc[x] = fmaf(w, src[x], acc[x]);
        }
        if (i0 + ni < nrec) continue;
        const int row = row0 + r;
        if (dst >= 0) {
          const size_t o = ((size_t)dst * e.c.Hkv + h) * kXRows + row;
#pragma unroll
          for (int x = 0; x < C; x += 2)
            *reinterpret_cast<float2*>(p.part_acc + o * D + lane * C + x) = make_float2(acc[x], acc[x + 1]);
          if (lane == 0) p.part_ml[o] = make_float2(M, bad ? kBadRecord : L);
        } else {
          const size_t o = (size_t)(s.q0 + row / e.G) * e.c.Hq + h * e.G + row % e.G;
          const bool none = bad || !(L > 0.f);
          const float inv = none ? 0.f : 1.f / L;
#pragma unroll
          for (int x = 0; x < C; x += 2)
            *reinterpret_cast<__half2*>(e.out + o * D + lane * C + x) =
                none ? __floats2half2_rn(0.f, 0.f) : __floats2half2_rn(acc[x] * inv, acc[x + 1] * inv);
          if (lane == 0 && e.lse) e.lse[o] = none ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
        }
      }
      __syncwarp();                                // the buffer is read before the next wave lands in it
    }
  }
}

// Takes a ticket on each of two counters (null: none) at once; bit x: this warp took the last of n[x] (the
// counter is left at zero). One fence and one round trip for both.
__device__ __forceinline__ uint32_t last_tickets(int* t0, int n0, int* t1, int n1) {
  uint32_t last = 0;
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    fence_acq_rel_gpu();                           // this warp's records first
    int o0 = -1, o1 = -1;
    if (t0) o0 = atomicAdd(t0, 1);
    if (t1) o1 = atomicAdd(t1, 1);
    if (t0 && o0 == n0 - 1) {
      *t0 = 0;
      last |= 1u;
    }
    if (t1 && o1 == n1 - 1) {
      *t1 = 0;
      last |= 2u;
    }
    if (last) fence_acq_rel_gpu();                 // and the others' before they are read
  }
  return __shfl_sync(0xffffffffu, last, 0);
}

}  // namespace xs

// ----------------------------------------------------------------------- kernel
template <int D, int VM, int NT>
__global__ void __launch_bounds__(kXThreads, 1)
extend_split_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV8,
                    const __grid_constant__ CUtensorMap tmV16, const ExtSplitParams p) {
  using namespace xs;
  using S = ExtSlot<D, VM>;
  constexpr int KS = D / 16;                       // k-steps of QK
  constexpr int MT = D / 16;                       // m-tiles of PV
  constexpr int CH = NT >= 4 ? 1 : 4 / NT;         // accumulation chains per tile of QK
  constexpr bool kQSmem = NT > 2;                  // query fragments in shared memory, else registers
  extern __shared__ uint8_t smem_raw[];
  __shared__ int warp_tot[kXWarps];
  uint8_t* smem = aligned_smem(smem_raw);
  const ExtendParams& e = p.e;
  const CacheView& c = e.c;
  int* cu = reinterpret_cast<int*>(smem + p.cu_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = c.Hkv, G = e.G, batch = c.batch;

  // ---- plan: this warp's range of pages
  const int total = plan(e, cu, warp_tot);
  const int nv = (int)gridDim.x * p.NG;
  const int vtotal = total + kSegmentCost * batch;
  const int per = total > 0 ? (vtotal + nv - 1) / nv : 1;
  if (total == 0 || (int)blockIdx.x * p.NG * per >= vtotal) return;
  for (int i = threadIdx.x; i < kXWarps * p.nsl; i += blockDim.x) {
    mbar_init(reinterpret_cast<uint64_t*>(smem + p.bar_off) + i, 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmK);
    if (VM == kXE4M3 || VM == kXMixed) tma_prefetch_desc(&tmV8);
    if (VM == kXFP16 || VM == kXMixed) tma_prefetch_desc(&tmV16);
  }
  __syncthreads();                                 // no barrier of the CTA follows
  const int h = warp % Hkv;
  const int v = (int)blockIdx.x * p.NG + warp / Hkv;
  const int start = page_at(cu, batch, v * per), end = page_at(cu, batch, min(vtotal, (v + 1) * per));
  if (start >= end) return;
  const int b_first = upper_bound_i(cu, batch + 1, start) - 1, b_last = upper_bound_i(cu, batch + 1, end - 1) - 1;
  const int n_my = end - start;

  Ring ring;
  ring.nsl = p.nsl;
  ring.k = smem + (size_t)warp * p.nsl * S::kK;
  ring.v = smem + p.v_off + (size_t)warp * p.nsl * S::kV;
  ring.full = reinterpret_cast<uint64_t*>(smem + p.bar_off) + warp * p.nsl;
  const int q4 = lane & 3, r8 = lane >> 2;
  const int lm_t = (lane & 7) + ((lane >> 3) & 1) * 8, lm_c = lane >> 4;   // ldmatrix row and 16-byte chunk of this lane

  // one scale for every code of the pool scales the output instead
  const bool scaled = VM == kXMixed || (VM == kXE4M3 && c.scale_mode == EKV_SCALE_PER_PAGE_HEAD);
  const float osc = VM == kXE4M3 && !scaled ? __ldg(c.v_scales) : 1.f;
  Meta cur, nxt, nxt2;
  meta_ids(e, cu, start, n_my, lane, cur);
  meta_ids(e, cu, start, n_my, 32 + lane, nxt);
  meta_mode<VM>(e, h, cur);
  for (int kk = 0; kk < min(ring.nsl, n_my); ++kk)
    fill<D, VM>(e, ring, kk, h, __shfl_sync(0xffffffffu, cur.page, kk), __shfl_sync(0xffffffffu, cur.flags, kk), &tmK,
                &tmV8, &tmV16);
  meta_mode<VM>(e, h, nxt);
  meta_ids(e, cu, start, n_my, 64 + lane, nxt2);

  int k = 0, s_idx = 0;
  uint32_t phase = 0;
  bool timed_out = false;
  for (int b = b_first; b <= b_last && !timed_out; ++b) {
    const int j0 = max(cu[b], start), j1 = min(cu[b + 1], end);
    if (j0 >= j1) continue;
    Seq sq;
    load_seq(e, b, sq);
    const int t0 = sq.L - sq.n;                    // position of the first new token
    const int R = sq.n * G, nt = (R + 7) / 8;      // rows and tiles in use
    // pages from here to there are seen in full by every row
    const int full_lo = max(0, sq.L - 1 - e.window + 1), full_hi = t0;   // first key of the last row's window, own key of row 0
    // B fragments of Q^T: lane holds Q[row = 8 i + r8][16 s + 2 q4 (+1)] and [+8]
    uint32_t qb[kQSmem ? 1 : NT][KS][2];
    const uint32_t q_sm = smem_u32(smem + p.q_off) + warp * (kXRows * D * 2);
    if (kQSmem) {
      // rows of D fp16 in 16-byte chunks, chunk c of row r at c ^ (r & 7)
      __syncwarp();
      for (int i = lane; i < NT * 8 * (D / 8); i += 32) {
        const int row = i / (D / 8), ch = i % (D / 8);
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (row < R)
          x = __ldg(reinterpret_cast<const uint4*>(e.q + ((size_t)(sq.q0 + row / G) * c.Hq + h * G + row % G) * D) + ch);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(q_sm + row * (D * 2) + ((ch ^ (row & 7)) << 4)),
                     "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w));
      }
      __syncwarp();
    } else {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int row = 8 * i + r8;
        const bool live = row < R;
        const __half* qr = e.q + ((size_t)(sq.q0 + (live ? row / G : 0)) * c.Hq + h * G + (live ? row % G : 0)) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          qb[i][s][0] = live ? __ldg(reinterpret_cast<const unsigned int*>(qr + 16 * s + 2 * q4)) : 0u;
          qb[i][s][1] = live ? __ldg(reinterpret_cast<const unsigned int*>(qr + 16 * s + 8 + 2 * q4)) : 0u;
        }
      }
    }
    float acc[NT][MT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int x = 0; x < MT; ++x) acc[i][x][0] = acc[i][x][1] = acc[i][x][2] = acc[i][x][3] = 0.f;
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
    }
    uint32_t bad_rows = 0;                         // bit 2 i + x: row 8 i + 2 q4 + x saw a failing page
    // the token of a row of this lane (rows past R count as the last row)
    const uint32_t rcp = 65536u / (uint32_t)G + 1u;   // row / G for row < 32, G <= 8
    auto token_of = [&](int row) { return min((int)((uint32_t)row * rcp >> 16), sq.n - 1); };

    const int r_end = j1 - start;
    for (; k < r_end; ++k) {
      if ((k & 31) == 0 && k > 0) {                // next batch of metadata
        cur = nxt;
        nxt = nxt2;
        meta_mode<VM>(e, h, nxt);
        meta_ids(e, cu, start, n_my, k + 64 + lane, nxt2);
      }
      if (!mbar_wait(&ring.full[s_idx], phase)) {
        if (lane == 0) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_TIMEOUT, blockIdx.x);
        for (int kk = k + 1; kk < min(k + ring.nsl, n_my); ++kk)
          mbar_wait(&ring.full[kk % ring.nsl], (uint32_t)(kk / ring.nsl) & 1u);
        timed_out = true;
        break;
      }
      const int flags = __shfl_sync(0xffffffffu, cur.flags, k & 31);
      const int key0 = __shfl_sync(0xffffffffu, cur.lp, k & 31) * kPage;
      const float lsc = scaled ? __shfl_sync(0xffffffffu, cur.lsc, k & 31) : 0.f;
      const float ivs = scaled ? __shfl_sync(0xffffffffu, cur.ivs, k & 31) : 1.f;
      const bool skip = (flags & kSkip) != 0;
      const bool e4 = VM == kXE4M3 || (VM == kXMixed && (flags & kE4));
      const bool bs = VM == kXMixed && (flags & kBs);
      const bool mx = VM == kXMicro || (VM == kXMixed && (flags & kMx));
      float sc[NT][4];
      uint32_t va[MT][4];
      if (!skip) {
        const uint32_t kp = smem_u32(ring.k + (size_t)s_idx * S::kK), vp = smem_u32(ring.v + (size_t)s_idx * S::kV);
        // ---- S^T = K Q^T
        uint32_t kf[KS][4];
#pragma unroll
        for (int s = 0; s < KS; ++s)
          ldsm_x4(kp + (s >> 2) * 2048 + swz128(lm_t * 128 + (2 * (s & 3) + lm_c) * 16), kf[s][0], kf[s][1], kf[s][2], kf[s][3]);
        float sx[NT][CH][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < CH; ++x) sx[i][x][0] = sx[i][x][1] = sx[i][x][2] = sx[i][x][3] = 0.f;
        if (kQSmem) {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if (i >= nt) continue;
#pragma unroll
            for (int s = 0; s < KS; s += 2) {
              // four 8x8 blocks: chunks 2s .. 2s+3 of rows 8i .. 8i+7, the B fragments of two k-steps
              uint32_t b0, b1, b2, b3;
              const int row = 8 * i + (lane & 7), ch = 2 * s + (lane >> 3);
              ldsm_x4(q_sm + row * (D * 2) + ((ch ^ (row & 7)) << 4), b0, b1, b2, b3);
              mma_f16(sx[i][0], kf[s][0], kf[s][1], kf[s][2], kf[s][3], b0, b1);
              mma_f16(sx[i][0], kf[s + 1][0], kf[s + 1][1], kf[s + 1][2], kf[s + 1][3], b2, b3);
            }
          }
        } else {
#pragma unroll
          for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int i = 0; i < NT; ++i)
              if (i < nt) mma_f16(sx[i][s % CH], kf[s][0], kf[s][1], kf[s][2], kf[s][3], qb[i][s][0], qb[i][s][1]);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            float t = sx[i][0][x];
#pragma unroll
            for (int y = 1; y < CH; ++y) t += sx[i][y][x];
            sc[i][x] = t;
          }
        // ---- V^T fragments: tokens 2 q4, 2 q4 + 1 (a0, a1) and + 8 (a2, a3); see the top
        if (mx) {
          uint32_t sw[4];                          // the scale bytes of the lane's 4 tokens
          bool sb_bad = false;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int t = 2 * q4 + (x & 1) + 8 * (x >> 1);
            const uint32_t a = vp + micro_scale_off(D) + t * (D / kMicroBlock);
            if (D == 128) {
              sw[x] = lds32(a);
            } else {
              uint16_t two;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(two) : "r"(a));
              sw[x] = two;
            }
            const bool seen = key0 + t >= t0 - e.window + 1 && key0 + t < sq.L;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
              if (seen && !micro_scale_ok((sw[x] >> (8 * j)) & 0xffu)) {   // a byte that no writer leaves: zeros
                sb_bad = true;
                sw[x] &= ~(0xffu << (8 * j));
              }
            }
          }
          if (sb_bad) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SCALE, b);
#pragma unroll
          for (int jj = 0; jj < D / 64; ++jj) {
            uint32_t w[4];                         // [block 2 jj, tokens 0-7], [8-15], [block 2 jj + 1, ...]
            ldsm_x4_trans(vp + lm_t * (D / 2) + (2 * jj + lm_c) * 16, w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int j = 2 * jj + y;
#pragma unroll
              for (int z = 0; z < 2; ++z) {        // tokens 0-7, 8-15
                const uint32_t reg = w[2 * y + z];
                const uint32_t ev = (reg & 0x0f0fu) | ((reg >> 12) & 0xf0f0u);
                const uint32_t od = ((reg >> 4) & 0x0f0fu) | ((reg >> 16) & 0xf0f0u);
                const uint32_t s2 = bits(__floats2half2_rn(__uint_as_float(((sw[2 * z] >> (8 * j)) & 0xffu) << 23),
                                                           __uint_as_float(((sw[2 * z + 1] >> (8 * j)) & 0xffu) << 23)));
                va[2 * j][2 * z] = fp4_pair(ev, s2);
                va[2 * j][2 * z + 1] = fp4_pair(od, s2);
                va[2 * j + 1][2 * z] = fp4_pair(ev >> 8, s2);
                va[2 * j + 1][2 * z + 1] = fp4_pair(od >> 8, s2);
              }
            }
          }
        } else if (e4 || bs) {
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int t = 2 * q4 + 8 * z, col = 32 * j + 4 * r8;
              const uint32_t w0 = lds32(vp + (D == 128 ? swz128(t * 128 + col) : swz64(t * 64 + col)));
              const uint32_t w1 = lds32(vp + (D == 128 ? swz128((t + 1) * 128 + col) : swz64((t + 1) * 64 + col)));
              if (bs) {                            // the byte is the high half of an fp16 word
                va[2 * j][2 * z] = (w0 & 0xffu) << 8 | (w1 & 0xffu) << 24;
                va[2 * j][2 * z + 1] = (w0 & 0xff00u) | (w1 & 0xff00u) << 16;
                va[2 * j + 1][2 * z] = ((w0 >> 8) & 0xff00u) | ((w1 << 8) & 0xff000000u);
                va[2 * j + 1][2 * z + 1] = ((w0 >> 16) & 0xff00u) | (w1 & 0xff000000u);
              } else {
                const uint32_t lo = __byte_perm(w0, w1, 0x5140), hi = __byte_perm(w0, w1, 0x7362);
                va[2 * j][2 * z] = bits(e4m3x2_to_half2((uint16_t)lo));
                va[2 * j][2 * z + 1] = bits(e4m3x2_to_half2((uint16_t)(lo >> 16)));
                va[2 * j + 1][2 * z] = bits(e4m3x2_to_half2((uint16_t)hi));
                va[2 * j + 1][2 * z + 1] = bits(e4m3x2_to_half2((uint16_t)(hi >> 16)));
              }
            }
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int t = 2 * q4 + 8 * z, d = 32 * j + 4 * r8;
              const uint32_t box = vp + (d >> 6) * 2048, col = (d & 63) * 2;
              const uint2 w0 = lds64(box + swz128(t * 128 + col)), w1 = lds64(box + swz128((t + 1) * 128 + col));
              va[2 * j][2 * z] = __byte_perm(w0.x, w1.x, 0x5410);
              va[2 * j][2 * z + 1] = __byte_perm(w0.x, w1.x, 0x7632);
              va[2 * j + 1][2 * z] = __byte_perm(w0.y, w1.y, 0x5410);
              va[2 * j + 1][2 * z + 1] = __byte_perm(w0.y, w1.y, 0x7632);
            }
        }
      }
      // ---- the slot is in registers: refill it with page k + nsl
      fence_reads_before_refill();
      __syncwarp();
      {
        const int kk = k + ring.nsl;
        if (kk < n_my) {
          const bool in_cur = (kk >> 5) == (k >> 5);
          const int pg = __shfl_sync(0xffffffffu, in_cur ? cur.page : nxt.page, kk & 31);
          const int fl = __shfl_sync(0xffffffffu, in_cur ? cur.flags : nxt.flags, kk & 31);
          fill<D, VM>(e, ring, s_idx, h, pg, fl, &tmK, &tmV8, &tmV16);
        }
      }
      if (skip) {                                  // rows that see a key of the page
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int t = t0 + token_of(8 * i + 2 * q4 + x);
            if (key0 <= t && key0 + kPage - 1 > t - e.window) bad_rows |= 1u << (2 * i + x);
          }
      } else {
        // ---- scores in log2 units, E4M3 scale included; tokens r8 and r8 + 8
        const bool partial = key0 < full_lo || key0 + kPage - 1 > full_hi;
        bool grows = false;
        float mxs[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[i][x] = fmaf(sc[i][x], e.qscale, lsc);
          if (partial) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int t = t0 + token_of(8 * i + 2 * q4 + x);
              const int lo = t - e.window;         // keys lo + 1 .. t
              if (key0 + r8 > t || key0 + r8 <= lo) sc[i][x] = -INFINITY;
              if (key0 + r8 + 8 > t || key0 + r8 + 8 <= lo) sc[i][2 + x] = -INFINITY;
            }
          }
          mxs[i][0] = fmaxf(sc[i][0], sc[i][2]);
          mxs[i][1] = fmaxf(sc[i][1], sc[i][3]);
          if (i < nt) grows |= mxs[i][0] > m[i][0] + 8.f || mxs[i][1] > m[i][1] + 8.f;
        }
        // the reference maximum moves only when a score passes it by 2^8 (the weights stay below 256)
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if (i >= nt) continue;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float t = mxs[i][x];
#pragma unroll
              for (int o = 4; o <= 16; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
              const float mn = fmaxf(m[i][x], t);
              const float a = mn == -INFINITY ? 1.f : ex2(m[i][x] - mn);
              m[i][x] = mn;
              l[i][x] *= a;
#pragma unroll
              for (int y = 0; y < MT; ++y) {
                acc[i][y][x] *= a;
                acc[i][y][2 + x] *= a;
              }
            }
          }
        }
        // value rows that no row of the sequence sees count as zero, whatever they hold
        if (partial) {
          const int lo = max(0, t0 - e.window + 1) - key0, hi = sq.L - key0;   // tokens lo .. hi - 1
          const int ta = 2 * q4;
          const uint32_t mlo = (ta >= lo && ta < hi ? 0xffffu : 0u) | (ta + 1 >= lo && ta + 1 < hi ? 0xffff0000u : 0u);
          const uint32_t mhi = (ta + 8 >= lo && ta + 8 < hi ? 0xffffu : 0u) | (ta + 9 >= lo && ta + 9 < hi ? 0xffff0000u : 0u);
#pragma unroll
          for (int y = 0; y < MT; ++y) {
            va[y][0] &= mlo;
            va[y][1] &= mlo;
            va[y][2] &= mhi;
            va[y][3] &= mhi;
          }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if (i >= nt) continue;
          // a row that has seen no key yet keeps m = -inf: its weights are 2^-inf = 0
          const float m0 = m[i][0] == -INFINITY ? 0.f : m[i][0], m1 = m[i][1] == -INFINITY ? 0.f : m[i][1];
          const float p00 = ex2(sc[i][0] - m0), p01 = ex2(sc[i][1] - m1), p10 = ex2(sc[i][2] - m0), p11 = ex2(sc[i][3] - m1);
          // the sum takes the weights unrounded: lse is an fp32 result
          l[i][0] = fmaf(p00 + p10, ivs, l[i][0]);
          l[i][1] = fmaf(p01 + p11, ivs, l[i][1]);
          const __half2 plo = __floats2half2_rn(p00, p01), phi = __floats2half2_rn(p10, p11);
          const uint32_t pb0 = movmatrix_trans(bits(plo)), pb1 = movmatrix_trans(bits(phi));
#pragma unroll
          for (int y = 0; y < MT; ++y) mma_f16(acc[i][y], va[y][0], va[y][1], va[y][2], va[y][3], pb0, pb1);
        }
      }
      if (++s_idx == ring.nsl) {
        s_idx = 0;
        phase ^= 1u;
      }
    }
    if (timed_out) break;
    // ---- the segment's end: the output if the sequence lies in this range, else a record
    const bool whole = cu[b] >= start && cu[b + 1] <= end;
    const int rec = 2 * v + (b == b_first ? 0 : 1);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (i >= nt) continue;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float t = l[i][x];
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        const int row = 8 * i + 2 * q4 + x;
        if (row >= R) continue;
        const bool bad = (bad_rows >> (2 * i + x)) & 1u;
        if (whole) {
          const size_t o = (size_t)(sq.q0 + row / G) * c.Hq + h * G + row % G;
          const float inv = bad || !(t > 0.f) ? 0.f : osc / t;
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            uint2 u;
            u.x = bits(__floats2half2_rn(acc[i][2 * j][x] * inv, acc[i][2 * j][2 + x] * inv));
            u.y = bits(__floats2half2_rn(acc[i][2 * j + 1][x] * inv, acc[i][2 * j + 1][2 + x] * inv));
            if (bad) u = make_uint2(0u, 0u);
            *reinterpret_cast<uint2*>(e.out + o * D + 32 * j + 4 * r8) = u;
          }
          if (r8 == 0 && e.lse) e.lse[o] = !bad && t > 0.f ? (m[i][x] + log2f(t)) * 0.69314718055994531f : -INFINITY;
        } else {
          const size_t o = ((size_t)rec * Hkv + h) * kXRows + row;
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
            *reinterpret_cast<float4*>(p.part_acc + o * D + 32 * j + 4 * r8) =
                make_float4(acc[i][2 * j][x] * osc, acc[i][2 * j][2 + x] * osc, acc[i][2 * j + 1][x] * osc, acc[i][2 * j + 1][2 + x] * osc);
          if (r8 == 0) p.part_ml[o] = make_float2(m[i][x], bad ? kBadRecord : t);
        }
      }
    }
  }
  // ---- joining: the sequences that continue in other ranges (a range's first and last segment at most)
  struct Side {
    int b, v0, n, first, gv, gn, gfirst;           // sequence, its ranges, its first record; this range's group
    int* ticket;
  } side[2];
  auto open = [&](int b, Side& x) {
    x.ticket = nullptr;
    if (cu[b] == cu[b + 1] || (cu[b] >= start && cu[b + 1] <= end)) return;
    x.b = b;
    ranges_of(cu, b, per, x.v0, x.n);
    // range v0 may begin inside the sequence before: then b is its last segment there
    x.first = 2 * x.v0 + (page_at(cu, batch, x.v0 * per) < cu[b] ? 1 : 0);
    const int g = x.n <= kJoin ? 0 : (v - x.v0) / kJoin;
    x.gv = x.v0 + g * kJoin;
    x.gn = min(kJoin, x.n - g * kJoin);
    x.gfirst = g == 0 ? x.first : 2 * x.gv;
    x.ticket = x.n <= kJoin ? p.ticket + b * kMaxKvHeads + h : p.group_ticket + (2 * x.gv + (g == 0 ? 1 : 0)) * Hkv + h;
  };
  open(b_first, side[0]);
  if (b_last != b_first) open(b_last, side[1]);
  else side[1].ticket = nullptr;
  if (!side[0].ticket && !side[1].ticket) return;
  const uint32_t last = last_tickets(side[0].ticket, side[0].ticket ? side[0].gn : 0, side[1].ticket, side[1].ticket ? side[1].gn : 0);
  for (int x = 0; x < 2; ++x) {
    if (!((last >> x) & 1u)) continue;
    const Side& d = side[x];
    Seq sq;
    load_seq(e, d.b, sq);
    uint8_t* buf = ring.k;
    const int bytes = ring.nsl * S::kK;
    if (d.n <= kJoin) {
      join<D>(p, h, sq, d.first, 2 * d.v0, 2, d.n, -1, buf, bytes);
      continue;
    }
    join<D>(p, h, sq, d.gfirst, 2 * d.gv, 2, d.gn, d.gfirst, buf, bytes);
    const int groups = (d.n + kJoin - 1) / kJoin;
    if (last_tickets(p.ticket + d.b * kMaxKvHeads + h, groups, nullptr, 0))
      join<D>(p, h, sq, d.first, 2 * d.v0, 2 * kJoin, groups, -1, buf, bytes);
  }
}

// Shared memory: K slots, V slots, barriers, plan, and (more than two tiles) the query rows.
template <int D, int VM, int NT>
size_t ext_split_layout(ExtSplitParams& p) {
  using S = ExtSlot<D, VM>;
  const int plan_bytes = (p.e.c.batch + 1 + 3) / 4 * 16;
  const int q_bytes = NT > 2 ? kXWarps * kXRows * D * 2 : 0;
  const int room = kSplitSmemMax - 1024 - plan_bytes - q_bytes;
  int nsl = room / (kXWarps * (S::kK + S::kV + 8));
  while (kXWarps * nsl * S::kK + (kXWarps * nsl * S::kV + 127) / 128 * 128 + kXWarps * nsl * 8 > room) --nsl;
  p.nsl = nsl > kMaxSlots ? kMaxSlots : nsl;
  p.v_off = kXWarps * p.nsl * S::kK;
  p.q_off = p.v_off + (kXWarps * p.nsl * S::kV + 127) / 128 * 128;
  p.bar_off = p.q_off + q_bytes;
  p.cu_off = p.bar_off + kXWarps * p.nsl * 8;
  return 1024 + p.cu_off + plan_bytes;
}

cudaError_t set_smem_attr(const void* kern, int bytes);

template <int D, int VM, int NT>
cudaError_t launch_ext_split(const CUtensorMap (&tm)[3], ExtSplitParams p, int grid, cudaStream_t st) {
  auto kern = extend_split_kernel<D, VM, NT>;
  const size_t smem = ext_split_layout<D, VM, NT>(p);
  cudaError_t e = set_smem_attr(reinterpret_cast<const void*>(kern), kSplitSmemMax);
  if (e != cudaSuccess) return e;
  kern<<<grid, kXThreads, smem, st>>>(tm[0], tm[1], tm[2], p);
  return cudaGetLastError();
}

template <int D, int VM>
cudaError_t launch_ext_split_nt(const CUtensorMap (&tm)[3], const ExtSplitParams& p, int grid, cudaStream_t st) {
  const int rows = p.e.G * p.e.max_q;
  if (rows <= 8) return launch_ext_split<D, VM, 1>(tm, p, grid, st);
  if (rows <= 16) return launch_ext_split<D, VM, 2>(tm, p, grid, st);
  return launch_ext_split<D, VM, 4>(tm, p, grid, st);
}

template <int D>
cudaError_t launch_ext_split_d(const CUtensorMap (&tm)[3], const ExtSplitParams& p, int vm, int grid, cudaStream_t st) {
  switch (vm) {
    case kXFP16: return launch_ext_split_nt<D, kXFP16>(tm, p, grid, st);
    case kXE4M3: return launch_ext_split_nt<D, kXE4M3>(tm, p, grid, st);
    case kXMicro: return launch_ext_split_nt<D, kXMicro>(tm, p, grid, st);
    default: return launch_ext_split_nt<D, kXMixed>(tm, p, grid, st);
  }
}

}  // namespace ekv
