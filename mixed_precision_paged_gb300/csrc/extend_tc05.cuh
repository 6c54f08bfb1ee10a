// extend_tc05.cuh -- attention of new tokens over the paged cache (decode steps, draft
// verification, prompt chunks behind a cached prefix) on the fifth-generation tensor cores.
//
// For a block of 128 keys and a tile of 128 query rows the work is two products,
//   S = Q K^T,  O += P V,  P = 2^(S sm_scale log2 e - m),
// 4 * 128 * 128 * D operations against 128 * D * (2 + 1) bytes of a K16/V8 block: with 256 rows the tensor
// pipe bounds it, and the softmax (128 exponentials a row and block) comes next. So:
//   * rows: a tile packs the G query heads of a KV head, row = token * G + g, 128 / G tokens each,
//     and a work item is a pair of tiles that share every block: one read of K and V serves 256
//     rows, and one tile's softmax runs while the other's products do.
//   * blocks: 8 pages by one TMA box each, 8-token groups of [D / 64][8 rows][128 B] (128B swizzle),
//     which serve as K-major B of S and, for V, as N-major B of the second product.
//   * values: FP16 pages land in a V stage directly. E4M3, BASE and microscaled pages land raw, in a ring
//     that one warp fills for all makers or each maker for itself (loads and conversions of one warp
//     wait for one another: 200 microscaled sequences 139 us, with the loader 129), and are expanded into
//     the V stage, exactly; E4M3 scales join the exponent, p' = 2^(score + log2 scale - m) with the
//     maximum m over the scaled scores, and the sum takes p' / scale: so codes enter the product exactly
//     as they are, and p' is rounded to fp16 once relative to the row's largest weight times scale;
//     one scale for all codes scales the output instead. A microscaled value is code * 2^k, exact in fp16.
//   * split: the blocks of all items form one stream, cut into equal ranges, one persistent CTA
//     each; an item that crosses a border leaves partial rows (m, l, O) in at most two slots a CTA, and
//     a second kernel joins them. Long causal chunks so balance to a block, and one short chunk
//     behind a long prefix still uses every SM.
// Roles: warp 0 checks the pages and loads Q and K; warp 1 issues the MMAs; warp 3 loads FP16 value
// pages; warps 4-7 and 8-11 are the softmax of tile 0 and 1, a thread per row; the others are makers,
// which expand the other pages, or their loader (warp 2 also owns tensor memory). The registers are
// split to match (setmaxnreg): 80, 176, 176 and 80 a thread, 512 = 4 x the 128 of launch. Tensor memory
// of tile t: S and P at 256 t, O at 256 t + 128. The order of the MMAs and the lazily moved maximum are those of the
// prefill (prefill_tc05.cu).
// The instruction cache is a resource here: sixteen warps run seven different loops, and once these no
// longer fitted it (a second copy of the makers' loop, deeper unrolling) every role slowed down two- to
// threefold, with the GPC's instruction cache at 86% of its request rate. So a role's loop stands once, the
// makers are driven by block descriptions instead of walking the plan, and unrolling is chosen by measurement.
// Every wait is bounded; a timeout is reported and every role winds down.
// Rounding: scores, maxima, sums, partial rows and outputs up to the last step are fp32. The weights go to fp16, which is
// what the tensor core multiplies by fp16 values (bf16 has three bits less, and TF32 half the rate and twice the bytes of V):
// up to 2^-11 of a weight, which the result's own rounding to fp16 hides but for a tenth (against 64 bits, relative:
// 2.0e-4 to 2.2e-4 over the measured cases, 1.9e-4 to 2.1e-4 with fp32 weights). ex2.approx is off by 2^-22.
// Measured, 32/8 heads, D 128: 32 x 1 token behind 8K keys of E4M3 144 us (5.6 TB/s, 6.6 between start and end), 48 x 5
// over mixed pages 147 us, 4,096 tokens behind 16K of E4M3 840 to 910 us (1,480 to 1,360 TFLOP/s): a step of two tiles
// takes 3,300 cycles for 2,176 of MMA, the hand-overs between softmax and products the rest.
#pragma once

#include "extend.cuh"
#include "micro.cuh"
#include "pool_maps.h"
#include "tc05.cuh"

namespace ekv {

enum ExtVMode { kXFP16 = 0, kXE4M3 = 1, kXMicro = 2, kXMixed = 3 };   // forms of a launch's value pages

constexpr float kBadRecord = -1.f;          // l of a row that saw a page which failed its checks
constexpr int kTRows = 128;                 // rows of a query tile (MMA M)
constexpr int kTKeys = 128;                 // keys of a block (N of S)
constexpr int kTPages = kTKeys / kPage;
constexpr int kT5Threads = 512;
constexpr int kAltRows = 64;                // rows of a sequence and KV head up to which blocks alternate
constexpr int kMetaAhead = 2;               // blocks that page lookups are ahead of the K loads
// The reference m of a row lies this far below its maximum (in log2), so weights are up to 2^7, and 2^15 before a
// reference is moved (8 later): near the top of fp16's range, so that weights keep all their bits down to 2^-21 of the largest
// weight times scale, and what is rounded below costs 2^-32 of it. With the maximum itself as the reference a page of
// zeros (scale 1) took that precision from pages whose scale is small: values of 1e-4 came out 3% off.
constexpr float kHeadroom = 7.f;
// E4M3 scales where they differ by page, or beside pages of other forms: a page beyond kScaleMost fails its check (above
// 2^25 no code but 0 stands for a value within fp16's range), and below kScaleLeast a scale counts as that (such values,
// under 448 * 2^-44 < 2^-35, leave no trace in an fp16 output). So 1 / scale is finite, and a weight p' = 2^(score +
// log2 scale - m) that ex2 flushes, below 2^-126, belongs to a key that is at most 2^-126 * 2^(40 + 44) = 2^-42 of the
// sum, however the scales differ.
constexpr float kScaleLeast = 1.f / (1ll << 44), kScaleMost = (float)(1ll << 40);

struct ExtTcSplit {                         // an item that crosses CTAs, for the joining kernel
  int n;                                    // CTAs it spans; 0: none
  int first;                                // its first slot; the others are 2 * (cta + H_kv), ...
  int b, h, i;
};

struct ExtTcParams {
  ExtendParams e;
  float* part_acc;                          // [2 * grid][256][D]
  float2* part_ml;                          // [2 * grid][256]
  ExtTcSplit* split;                        // [grid]
  const float* scale_ptr;                   // one E4M3 scale for every code (it scales the output), or null
  int nw;                                   // ALT: softmax warps of a stream, for rows below 32 * nw
  int v16_mul, v16_head;                    // FP16 value map: index = page * v16_mul + head * v16_head
#ifdef EKV_TEST_WAIT_TIMEOUT
  int inject_timeout;                       // test build only: the wait of CTA 0 that runs out, see the kernel; 0: none
#endif
};

template <int D, int VM, bool ALT>
struct XT {
  static constexpr int NB = D / 64;                    // 64-value slabs of a row
  static constexpr int GB = NB * 1024;                 // bytes of an 8-token group
  static constexpr int QB = (ALT ? kAltRows : kTRows) * D * 2;   // a query tile (ALT: or two of half the rows)
  static constexpr int IB = kTKeys * D * 2;            // a K or V block
  static constexpr int RB = VM == kXFP16 ? 0 : kTKeys * D;   // a raw block: a page at every 16 * D bytes
  static constexpr int NQ = ALT ? 1 : 2;               // query tiles
  static constexpr int NK = (VM == kXFP16 || ALT ? (D == 128 ? 3 : 5) : (D == 128 ? 2 : 4)) + (ALT && D == 64 ? 1 : 0);
  static constexpr int NV = (D == 128 ? 2 : 4) + (ALT && VM == kXFP16 ? 1 : 0);
  static constexpr int NR = (D == 128 ? 2 : 4) + (ALT ? 1 : 0);
  // maker warps: warps 2 and 13-15, warp 3 too where there are no FP16 pages for it to load, and warp 12
  // too where blocks are shared by two tiles and so last longer
  static constexpr int MK = VM == kXFP16 || VM == kXMixed ? 4 : ALT ? 5 : 6;
  // five or four makers leave warp 12 to load the raw pages for all of them
  static constexpr bool kLoader = VM != kXFP16 && MK < 6;
  // Block descriptions. One is written once the K stage NK + kMetaAhead + 1 blocks back is free, so
  // once that block's S is issued, which is behind the product of the block before (ALT: two before).
  static constexpr int NM = D == 128 ? 8 : 12;
  static constexpr int NS = 8;                         // segment descriptions (see the producer)
  static_assert(NM >= NK + kMetaAhead + (ALT ? 3 : 2), "a description is read until its block's weights are handed over");
};

struct BlockMeta {
  int page[kTPages];
  float lsc[kTPages];                       // log2 of the scale
  float ivs[kTPages];                       // and its reciprocal
  int bad;                                  // bit per page that failed its checks
  int qtok;                                 // a segment's first block: first row of its queries; else -1
  uint8_t flags[kTPages];                   // kSkip: not loaded
  uint8_t tiles;                            // bit per tile with blocks in the segment
  uint8_t last;                             // the CTA's last block
  uint8_t z0, z1;                           // keys of the block that some row of the item sees: [z0, z1)
};

struct SegMeta {                            // a segment: the blocks of one item in one CTA's range
  int n;                                    // blocks; 0: no segment follows
  int nt[2];                                // of them, those that each tile takes part in, from the first on
  int ja;                                   // first block, of the sequence
  int q0, ntok, t0;                         // the sequence: first row of q, new tokens, position of the first
  int i;                                    // the item
  int slot;                                 // of the partial rows; -1: the whole item
};

template <int D, int VM, bool ALT>
struct XTBars {
  using C = XT<D, VM, ALT>;
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[C::NK], k_empty[C::NK];
  uint64_t raw_full[C::NR][C::MK], raw_empty[C::NR];   // (with a loader warp: raw_full[..][0])
  uint64_t v_full[C::NV], v_empty[C::NV];
  uint64_t v_dir[C::NV];                    // FP16 pages of a stage whose edge rows are zeroed after they land
  uint64_t meta_full[C::NM];
  uint64_t seg_full[C::NS], seg_empty[C::NS];
  uint64_t s_full[2], p_full[2], pv_done[2], o_free[2];
  uint64_t mma_final;
  uint64_t x_full[2];                       // ALT: a stream's (m, l) of the segment posted
  float2 xch[2][ALT ? kAltRows : 1];
  BlockMeta meta[C::NM];
  SegMeta seg[C::NS];
  long long red[kT5Threads / 32];
  int st_b, st_off;                         // where this CTA's range begins: sequence, blocks into it
  uint32_t tmem_base;
  int abort;
};

template <int D, int VM, bool ALT>
constexpr int xt_smem_bytes() {
  using C = XT<D, VM, ALT>;
  return C::NQ * C::QB + C::NK * C::IB + C::NV * C::IB + C::NR * C::RB + (int)sizeof(XTBars<D, VM, ALT>);
}

namespace xt {

constexpr int kSkip = 1, kE4 = 2, kBs = 4, kMx = 8;   // a page's flags: not loaded; its form (FP16: 0)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// One sequence's part in the plan.
struct Seq {
  int L, n, q0;            // tokens, new tokens, first row of q
};

// Reads sequence b; false when it has no new tokens (see seq_ok for its checks).
__device__ __forceinline__ bool load_seq(const ExtendParams& e, int b, Seq& s) {
  const CacheView& c = e.c;
  s.q0 = __ldg(c.cu_q + b);
  s.n = __ldg(c.cu_q + b + 1) - s.q0;
  s.L = __ldg(c.seq_lens + b);
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

// A warp's wait for a phase, bounded, that also gives up once another role has: false then. One compact loop:
// it stands at every wait of every role (see the instruction cache below).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = globaltimer_ns();
    while (!(ok = mbar_try_wait(bar, parity)))
      if (*abort || globaltimer_ns() - t0 > kWaitTimeoutNs) break;
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void give_up(int* err, volatile int* abort) {
  if (!*abort) report_error(err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_TIMEOUT, -1);
  *abort = 1;
}
// A bounded wait that ignores an abort: for copies in flight at the end.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
  }
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// (d0, d1) = (a0, a1) * b + c, and (a0, a1) += (b0, b1): packed FP32 instructions
__device__ __forceinline__ void ffma2(float& d0, float& d1, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %5};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void fadd2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 ra, rb;\n\t"
      "mov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %3};\n\t"
      "add.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ void tst16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// ------------------------------------------------------------------------ plan
// The sum of floor((a i + b) / m) over i < n, a and b >= 0. Multiples of m within a and b are summed at once. What
// is left (a, b < m) counts the pairs (i, k >= 1) with k m <= a i + b: of all n K of them, K the last term's floor, without
// those with i < ceil((k m - b) / a), which over k = 1 .. K are a sum of this kind with a and m exchanged.
// In 32 bits that wrap, as the result is below 2^31 (n <= 2^16 items of up to 2^14 blocks, and K <= n).
__device__ __forceinline__ int sum_of_floors(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  uint32_t total = 0, sign = 1;                        // sign: 1 or -1
  while (n > 0) {
    const uint32_t ra = a % m, rb = b % m, K = (ra * (n - 1) + rb) / m;
    total += sign * (n * (n - 1) / 2 * (a / m) + n * (b / m) + n * K);
    sign = 0u - sign;
    n = K;                                             // ceil((k m - rb) / ra) = floor((m (k - 1) + m - rb + ra - 1) / ra)
    a = m;
    b = m - rb + ra - 1;
    m = ra;
  }
  return (int)total;
}

// What an item's start and end (queries, first scores, epilogue) cost, in blocks. ALT, 1 / 2 / 3 / 4: 200 microscaled
// sequences of 1-4 tokens 125 / 123 / 121 / 122 us; pairs, 1 / 2: chunks 229.4 / 229.6 us.
template <bool ALT>
constexpr int kItemCost = ALT ? 3 : 1;

// The items of one sequence and KV head: pairs of tiles, `step` tokens each.
struct Items {
  int n, t0, np;              // new tokens, position of the first, items
  int step, window;
  // keys of item i: [lo, hi)
  __device__ __forceinline__ int lo(int i) const {
    const int first = t0 + i * step;
    return first < window ? 0 : first - window + 1;
  }
  __device__ __forceinline__ int hi(int i) const { return t0 + min((i + 1) * step, n); }
  __device__ __forceinline__ int jlo(int i) const { return lo(i) / kTKeys; }
  __device__ __forceinline__ int jhi(int i) const { return (hi(i) + kTKeys - 1) / kTKeys; }
  // blocks, and kItemCost each, of the items before i
  template <bool ALT>
  __device__ __forceinline__ int before(int i) const {
    if (i <= 0) return 0;
    if (ALT) return kItemCost<ALT> + jhi(0) - jlo(0);      // (one item)
    const int full = i == np ? np - 1 : i;            // the last item may be short
    int s = kItemCost<ALT> * i + sum_of_floors(full, kTKeys, step, t0 + step + kTKeys - 1);
    if (i == np) s += jhi(np - 1);
    const int i0 = t0 >= window - 1 ? 0 : min(i, (window - 2 - t0) / step + 1);   // items whose window starts at key 0
    if (i > i0) s -= sum_of_floors(i - i0, kTKeys, step, t0 + i0 * step - window + 1);
    return s;
  }
};
template <bool ALT>
__device__ __forceinline__ Items items_of(const ExtendParams& e, const Seq& s) {
  Items it;
  it.n = s.n;
  it.t0 = s.L - s.n;
  it.step = (ALT ? 1 : 2) * e.tile_tokens;
  it.np = (s.n + it.step - 1) / it.step;
  it.window = e.window;
  return it;
}

// The producer's walk over the CTA's segments.
struct Walk {
  int b, i, j;              // next: sequence, item, block (j may lie kItemCost before the item's first)
  int budget;               // blocks left in the CTA's range
  int index, u;             // segments and blocks so far
  int q0;                   // the sequence's first row of q
  Items it;
};
struct Segment {
  int ja, jb;               // blocks
  int jlo, jhi;             // of the whole item
  int i, slot;
  int b, q0, n, t0;         // the sequence: its index, first row of q, new tokens, position of the first
  int lo, hi;               // keys that the item sees
  int nt[2];                // blocks that each tile takes part in, from ja on
  bool whole;
};

template <bool ALT>
__device__ __forceinline__ bool walk_next(const ExtendParams& e, Walk& w, Segment& sg) {
  while (w.budget > 0 && w.b < e.c.batch) {
    sg.jlo = w.it.jlo(w.i);
    sg.jhi = w.it.jhi(w.i);
    sg.i = w.i;
    sg.b = w.b;
    sg.q0 = w.q0;
    sg.n = w.it.n;
    sg.t0 = w.it.t0;
    sg.lo = w.it.lo(w.i);
    sg.hi = w.it.hi(w.i);
    const int ja = w.j, jb = min(sg.jhi, w.j + w.budget);
    w.budget -= jb - ja;
    w.j = jb;
    sg.ja = max(ja, sg.jlo);
    sg.jb = jb;
    sg.whole = sg.ja == sg.jlo && jb == sg.jhi;
    if (ALT) {                                       // one tile, its blocks in turn
      sg.nt[0] = (jb - sg.ja + 1 - (w.u & 1)) / 2;
      sg.nt[1] = (jb - sg.ja + (w.u & 1)) / 2;
    } else {                                         // tile 0 ends with its own last token's block
      const int half = w.it.step / 2;
      const int e0 = (w.it.t0 + min(w.i * w.it.step + half, w.it.n) + kTKeys - 1) / kTKeys;
      sg.nt[0] = max(0, min(jb, e0) - sg.ja);
      sg.nt[1] = w.i * w.it.step + half < w.it.n ? max(0, jb - sg.ja) : 0;
    }
    if (jb == sg.jhi) {                              // on to the next item
      if (++w.i == w.it.np) {
        w.i = 0;
        Seq sq;
        do {
          ++w.b;
        } while (w.b < e.c.batch && (!load_seq(e, w.b, sq) || !seq_ok(e, sq)));
        if (w.b < e.c.batch) {
          w.q0 = sq.q0;
          w.it = items_of<ALT>(e, sq);
        }
      }
      if (w.b < e.c.batch) w.j = w.it.jlo(w.i) - kItemCost<ALT>;
    }
    if (sg.ja < sg.jb) {
      sg.slot = 2 * (int)blockIdx.x + (w.index == 0 ? 0 : 1);
      ++w.index;
      w.u += sg.jb - sg.ja;
      return true;
    }
  }
  return false;
}

}  // namespace xt

// -------------------------------------------------------------------- the kernel
// PS: E4M3 scales differ by page (and head), or pages differ in form. ALT: every sequence's rows are at most
// kAltRows; its key blocks alternate between the two softmax groups ("streams"), whose results are joined
// at the end of a segment: with one tile in use, a block's chain (S, softmax, P V: ~3,300 cycles) would bound
// the stream at two thirds of HBM rate; two chains in turn leave it to the loads.
template <int D, int VM, bool PS, bool ALT>
__global__ void __launch_bounds__(kT5Threads, 1)
extend_tc05_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv16, const __grid_constant__ CUtensorMap tv8,
                   const ExtTcParams p) {
  using namespace xt;
  using C = XT<D, VM, ALT>;
  using Bars = XTBars<D, VM, ALT>;
  constexpr int NK = C::NK, NV = C::NV, NR = C::NR, NM = C::NM, NB = C::NB;
  extern __shared__ __align__(1024) uint8_t sm_1k[];   // (no room to align by hand)
  uint8_t* sQ = sm_1k;                                  // [2][NB][128 rows][128 B]
  uint8_t* sK = sQ + C::NQ * C::QB;                    // [NK][16 groups][NB][8 rows][128 B]
  uint8_t* sV = sK + NK * C::IB;
  uint8_t* sR = sV + NV * C::IB;                       // [NR][8 pages][16 * D B]
  Bars* bars = reinterpret_cast<Bars*>(sR + NR * C::RB);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ExtendParams& e = p.e;
  const CacheView& c = e.c;
  if (smem_u32(sm_1k) & 1023u) {                       // the swizzled layouts would not hold
    if (threadIdx.x == 0) {
      report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_TIMEOUT, -2);
      p.split[blockIdx.x].n = 0;
    }
    return;
  }
  const int nw = ALT ? p.nw : kTRows / 32;             // softmax warps per tile (ALT: those with rows)
  constexpr bool kDirect = VM == kXFP16 || VM == kXMixed, kRaw = VM != kXFP16;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], 1);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], nw);
      mbar_init(&bars->pv_done[t], 1);
      mbar_init(&bars->o_free[t], ALT ? 2 * nw : nw);
      mbar_init(&bars->x_full[t], nw);
    }
    for (int s = 0; s < NK; ++s) mbar_init(&bars->k_full[s], 1), mbar_init(&bars->k_empty[s], 1);
    for (int s = 0; s < NR; ++s) {
      for (int x = 0; x < C::MK; ++x) mbar_init(&bars->raw_full[s][x], !C::kLoader && x + C::MK < kTPages ? 2 : 1);
      mbar_init(&bars->raw_empty[s], C::MK);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&bars->v_full[s], C::MK + (kDirect ? 1 : 0));
      mbar_init(&bars->v_empty[s], 1);
      mbar_init(&bars->v_dir[s], 1);
    }
    for (int s = 0; s < NM; ++s) mbar_init(&bars->meta_full[s], 1);
    for (int s = 0; s < C::NS; ++s) mbar_init(&bars->seg_full[s], 1), mbar_init(&bars->seg_empty[s], 1 + 2 * nw);
    mbar_init(&bars->mma_final, 1);
    bars->abort = 0;
    fence_barrier_init();
#ifdef EKV_TEST_WAIT_TIMEOUT
    if (p.inject_timeout && blockIdx.x == 0) {           // test build only: 16 bytes that no copy delivers
      uint64_t* const waits[] = {&bars->q_full[0], &bars->k_full[1], &bars->v_full[0], &bars->raw_full[1][0], &bars->s_full[0],
                                 &bars->p_full[0], &bars->pv_done[0], &bars->seg_full[0], &bars->meta_full[1]};
      mbar_expect_tx(waits[p.inject_timeout - 1], 16);
    }
#endif
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    if (VM == kXFP16 || VM == kXMixed) tma_prefetch_desc(&tv16);
    if (VM == kXE4M3 || VM == kXMixed) tma_prefetch_desc(&tv8);
  }
  if (warp == 2) tc05::tmem_alloc(&bars->tmem_base, 512);

  // ---- plan: the blocks of all items, in equal ranges (see the top), kT5Threads sequences at a time
  const int tid = threadIdx.x;
  bool fails = false;
  auto cost = [&](int b) -> long long {
    Seq s;
    if (b >= c.batch || !load_seq(e, b, s)) return 0;
    if (seq_ok(e, s)) {
      const Items it = items_of<ALT>(e, s);
      return it.before<ALT>(it.np);
    }
    fails = true;
    return 0;
  };
  auto warp_incl = [&](long long x) {                  // inclusive prefix sum over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += v;
    }
    return x;
  };
  // CTA x works on KV head x mod H_kv and range x / H_kv: the heads of a page are read at about the
  // same time
  const int ranges = (int)gridDim.x / c.Hkv, h = (int)blockIdx.x % c.Hkv;
  const int chunks = (c.batch + kT5Threads - 1) / kT5Threads;
  long long mine = 0, incl = 0, total = 0, carry = 0, per = 0, start = 0;
  int budget0 = 0;
  // the total, and then the sequence of position `start`; one chunk's costs serve both
#pragma unroll 1
  for (int x = 0; x < 2 * chunks; ++x) {
    const int b0 = (x < chunks ? x : x - chunks) * kT5Threads;
    if (x == 0 || chunks > 1) {
      mine = cost(b0 + tid);
      incl = warp_incl(mine);
      if (x > 0) __syncthreads();                        // the last use of red is behind
      if (lane == 31) bars->red[warp] = incl;
      tc05::fence_before_sync();
      const int any_fails = __syncthreads_or(fails && x < chunks);
      tc05::fence_after_sync();
      if (any_fails && blockIdx.x == 0) {                // reported and zeroed once
        for (int b = b0; b < min(b0 + kT5Threads, c.batch); ++b) {
          Seq s;
          if (!load_seq(e, b, s) || seq_ok(e, s)) continue;
          if (tid == 0) report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SEQ_LEN, b);
          zero_rows(e, s);
        }
        fails = false;
      }
    }
    const long long sums = warp_incl(lane < kT5Threads / 32 ? bars->red[lane] : 0);
    const long long before = carry + (warp > 0 ? __shfl_sync(0xffffffffu, sums, warp - 1) : 0);
    carry += __shfl_sync(0xffffffffu, sums, 31);
    if (x < chunks) {
      if (x == chunks - 1) {
        total = carry;
        carry = 0;
        per = total <= INT_MAX ? ((uint32_t)total + ranges - 1u) / (uint32_t)ranges : (total + ranges - 1) / ranges;
        if (per <= kItemCost<ALT>) per = kItemCost<ALT> + 1;
        start = (int)blockIdx.x / c.Hkv < ranges ? per * ((int)blockIdx.x / c.Hkv) : total;
        budget0 = (int)max(0ll, min(per, total - start));
        if (budget0 == 0) break;
      }
      continue;
    }
    const long long at = start - (before + incl - mine);
    if (mine > 0 && at >= 0 && at < mine) {
      bars->st_b = b0 + tid;
      bars->st_off = (int)at;
    }
    if (carry > start) break;
  }
  __syncthreads();
  // (kItemCost + 1 units hold a block, and the last unit of all is one: a range that is not empty has blocks)
  const bool any = budget0 > 0;
  const uint32_t tbase = bars->tmem_base;
  const int TT = e.tile_tokens;                        // tokens of a tile
  const int nqb = ALT ? 2 / nw : 2;                    // query buffers: tiles, or (ALT, few rows) segments in turn
  const int q_slab = (ALT ? 32 * nw : kTRows) * 128, q_buf = NB * q_slab;
  const int h_rows = TT * e.G;

  // (each register split stands at the head of its roles' code)
  if (warp < 4 || warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 0) {
      // ------------------------------------------- producer: page checks, Q, K
      // Pages are looked up in batches of four blocks, a page per lane: a batch's ids are fetched two
      // batches ahead and its modes and scales one ahead, across segments. A block's description is
      // posted kMetaAhead blocks before its keys are loaded, for the makers, whose loads take as long.
      // Its walk is the only one: what the MMA and softmax warps need of a segment is posted in a ring of NS
      // descriptions (a walk of every role's own cost each item 10,000 cycles of cold code). Up to
      // four segments may be posted whose keys are not loaded yet, and a description is free once its
      // readers are through with the segment before: eight always leave the producer its way.
      int u = 0, k = 0;                                  // blocks described, blocks whose keys were loaded
      uint32_t ql[2] = {0u, 0u}, qseg = 0, nseg = 0;
      bool ok = true, ended = false;
      Walk w;
      w.b = 0;
      w.index = w.u = 0;
      w.budget = budget0;
      if (any) {
        w.b = bars->st_b;
        Seq sq;
        load_seq(e, w.b, sq);
        w.q0 = sq.q0;
        w.it = items_of<ALT>(e, sq);
        const int off = bars->st_off;
        int lo = 0, n = w.it.np, before = 0;             // the item: the last that begins at or before `off`
        while (n > 1) {                                  // among n from lo on; 32 are looked at together
          const int step = (n + 31) / 32, at = lo + lane * step;
          const int x = lane * step < n ? w.it.before<ALT>(at) : INT_MAX;
          const int last = __popc(__ballot_sync(0xffffffffu, x <= off)) - 1;
          before = __shfl_sync(0xffffffffu, x, last);
          n = min(step, n - last * step);
          lo += last * step;
        }
        w.i = lo;
        w.j = w.it.jlo(lo) - kItemCost<ALT> + off - before;
      }
      ExtTcSplit split;
      split.n = 0;
      struct Batch {
        int b, j0, nb, lo, hi, qtok, tiles;              // keys [lo, hi); qtok < 0: not a segment's first batch
      };
      Segment sg;
      sg.ja = sg.jb = 0;
      auto next_batch = [&](Batch& x) {
        x.qtok = -1;
        x.tiles = 0;
        x.nb = 0;
        if (sg.ja >= sg.jb) {
          if (ended) return;
          ended = !walk_next<ALT>(e, w, sg);
          if (nseg >= C::NS) ok = wait_warp(&bars->seg_empty[nseg % C::NS], (nseg / C::NS - 1u) & 1u, abort);
          if (!ok) return;
          if (lane == 0) {
            SegMeta& sm = bars->seg[nseg % C::NS];
            sm.n = ended ? 0 : sg.jb - sg.ja;
            sm.nt[0] = sg.nt[0];
            sm.nt[1] = sg.nt[1];
            sm.ja = sg.ja;
            sm.q0 = sg.q0;
            sm.ntok = sg.n;
            sm.t0 = sg.t0;
            sm.i = sg.i;
            sm.slot = sg.whole ? -1 : sg.slot;
            mbar_arrive(&bars->seg_full[nseg % C::NS]);
          }
          __syncwarp();
          ++nseg;
          if (ended) return;
          x.qtok = sg.q0 + C::NQ * sg.i * TT;
          x.tiles = (sg.nt[0] > 0 ? 1 : 0) | (sg.nt[1] > 0 ? 2 : 0);
          if (sg.ja == sg.jlo && sg.jb < sg.jhi) {       // the item goes on in later CTAs
            split.n = 1 + (int)((sg.jhi - sg.jb + per - 1) / per);
            split.first = sg.slot;
            split.b = sg.b;
            split.h = h;
            split.i = sg.i;
          }
        }
        x.b = sg.b;
        x.j0 = sg.ja;
        x.nb = min(32 / kTPages, sg.jb - sg.ja);
        x.lo = sg.lo;
        x.hi = sg.hi;
        sg.ja += x.nb;
      };
      auto in_batch = [&](const Batch& x) {
        const int k0 = x.j0 * kTKeys + lane * kPage;
        return lane < x.nb * kTPages && k0 + kPage > x.lo && k0 < x.hi;
      };
      auto ids = [&](const Batch& x) {
        return in_batch(x) ? __ldg(c.block_table + (size_t)x.b * c.bt_stride + x.j0 * kTPages + lane) : 0;
      };
      auto lookup = [&](const Batch& x, int id, int& mode, float& vs) {
        mode = VM == kXFP16 ? EKV_MODE_TARGET_FP16 : VM == kXE4M3 ? EKV_MODE_COMPACT_E4M3
               : VM == kXMicro ? EKV_MODE_MICRO_FP4 : c.uniform_mode;
        vs = 0.f;
        if (!in_batch(x) || id < 0 || id >= c.num_pages) return;
        if (VM == kXMixed && c.page_mode) mode = (int)__ldg(c.page_mode + id);
        if ((VM == kXE4M3 || VM == kXMixed) && c.v_scales)
          vs = __ldg(c.v_scales + (c.scale_mode == EKV_SCALE_PER_TENSOR ? 0 : (size_t)id * c.Hkv + h));
      };
      // the queries (first block of a segment) and keys of block k
      auto load_k = [&]() {
        const BlockMeta& mt = bars->meta[k % NM];
        if (mt.qtok >= 0) {
          const int tiles = ALT ? 1 << (qseg % nqb) : mt.tiles;
          ++qseg;
          for (int t = 0; t < 2 && ok; ++t) {
            if (!((tiles >> t) & 1)) continue;
            if (ql[t] > 0) ok = wait_warp(&bars->q_empty[t], (ql[t] - 1u) & 1u, abort);
            if (!ok) return;
            if (lane == 0) {
              mbar_arrive_expect_tx(&bars->q_full[t], (uint32_t)(h_rows * D * 2));
              for (int s = 0; s < NB; ++s)
                tma_load_5d(sQ + t * q_buf + s * q_slab, &tq, 0, 0, s, h, mt.qtok + (ALT ? 0 : t * TT), &bars->q_full[t]);
            }
            ++ql[t];
          }
        }
        const int ks = k % NK;
        if (k >= NK) ok = wait_warp(&bars->k_empty[ks], (uint32_t)(k / NK - 1) & 1u, abort);
        if (!ok) return;
        const bool load = lane < kTPages && !(mt.flags[lane & (kTPages - 1)] & kSkip);
        const int n = __popc(__ballot_sync(0xffffffffu, load));
        if (lane == 0) mbar_arrive_expect_tx(&bars->k_full[ks], (uint32_t)n * (kPage * D * 2));
        __syncwarp();
        if (load)
          tma_load_5d(sK + ks * C::IB + lane * (2 * C::GB), &tk, 0, 0, 0, 0, mt.page[lane] * kPage * c.Hkv + h,
                      &bars->k_full[ks]);
        ++k;
      };
      Batch b0, b1, b2;
      int id0 = 0, id1 = 0, id2 = 0, mode0 = 0, mode1 = 0;
      float vs0 = 0.f, vs1 = 0.f;
      b1.nb = b2.nb = 0;
#pragma unroll 1
      for (int round = 0; ok; ++round) {
        b0 = b1;
        id0 = id1;
        mode0 = mode1;
        vs0 = vs1;
        b1 = b2;
        id1 = id2;
        next_batch(b2);                                  // two batches ahead
        id2 = ids(b2);
        lookup(b1, id1, mode1, vs1);
        if (round < 2) continue;
        // this batch's pages
        int flags = kSkip, detail = EKV_DETAIL_NONE;
        float vs = 1.f;
        if (in_batch(b0)) {
          flags = mode0 == EKV_MODE_COMPACT_E4M3 ? kE4 : mode0 == EKV_MODE_BASE ? kBs
                  : mode0 == EKV_MODE_MICRO_FP4 ? kMx : 0;
          if (id0 < 0 || id0 >= c.num_pages) detail = EKV_DETAIL_PAGE_ID;
          else if (mode0 > EKV_MODE_MICRO_FP4) detail = EKV_DETAIL_PAGE_MODE;
          else if ((flags & kE4) && !(PS ? vs0 > 0.f && vs0 <= kScaleMost : scale_ok(vs0))) detail = EKV_DETAIL_SCALE;
          else if (PS && (flags & kE4)) vs = fmaxf(vs0, kScaleLeast);
          if (detail) {
            report_error(c.err, EKV_ERR_DEVICE_CHECK, detail, b0.b);
            flags = kSkip;
          }
        }
        const float lsc = log2f(vs), ivs = 1.f / vs;
        const uint32_t bad = __ballot_sync(0xffffffffu, detail != EKV_DETAIL_NONE);
        const bool end = b0.nb == 0;                     // only the keys of the last blocks are left
#pragma unroll 1
        for (int i = 0; i < (end ? kMetaAhead : b0.nb) && ok; ++i) {
          if (!end) {
            BlockMeta& mt = bars->meta[u % NM];
            const int pg = lane & (kTPages - 1);
            if (lane / kTPages == i) {
              mt.page[pg] = id0;
              mt.flags[pg] = (uint8_t)flags;
              mt.lsc[pg] = lsc;
              mt.ivs[pg] = ivs;
              if (pg == 0) {
                mt.bad = (int)((bad >> (i * kTPages)) & 0xffu);
                mt.qtok = i == 0 ? b0.qtok : -1;
                mt.tiles = (uint8_t)b0.tiles;
                mt.last = i + 1 == b0.nb && b1.nb == 0;
                mt.z0 = (uint8_t)max(0, b0.lo - (b0.j0 + i) * kTKeys);
                mt.z1 = (uint8_t)min(kTKeys, b0.hi - (b0.j0 + i) * kTKeys);
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->meta_full[u % NM]);
            ++u;
          }
          if (end ? k < u : u > kMetaAhead) load_k();
        }
        if (end) break;
      }
      if (!ok && lane == 0) give_up(c.err, abort);
      if (lane == 0) p.split[blockIdx.x] = split;
      // the copies still in flight land before the CTA can exit
#pragma unroll 1
      for (int v = max(0, k - NK); v < k; ++v) drain(&bars->k_full[v % NK], (v / NK) & 1);
      for (int t = 0; t < 2; ++t)
        if (ql[t] > 0) drain(&bars->q_full[t], (ql[t] - 1u) & 1u);
    } else if (kDirect && warp == 3) {
      // ------------------------------------------------ loads of FP16 value pages
      int u = 0;
      uint32_t dir_used = 0, dir_ph = 0;                 // bit s: v_dir[s] has had a phase; parity of its next
      bool ok = any;
      const bool run = ok;
      for (bool last = false; ok && !last; ++u) {
        const int vs = u % NV;
        ok = wait_warp(&bars->meta_full[u % NM], (uint32_t)(u / NM) & 1u, abort);
        if (ok && u >= NV) ok = wait_warp(&bars->v_empty[vs], (uint32_t)(u / NV - 1) & 1u, abort);
        if (!ok) break;
        const BlockMeta& mt = bars->meta[u % NM];
        last = mt.last;
        const int flags = lane < kTPages ? mt.flags[lane] : kSkip;
        const int page = lane < kTPages ? mt.page[lane] : 0;
        // a stage with rows to zero is announced on a barrier of its own; they are zeroed once it has landed
        const bool edge = mt.z0 > 0 || mt.z1 < kTKeys;
        const uint32_t dmask = __ballot_sync(0xffffffffu, flags == 0);
        uint64_t* bar = edge ? &bars->v_dir[vs] : &bars->v_full[vs];
        if (lane == 0) {
          if (edge) mbar_arrive(&bars->v_full[vs]);
          if (!edge || dmask) mbar_arrive_expect_tx(bar, (uint32_t)__popc(dmask) * (kPage * D * 2));
        }
        if (edge && dmask) dir_used |= 1u << vs, dir_ph ^= 1u << vs;
        __syncwarp();
        if (flags == 0)
          tma_load_5d(sV + vs * C::IB + lane * (2 * C::GB), &tv16, 0, 0, 0, 0, page * p.v16_mul + h * p.v16_head, bar);
      }
      if (!ok && run && lane == 0) give_up(c.err, abort);
      if (run)
        for (int v = max(0, u - NV); v < u; ++v) {
          const int s = v % NV;
          if ((dir_used >> s) & 1u) drain(&bars->v_dir[s], ((dir_ph >> s) & 1u) ^ 1u);
          drain(&bars->v_full[s], (uint32_t)(v / NV) & 1u);
        }
    } else if (warp == 1) {
      // ------------------------------------------------------------- MMA issuer
      constexpr uint32_t idS = tc05::idesc_f16_f32(kTRows, kTKeys, false);
      constexpr uint32_t idO = tc05::idesc_f16_f32(kTRows, D, true);
      constexpr uint32_t HIQ = tc05::sdesc_hi(1024), HIB = tc05::sdesc_hi(C::GB);
      const uint32_t q_lo = tc05::sdesc_lo(smem_u32(sQ), 16);
      const uint32_t k_lo = tc05::sdesc_lo(smem_u32(sK), 16);
      const uint32_t v_lo = tc05::sdesc_lo(smem_u32(sV), 1024);     // the next 64 columns lie 1024 B on
      int ks = 0, vst = 0, qbuf = 0;                     // qbuf (ALT): the segment's query buffer
      uint32_t kph = 0, vph = 0;
      uint32_t qc[2] = {0u, 0u}, pc[2] = {0u, 0u}, oc[2] = {0u, 0u};
      auto issue_s = [&](int t) {                        // S_t = Q_t K^T from stage ks
        const uint32_t qa = q_lo + (ALT ? qbuf : t) * (q_buf >> 4), ka = k_lo + ks * (C::IB >> 4);
        const uint32_t d = tbase + t * 256;
        if (tc05::elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc05::mma_ss(d, tc05::sdesc_join(qa + (((k >> 2) * q_slab + (k & 3) * 32) >> 4), HIQ),
                         tc05::sdesc_join(ka + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), HIB), idS, k > 0);
          tc05::commit(&bars->s_full[t]);
        }
        __syncwarp();
      };
      auto commit_one = [&](uint64_t* bar) {
        if (tc05::elect_one()) tc05::commit(bar);
        __syncwarp();
      };
      bool ok = true;
      if (ALT) {
        // Block g of the range belongs to stream g mod 2: O_t += P_t V, and then S_t of block g + 2 over P_t, of the
        // next segment too. js of ns: the segment of S; jp of np: that of the products; nq: lengths between.
        int gs = 0, gp = 0, js = 0, ns = 0, jp = 0, np = 0, nq[3] = {0, 0, 0};
        uint32_t segs = 0, segp = 0;
        bool more = true;
        while (ok) {
          while (more && gs < gp + 2) {
            if (js == ns) {
              ok = wait_warp(&bars->seg_full[segs % C::NS], (segs / C::NS) & 1u, abort);
              if (!ok) break;
              ns = bars->seg[segs % C::NS].n;
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars->seg_empty[segs % C::NS]);
              ++segs;
              js = 0;
              more = ns > 0;
              if (!more) break;
              if (nq[0] == 0) nq[0] = ns;
              else if (nq[1] == 0) nq[1] = ns;
              else nq[2] = ns;
              ok = wait_warp(&bars->q_full[qbuf], qc[qbuf] & 1u, abort);
              ++qc[qbuf];
            }
            if (ok) ok = wait_warp(&bars->k_full[ks], kph, abort);
            if (!ok) break;
            tc05::fence_after_sync();
            issue_s(gs & 1);
            commit_one(&bars->k_empty[ks]);
            if (++ks == NK) ks = 0, kph ^= 1u;
            ++gs;
            if (++js == ns) {
              commit_one(&bars->q_empty[qbuf]);
              if (++qbuf == nqb) qbuf = 0;
            }
          }
          if (!ok || gp == gs) break;
          if (jp == np) {
            np = nq[0];
            nq[0] = nq[1];
            nq[1] = nq[2];
            nq[2] = 0;
            jp = 0;
            // the last segment's O is read out by both streams together
            if (segp > 0) ok = wait_warp(&bars->o_free[0], (segp - 1u) & 1u, abort);
            ++segp;
          }
          const int t = gp & 1;
          if (ok) ok = wait_warp(&bars->v_full[vst], vph, abort);
          if (ok) ok = wait_warp(&bars->p_full[t], pc[t] & 1u, abort);
          ++pc[t];
          if (!ok) break;
          tc05::fence_after_sync();
          const uint32_t va = v_lo + vst * (C::IB >> 4), pa = tbase + t * 256, od = tbase + t * 256 + 128;
          if (tc05::elect_one()) {
#pragma unroll
            for (int k = 0; k < kTKeys / 16; ++k)
              tc05::mma_ts(od, pa + 8 * k, tc05::sdesc_join(va + k * (2 * C::GB >> 4), HIB), idO, jp > 1 || k > 0);
            if (jp + 2 >= np) tc05::commit(&bars->pv_done[t]);
            tc05::commit(&bars->v_empty[vst]);
          }
          __syncwarp();
          if (++vst == NV) vst = 0, vph ^= 1u;
          ++jp;
          ++gp;
        }
      }
      for (uint32_t seg = 0; !ALT && ok; ++seg) {
        ok = wait_warp(&bars->seg_full[seg % C::NS], (seg / C::NS) & 1u, abort);
        if (!ok) break;
        const SegMeta sg = bars->seg[seg % C::NS];
        const int n = sg.n;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_empty[seg % C::NS]);
        if (n == 0) break;
        ok = wait_warp(&bars->k_full[ks], kph, abort);
        for (int t = 0; t < 2 && ok; ++t) {
          if (sg.nt[t] == 0) continue;
          ok = wait_warp(&bars->q_full[t], qc[t] & 1u, abort);
          ++qc[t];
          if (!ok) break;
          tc05::fence_after_sync();
          issue_s(t);
          if (sg.nt[t] == 1) commit_one(&bars->q_empty[t]);
        }
        if (!ok) break;
        commit_one(&bars->k_empty[ks]);
        if (++ks == NK) ks = 0, kph ^= 1u;
        for (int j = 0; ok && j < n; ++j) {
          ok = wait_warp(&bars->v_full[vst], vph, abort);
          if (!ok) break;
          tc05::fence_after_sync();
          const uint32_t va = v_lo + vst * (C::IB >> 4);
          bool k_ready = false;
          for (int t = 0; t < 2 && ok; ++t) {
            if (j >= sg.nt[t]) continue;
            if (j == 0 && oc[t] > 0) ok = wait_warp(&bars->o_free[t], (oc[t] - 1u) & 1u, abort);
            if (ok) ok = wait_warp(&bars->p_full[t], pc[t] & 1u, abort);
            ++pc[t];
            if (!ok) break;
            tc05::fence_after_sync();
            const uint32_t pa = tbase + t * 256, od = tbase + t * 256 + 128;
            if (tc05::elect_one()) {
#pragma unroll
              for (int k = 0; k < kTKeys / 16; ++k)
                tc05::mma_ts(od, pa + 8 * k, tc05::sdesc_join(va + k * (2 * C::GB >> 4), HIB), idO, j > 0 || k > 0);
              if (j + 1 == sg.nt[t]) tc05::commit(&bars->pv_done[t]);
            }
            __syncwarp();
            if (j + 1 < sg.nt[t]) {                      // the next S overwrites P, behind its product
              ok = k_ready || wait_warp(&bars->k_full[ks], kph, abort);
              if (!ok) break;
              k_ready = true;
              tc05::fence_after_sync();
              issue_s(t);
              if (j + 2 == sg.nt[t]) commit_one(&bars->q_empty[t]);
            }
          }
          if (!ok) break;
          if (tc05::elect_one()) {
            tc05::commit(&bars->v_empty[vst]);
            if (j + 1 < n) tc05::commit(&bars->k_empty[ks]);
          }
          __syncwarp();
          if (++vst == NV) vst = 0, vph ^= 1u;
          if (j + 1 < n && ++ks == NK) ks = 0, kph ^= 1u;
        }
        for (int t = 0; t < 2; ++t)
          if (sg.nt[t] > 0) ++oc[t];
      }
      if (!ok && lane == 0) give_up(c.err, abort);
      commit_one(&bars->mma_final);
      if (lane == 0) drain(&bars->mma_final, 0);
    } else if (C::kLoader && warp == 12) {
      // ------------------------------------- raw value pages: a page per lane, a block per stage
      bool ok = any;
      const bool run = ok;
      int v = 0;
      for (bool last = false; ok && !last; ++v) {
        const int rs = v % NR;
        ok = wait_warp(&bars->meta_full[v % NM], (uint32_t)(v / NM) & 1u, abort);
        if (ok && v >= NR) ok = wait_warp(&bars->raw_empty[rs], (uint32_t)(v / NR - 1) & 1u, abort);
        if (!ok) break;
        const BlockMeta& mt = bars->meta[v % NM];
        last = mt.last;
        const int pg = lane & (kTPages - 1), flags = lane < kTPages ? mt.flags[pg] : kSkip;
        const bool mx = VM == kXMicro ? !(flags & kSkip) : VM == kXMixed && (flags & kMx);
        const bool by = flags & (kE4 | kBs);
        const uint32_t bytes = __reduce_add_sync(0xffffffffu, mx ? micro_head_bytes(D) : by ? kPage * D : 0);
        if (lane == 0) mbar_arrive_expect_tx(&bars->raw_full[rs][0], bytes);
        __syncwarp();
        uint8_t* dst = sR + rs * C::RB + pg * (kPage * D);
        if (mx)
          bulk_load(dst, c.v_pages + (size_t)mt.page[pg] * c.v_page_stride + h * micro_head_bytes(D), micro_head_bytes(D),
                    &bars->raw_full[rs][0]);
        else if (by)
          tma_load_4d(dst, &tv8, 0, h, 0, mt.page[pg], &bars->raw_full[rs][0]);
      }
      if (!ok && run && lane == 0) give_up(c.err, abort);
#pragma unroll 1
      for (int x = max(0, v - NR); x < v; ++x) drain(&bars->raw_full[x % NR][0], (uint32_t)(x / NR) & 1u);
    } else if (C::MK == 6 || warp != 12) {
      // ---------------------------- the V stages: pages vi, vi + MK of every block
      // (index: C::MK 6: warps 2, 3, 12-15; 5: 13, 2, 3, 14, 15; 4: 13, 14, 15, 2)
      const int vi = C::MK == 6 ? (warp < 4 ? warp - 2 : warp - 10)
                     : C::MK == 5 ? (warp == 13 ? 0 : warp < 4 ? warp - 1 : warp - 11)
                                  : (warp < 4 ? 3 : warp - 13);
      int issued = 0;
      uint32_t dir_ph = 0;                               // bit s: parity of v_dir[s]'s next phase
      bool ok = any, more = any;                         // more: blocks left to issue
      const bool run = ok;
      const int pg = min(vi + (lane & 1) * C::MK, kTPages - 1);   // lane 0's and lane 1's page
      const bool two = vi + C::MK < kTPages;
      // this warp's raw pages of the next block that has none in flight: a ring of its own
      auto issue = [&]() {
        ok = wait_warp(&bars->meta_full[issued % NM], (uint32_t)(issued / NM) & 1u, abort);
        if (!ok) return;
        const BlockMeta& mt = bars->meta[issued % NM];
        more = !mt.last;
        if (kRaw) {
          const int rs = issued % NR;
          uint64_t* bar = &bars->raw_full[rs][vi];
          // lane 0's page and, where there is one, lane 1's: an arrival and its bytes each
          if (lane < (two ? 2 : 1)) {
            const int flags = mt.flags[pg];
            uint8_t* dst = sR + rs * C::RB + pg * (kPage * D);
            const bool mx = VM == kXMicro ? !(flags & kSkip) : VM == kXMixed && (flags & kMx);
            const bool by = flags & (kE4 | kBs);
            mbar_arrive_expect_tx(bar, mx ? micro_head_bytes(D) : by ? kPage * D : 0);
            if (mx)
              bulk_load(dst, c.v_pages + (size_t)mt.page[pg] * c.v_page_stride + h * micro_head_bytes(D),
                      micro_head_bytes(D), bar);
            else if (by)
              tma_load_4d(dst, &tv8, 0, h, 0, mt.page[pg], bar);
          }
          __syncwarp();
        }
        ++issued;
      };
      // A lane's 16 E4M3 codes of a row become the 16-byte chunks 2 c and 2 c + 1, its 32 microscaled ones chunks
      // 4 c .. 4 c + 3. The lanes are dealt over chunks, rows and slabs such that the eight that store at a
      // time meet eight chunk places (chunk ^ row): rows r, r ^ 1 with four c each, or four rows with two.
      const int c8 = lane & 3, s8 = D == 128 ? (lane >> 3) & 1 : 0;
      const int t8 = D == 128 ? ((lane >> 2) & 1) | ((lane >> 4) << 1) : lane >> 2;
      const int c4 = lane & 1, t4 = D == 128 ? ((lane >> 1) & 3) | ((lane >> 4) << 2) : lane >> 1;
      for (int u = 0; ok && (more || u < issued); ++u) {
        if (!C::kLoader)
          while (ok && more && issued < u + (kRaw ? NR : 1)) issue();
        const int vs = u % NV, rs = u % NR;
        if (ok && kRaw) ok = wait_warp(&bars->raw_full[rs][C::kLoader ? 0 : vi], (uint32_t)(u / NR) & 1u, abort);
        if (ok && u >= NV) ok = wait_warp(&bars->v_empty[vs], (uint32_t)(u / NV - 1) & 1u, abort);
        if (!ok) break;
        const BlockMeta& mt = bars->meta[u % NM];
        if (C::kLoader) more = !mt.last;
        const bool edge = mt.z0 > 0 || mt.z1 < kTKeys;
#pragma unroll 1
        for (int page = vi; page < kTPages; page += C::MK) {
          const int fl = mt.flags[page];
          uint8_t* dv = sV + vs * C::IB + page * (2 * C::GB);
          const uint8_t* src = sR + rs * C::RB + page * (kPage * D);
          if (VM == kXMicro ? !(fl & kSkip) : VM == kXMixed && (fl & kMx)) {
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
              const int t = t4 + x * (1024 / D), r = t & 7, q = 2 * s8 + c4;
              const uint4 codes = *reinterpret_cast<const uint4*>(src + t * (D / 2) + q * 16);
              uint32_t sb = src[micro_scale_off(D) + t * (D / kMicroBlock) + q];
              if (!micro_scale_ok(sb)) {
                if (page * kPage + t >= mt.z0 && page * kPage + t < mt.z1)
                  report_error(c.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SCALE, -1);
                sb = 0;
              }
              const __half2 s2 = micro_scale_h2(sb);
              uint8_t* row = dv + (t >> 3) * C::GB + s8 * 1024 + r * 128;
              *reinterpret_cast<uint4*>(row + ((4 * c4) ^ r) * 16) = micro_decode8(codes.x, s2);
              *reinterpret_cast<uint4*>(row + ((4 * c4 + 1) ^ r) * 16) = micro_decode8(codes.y, s2);
              *reinterpret_cast<uint4*>(row + ((4 * c4 + 2) ^ r) * 16) = micro_decode8(codes.z, s2);
              *reinterpret_cast<uint4*>(row + ((4 * c4 + 3) ^ r) * 16) = micro_decode8(codes.w, s2);
            }
          } else if (kRaw && (fl & (kE4 | kBs))) {
#pragma unroll (VM == kXMixed ? 2 : D / 32)
            for (int x = 0; x < D / 32; ++x) {
              const int t = t8 + x * (512 / D), r = t & 7, ch = 4 * s8 + c8;
              uint4 lo, hi;
              const uint32_t at = D == 128 ? swz128(t * 128 + ch * 16) : swz64(t * 64 + ch * 16);
              const uint4 q = *reinterpret_cast<const uint4*>(src + at);
              if (VM == kXMixed && (fl & kBs)) {
                lo = make_uint4(__byte_perm(q.x, 0u, 0x1404), __byte_perm(q.x, 0u, 0x3424), __byte_perm(q.y, 0u, 0x1404),
                                __byte_perm(q.y, 0u, 0x3424));
                hi = make_uint4(__byte_perm(q.z, 0u, 0x1404), __byte_perm(q.z, 0u, 0x3424), __byte_perm(q.w, 0u, 0x1404),
                                __byte_perm(q.w, 0u, 0x3424));
              } else {
                lo = make_uint4(bits(e4m3x2_to_half2((uint16_t)q.x)), bits(e4m3x2_to_half2((uint16_t)(q.x >> 16))),
                                bits(e4m3x2_to_half2((uint16_t)q.y)), bits(e4m3x2_to_half2((uint16_t)(q.y >> 16))));
                hi = make_uint4(bits(e4m3x2_to_half2((uint16_t)q.z)), bits(e4m3x2_to_half2((uint16_t)(q.z >> 16))),
                                bits(e4m3x2_to_half2((uint16_t)q.w)), bits(e4m3x2_to_half2((uint16_t)(q.w >> 16))));
              }
              uint8_t* row = dv + (t >> 3) * C::GB + s8 * 1024 + r * 128;
              *reinterpret_cast<uint4*>(row + ((2 * c8) ^ r) * 16) = lo;
              *reinterpret_cast<uint4*>(row + ((2 * c8 + 1) ^ r) * 16) = hi;
            }
          }
        }
        if (kDirect && edge && __any_sync(0xffffffffu, lane < kTPages && mt.flags[lane & (kTPages - 1)] == 0)) {
          ok = wait_warp(&bars->v_dir[vs], (dir_ph >> vs) & 1u, abort);
          dir_ph ^= 1u << vs;
          if (!ok) break;
        }
        // keys that no row of the item sees, and pages that were not loaded: zeros, whatever they hold
        const uint32_t smask = __ballot_sync(0xffffffffu, lane < kTPages && (mt.flags[lane & (kTPages - 1)] & kSkip));
        if (edge || smask) {
          __syncwarp();
          for (int page = vi; page < kTPages; page += C::MK)
            for (int x = lane; x < kPage * (D / 8); x += 32) {
              const int key = page * kPage + x / (D / 8), cz = x % (D / 8);
              if (key < mt.z0 || key >= mt.z1 || ((smask >> page) & 1u))
                *reinterpret_cast<uint4*>(sV + vs * C::IB + (key >> 3) * C::GB + (cz >> 3) * 1024 + (key & 7) * 128 +
                                          (cz & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        fence_async();                                   // written for the MMAs; the raw bytes read for their refill
        __syncwarp();
        if (C::kLoader && lane == 0) mbar_arrive(&bars->raw_empty[rs]);
        if (lane == 0) mbar_arrive(&bars->v_full[vs]);
      }
      if (!ok && run && lane == 0) give_up(c.err, abort);
      if (kRaw && !C::kLoader)
#pragma unroll 1
      for (int v = max(0, issued - NR); v < issued; ++v) drain(&bars->raw_full[v % NR][vi], (uint32_t)(v / NR) & 1u);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    if (!ALT || (warp & 3) < nw) {                     // (the others have no rows)
      // ------------------------------------------------------- softmax, tile t
      const int t = (warp - 4) >> 2, r = threadIdx.x - 128 - t * kTRows;
      const uint32_t lanebase = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const float qs = e.qscale;
      const float osc = p.scale_ptr ? __ldg(p.scale_ptr) : 1.f;   // one E4M3 scale for every code
      const uint32_t t_s = tbase + t * 256 + lanebase, t_o = tbase + t * 256 + 128 + lanebase;
      uint32_t sc = 0, pvc = 0, seg = 0;                 // phases: s_full, pv_done; segments
      int u = 0;
      bool ok = true;
      const int tok_t = r / e.G;                         // this thread's token within the tile
      while (ok) {
        // what the rows need of the segment; orow < 0: a row past the sequence
        int nmine, u0 = u, ja, pos, lo, all_lo, all_hi, slot;
        long long orow;
        const uint32_t rs = seg % C::NS;
        ok = wait_warp(&bars->seg_full[rs], (seg / C::NS) & 1u, abort);
        if (!ok) break;
        {
          const SegMeta& sg = bars->seg[rs];
          const int n = sg.n;
          nmine = sg.nt[t];
          ja = sg.ja;
          const int first = (ALT ? sg.i : 2 * sg.i + t) * TT;   // the tile's first token
          const int tok = first + tok_t;
          pos = sg.t0 + tok;
          lo = max(pos - e.window, -1);                  // the row sees keys lo + 1 .. pos
          // keys that every valid row sees: from the last row's window start to the first row's own
          all_lo = sg.t0 + min(first + TT, sg.ntok) - 1 - e.window;
          all_hi = sg.t0 + first;
          slot = sg.slot;
          orow = tok_t < TT && tok < sg.ntok ? (long long)(sg.q0 + tok) * c.Hq + h * e.G + r % e.G : -1;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->seg_empty[rs]);
          if (n == 0) break;
          u += n;
          ++seg;
        }
        const bool valid = orow >= 0, whole = slot < 0;
        float m_ref = -INFINITY, l = 0.f;
        bool bad = false;
        for (int jj = 0; jj < nmine; ++jj) {
          const int blk = ALT ? 2 * jj + (t ^ (u0 & 1)) : jj;   // block of the segment
          ok = wait_warp(&bars->meta_full[(u0 + blk) % NM], (uint32_t)((u0 + blk) / NM) & 1u, abort);
          if (ok) ok = wait_warp(&bars->s_full[t], sc & 1u, abort);
          ++sc;
          if (!ok) break;
          tc05::fence_after_sync();
          const BlockMeta& mt = bars->meta[(u0 + blk) % NM];
          const int k0 = (ja + blk) * kTKeys;
          const int badp = mt.bad;
          const bool masked = k0 + kTKeys - 1 > all_hi || k0 <= all_lo || badp;
          const int hi_c = pos - k0, lo_c = lo - k0;
          if (badp) {
            for (int pg = 0; pg < kTPages; ++pg)
              if (((badp >> pg) & 1) && pg * kPage <= hi_c && pg * kPage + kPage - 1 > lo_c) bad = true;
          }
          // The row's maximum, in log2 units. NH 1: the row stays in registers. NH 4: a quarter of it at a time, read
          // again for the weights (and written back where masked), for a quarter of the code: the loops of
          // a CTA's roles share one instruction cache, and where the makers' loop is the long one (mixed
          // pages) or each softmax warp runs alone (ALT) that counts for more than the second read.
          // NH 1 / 2 / 4: a token behind 8K keys (32 sequences) 152 / 146 / 144 us, 48 x 5 tokens over mixed
          // pages 166 / 151 / 147 us, mixed chunks under a window 146 / 136 / 135 us, 4,096 tokens behind 16K of E4M3
          // 844 / 852 / 936 us.
          constexpr int NH = ALT || VM == kXMixed ? 4 : 1, NC = 4 / NH;
          uint32_t a[NC][32];
          float mx = -INFINITY;
#pragma unroll 1
          for (int hf = 0; hf < NH; ++hf) {
#pragma unroll
            for (int c4 = 0; c4 < NC; ++c4) tc05::ld32(t_s + 32 * (NC * hf + c4), a[c4]);
            tc05::wait_ld();
            if (masked) {
              const int lc = lo_c - 32 * NC * hf;        // keys lc + 1 .. lc + seen of these
              const uint32_t seen = (uint32_t)max(hi_c - lo_c, 0);
#pragma unroll
              for (int c4 = 0; c4 < NC; ++c4)
#pragma unroll
                for (int x = 0; x < 32; ++x)
                  if ((uint32_t)(32 * c4 + x - lc - 1) >= seen) a[c4][x] = __float_as_uint(-INFINITY);
              if (NH > 1) {
#pragma unroll
                for (int c4 = 0; c4 < NC; ++c4) tc05::st32(t_s + 32 * (NC * hf + c4), a[c4]);
                tc05::wait_st();
              }
            }
#pragma unroll
            for (int c4 = 0; c4 < NC; ++c4) {
              float m8[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t* y = a[c4] + 8 * q;
                m8[q] = fmaxf(max3(max3(__uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2])),
                                   __uint_as_float(y[3]), __uint_as_float(y[4])),
                              max3(__uint_as_float(y[5]), __uint_as_float(y[6]), __uint_as_float(y[7])));
              }
              if (PS) {
                const float* lsc = mt.lsc + 2 * (NC * hf + c4);
                mx = max3(mx, fmaf(fmaxf(m8[0], m8[1]), qs, lsc[0]), fmaf(fmaxf(m8[2], m8[3]), qs, lsc[1]));
              } else {
                mx = max3(mx, max3(m8[0], m8[1], m8[2]), m8[3]);
              }
            }
          }
          mx = PS ? mx - kHeadroom : fmaf(mx, qs, -kHeadroom);
          const float m_new = fmaxf(m_ref, mx);
          const bool need = m_new > m_ref + 8.f;
          if (__any_sync(0xffffffffu, need)) {
            const float alpha = need ? ex2(m_ref - m_new) : 1.f;
            if (jj > 0) {
#pragma unroll 1
              for (int x = 0; x < D / 16; ++x) {
                uint32_t o[16];
                tld16(t_o + 16 * x, o);
                tc05::wait_ld();
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * alpha);
                tst16(t_o + 16 * x, o);
              }
            }
            l *= alpha;
            if (need) m_ref = m_new;
          }
          // a row that has seen no key yet keeps m = -inf: its weights are 2^-inf = 0
          const float nm = m_ref == -INFINITY ? 0.f : -m_ref;
          // (P's columns 16 c .. of chunk c lie over S columns that have been read by then)
#pragma unroll 1
          for (int hf = 0; hf < NH; ++hf) {
            if (NH > 1) {
#pragma unroll
              for (int c4 = 0; c4 < NC; ++c4) tc05::ld32(t_s + 32 * (NC * hf + c4), a[c4]);
              tc05::wait_ld();
            }
#pragma unroll
            for (int c4 = 0; c4 < NC; ++c4) {
#pragma unroll
              for (int pg = 0; pg < 2; ++pg) {
                const float add = PS ? nm + mt.lsc[2 * (NC * hf + c4) + pg] : nm;
                float la[2] = {0.f, 0.f}, lb[2] = {0.f, 0.f};
#pragma unroll
                for (int x = 8 * pg; x < 8 * pg + 8; ++x) {
                  float a0, a1;
                  ffma2(a0, a1, __uint_as_float(a[c4][2 * x]), __uint_as_float(a[c4][2 * x + 1]), qs, add);
                  const float p0 = ex2(a0), p1 = ex2(a1);
                  fadd2(la[x & 1], lb[x & 1], p0, p1);
                  a[c4][x] = pack2(p0, p1);
                }
                fadd2(la[0], lb[0], la[1], lb[1]);
                l = PS ? fmaf(la[0] + lb[0], mt.ivs[2 * (NC * hf + c4) + pg], l) : l + (la[0] + lb[0]);
              }
              tst16(t_s + 16 * (NC * hf + c4), &a[c4][0]);
            }
          }
          tc05::wait_st();
          tc05::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_full[t]);
        }
        if (!ok) break;
        const size_t prow = (size_t)max(slot, 0) * (2 * kTRows) + (ALT ? 0 : t) * kTRows + r;
        if (ALT) {
          // join the streams: each posts (m, l) and reads the other's, and takes half of the columns of
          // both O, which lie in its own tensor-memory lanes
          if (nmine > 0) {
            ok = wait_warp(&bars->pv_done[t], pvc & 1u, abort);
            ++pvc;
            if (!ok) break;
          }
          // the other stream has read what the last segment posted (it arrived here afterwards)
          if (seg > 1) ok = wait_warp(&bars->o_free[0], seg & 1u, abort);
          if (!ok) break;
          float2 (&xch)[2][ALT ? kAltRows : 1] = bars->xch;
          xch[t][r] = make_float2(m_ref, bad ? kBadRecord : l);
          tc05::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->x_full[t]);
          ok = wait_warp(&bars->x_full[1 - t], (seg - 1u) & 1u, abort);
          if (!ok) break;
          tc05::fence_after_sync();
          const float2 other = xch[1 - t][r];
          bad = bad || other.y < 0.f;
          const float M = fmaxf(m_ref, other.x);
          float w0 = l != 0.f ? ex2(m_ref - M) : 0.f, w1 = other.y != 0.f ? ex2(other.x - M) : 0.f;
          const float L = fmaf(l, w0, other.y * w1);     // (of no use where bad)
          if (t == 1) {                                  // w0 weighs stream 0
            const float x = w0;
            w0 = w1;
            w1 = x;
          }
          const bool none = bad || L == 0.f;             // (a NaN goes on to the output)
          const float inv = none ? 0.f : osc / L;
#pragma unroll 1
          for (int x = 0; x < D / 64; ++x) {
            const int col = t * (D / 2) + 32 * x;
            uint32_t o0[32], o1[32];
            tc05::ld32(tbase + 128 + lanebase + col, o0);
            tc05::ld32(tbase + 384 + lanebase + col, o1);
            tc05::wait_ld();
            if (x == D / 64 - 1) {
              tc05::fence_before_sync();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars->o_free[0]);
            }
#pragma unroll
            for (int y = 0; y < 32; ++y) {               // (a stream without blocks left no O: weight 0)
              const float a0 = w0 > 0.f ? __uint_as_float(o0[y]) * w0 : 0.f;
              o0[y] = __float_as_uint(w1 > 0.f ? fmaf(__uint_as_float(o1[y]), w1, a0) : a0);
            }
            if (valid && whole) {
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                uint4 q;
                q.x = pack2(__uint_as_float(o0[8 * y + 0]) * inv, __uint_as_float(o0[8 * y + 1]) * inv);
                q.y = pack2(__uint_as_float(o0[8 * y + 2]) * inv, __uint_as_float(o0[8 * y + 3]) * inv);
                q.z = pack2(__uint_as_float(o0[8 * y + 4]) * inv, __uint_as_float(o0[8 * y + 5]) * inv);
                q.w = pack2(__uint_as_float(o0[8 * y + 6]) * inv, __uint_as_float(o0[8 * y + 7]) * inv);
                if (none) q = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4*>(e.out + orow * D + col + 8 * y) = q;
              }
            } else if (valid) {
#pragma unroll
              for (int y = 0; y < 8; ++y)
                *reinterpret_cast<uint4*>(p.part_acc + prow * D + col + 4 * y) =
                    make_uint4(o0[4 * y], o0[4 * y + 1], o0[4 * y + 2], o0[4 * y + 3]);
            }
          }
          if (valid && t == 0) {
            if (!whole) p.part_ml[prow] = make_float2(M, bad ? kBadRecord : L);
            else if (e.lse) e.lse[orow] = none ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
          }
          continue;
        }
        if (nmine == 0) {
          if (!whole && valid) p.part_ml[prow] = make_float2(-INFINITY, 0.f);
          continue;
        }
        ok = wait_warp(&bars->pv_done[t], pvc & 1u, abort);
        ++pvc;
        if (!ok) break;
        tc05::fence_after_sync();
        const bool none = bad || l == 0.f;               // (a NaN goes on to the output)
        const float inv = none ? 0.f : osc / l;
#pragma unroll 1
        for (int x = 0; x < D / 32; ++x) {
          uint32_t o[32];
          tc05::ld32(t_o + 32 * x, o);
          tc05::wait_ld();
          if (x == D / 32 - 1) {                         // O is read out: the next item may overwrite it
            tc05::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->o_free[t]);
          }
          if (valid && whole) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint4 q;
              q.x = pack2(__uint_as_float(o[8 * y + 0]) * inv, __uint_as_float(o[8 * y + 1]) * inv);
              q.y = pack2(__uint_as_float(o[8 * y + 2]) * inv, __uint_as_float(o[8 * y + 3]) * inv);
              q.z = pack2(__uint_as_float(o[8 * y + 4]) * inv, __uint_as_float(o[8 * y + 5]) * inv);
              q.w = pack2(__uint_as_float(o[8 * y + 6]) * inv, __uint_as_float(o[8 * y + 7]) * inv);
              if (none) q = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(e.out + orow * D + 32 * x + 8 * y) = q;
            }
          } else if (valid) {
#pragma unroll
            for (int y = 0; y < 8; ++y)
              *reinterpret_cast<uint4*>(p.part_acc + prow * D + 32 * x + 4 * y) =
                  make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
          }
        }
        if (valid) {
          if (!whole) p.part_ml[prow] = make_float2(m_ref, bad ? kBadRecord : l);
          else if (e.lse) e.lse[orow] = none ? -INFINITY : (m_ref + log2f(l)) * 0.69314718055994531f;
        }
      }
      if (!ok && lane == 0) give_up(c.err, abort);
    }
  }
  tc05::fence_before_sync();
  __syncthreads();
  if (warp == 2) {
    tc05::fence_after_sync();
    tc05::tmem_free(tbase, 512);
  }
}

// Joins the items that crossed CTAs: block (x, y) takes rows 32 y .. 32 y + 31 of the item that
// begins in CTA x and ends in a later one, eight threads a row with D / 8 columns each, in the order of its
// blocks; the loads are independent of the running maximum. Its blocks are dispatched as the last CTAs of the
// attention leave: dispatched at its start they took 2-4 us from it. (Joined by the last of an item's
// CTAs instead, behind a ticket, chunks took 40 us longer: one CTA per item is too few loads in flight.)
//   M = max m_i,  L = sum l_i 2^(m_i - M),  out = sum acc_i 2^(m_i - M) / L
template <int D, bool ALT>
__global__ void __launch_bounds__(256)
extend_join_kernel(const ExtTcParams p) {
  griddep_wait();
  const ExtTcSplit s = p.split[blockIdx.x];
  if (s.n == 0) return;
  const ExtendParams& e = p.e;
  constexpr int C = D / 8;
  const int row = blockIdx.y * 32 + (threadIdx.x >> 3), c0 = (threadIdx.x & 7) * 4;
  const int TT = e.tile_tokens, t = row / kTRows, r = row % kTRows;
  const int q0 = __ldg(e.c.cu_q + s.b), n = __ldg(e.c.cu_q + s.b + 1) - q0;
  const int tok = (ALT ? s.i : 2 * s.i + t) * TT + r / e.G;
  if (r >= TT * e.G || tok >= n) return;
  auto at = [&](int i) { return (size_t)(i == 0 ? s.first : 2 * ((int)blockIdx.x + i * e.c.Hkv)) * (2 * kTRows) + row; };
  float M = -INFINITY, L = 0.f, acc[C];
  bool bad = false;
#pragma unroll
  for (int y = 0; y < C; ++y) acc[y] = 0.f;
#pragma unroll 2
  for (int i = 0; i < s.n; ++i) {
    const float2 ml = p.part_ml[at(i)];
    const float4* src = reinterpret_cast<const float4*>(p.part_acc + at(i) * D + c0);
    float4 v[C / 4];
#pragma unroll
    for (int y = 0; y < C / 4; ++y) v[y] = src[8 * y];
    bad |= ml.y < 0.f;
    if (ml.y == 0.f) continue;                         // (a record without keys holds no sums)
    const float m = fmaxf(M, ml.x), a = L == 0.f ? 0.f : exp2f(M - m), w = exp2f(ml.x - m);
    M = m;
    L = fmaf(L, a, ml.y * w);
#pragma unroll
    for (int y = 0; y < C / 4; ++y) {
      acc[4 * y] = fmaf(acc[4 * y], a, v[y].x * w);
      acc[4 * y + 1] = fmaf(acc[4 * y + 1], a, v[y].y * w);
      acc[4 * y + 2] = fmaf(acc[4 * y + 2], a, v[y].z * w);
      acc[4 * y + 3] = fmaf(acc[4 * y + 3], a, v[y].w * w);
    }
  }
  const size_t o = (size_t)(q0 + tok) * e.c.Hq + s.h * e.G + r % e.G;
  const bool none = bad || L == 0.f;
  const float inv = none ? 0.f : (p.scale_ptr ? __ldg(p.scale_ptr) : 1.f) / L;
#pragma unroll
  for (int y = 0; y < C / 4; ++y) {
    uint2 q = make_uint2(xt::pack2(acc[4 * y] * inv, acc[4 * y + 1] * inv),
                         xt::pack2(acc[4 * y + 2] * inv, acc[4 * y + 3] * inv));
    if (none) q = make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(e.out + o * D + c0 + 32 * y) = q;
  }
  if (c0 == 0 && e.lse) e.lse[o] = none ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------------- host
// FP16 page slices of one KV head as 8-token groups: 5-D view (d mod 64, t mod 8, d / 64, t / 8, place) of
// an fp16 pool, `place` counting `unit` bytes, so that one coordinate names page and head; the
// box {64, 8, D / 64, 2, 1} lands as [2][D / 64][8][128 B].
inline bool encode_group_map(CUtensorMap* tm, const void* base, int D, int Hkv, unsigned long long places, int unit) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t row = (cuuint64_t)Hkv * D * 2;
  cuuint64_t dims[5] = {64, 8, (cuuint64_t)(D / 64), 2, (cuuint64_t)places};
  cuuint64_t strides[4] = {row, 128, 8 * row, (cuuint64_t)unit};
  cuuint32_t box[5] = {64, 8, (cuuint32_t)(D / 64), 2, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows: 5-D view (d mod 64, g, d / 64, KV head, token) of q [T][Hq][D], `stride` values between tokens; the
// box {64, G, 1, 1, TT} lands TT * G rows of 128 B, row = token * G + g. Tokens past T read as zeros.
inline bool encode_query_map(CUtensorMap* tm, const void* q, int D, int Hkv, int G, int T, int tile_tokens, long long stride) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[5] = {64, (cuuint64_t)G, (cuuint64_t)(D / 64), (cuuint64_t)Hkv, (cuuint64_t)T};
  cuuint64_t strides[4] = {(cuuint64_t)D * 2, 128, (cuuint64_t)G * D * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[5] = {64, (cuuint32_t)G, 1, 1, (cuuint32_t)tile_tokens};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void*>(q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct ExtTcMaps {
  CUtensorMap q, k, v16, v8;
};

template <int D, int VM, bool PS, bool ALT>
cudaError_t launch_ext_tc(const ExtTcMaps& m, const ExtTcParams& p, int grid, cudaStream_t st) {
  auto kern = extend_tc05_kernel<D, VM, PS, ALT>;
  constexpr int smem = xt_smem_bytes<D, VM, ALT>();
  static_assert(smem <= 232448, "shared memory of one CTA");
  cudaError_t err = set_smem_attr(reinterpret_cast<const void*>(kern), smem);
  if (err != cudaSuccess) return err;
  kern<<<grid, kT5Threads, smem, st>>>(m.q, m.k, m.v16, m.v8, p);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, ALT ? p.nw : 2 * kTRows / 32);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, extend_join_kernel<D, ALT>, p);
}

template <int D, bool ALT>
cudaError_t launch_ext_tc_alt(const ExtTcMaps& m, const ExtTcParams& p, int vm, int grid, cudaStream_t st) {
  switch (vm) {
    case kXFP16: return launch_ext_tc<D, kXFP16, false, ALT>(m, p, grid, st);
    case kXE4M3:
      return p.scale_ptr ? launch_ext_tc<D, kXE4M3, false, ALT>(m, p, grid, st)
                         : launch_ext_tc<D, kXE4M3, true, ALT>(m, p, grid, st);
    case kXMicro: return launch_ext_tc<D, kXMicro, false, ALT>(m, p, grid, st);
    default: return launch_ext_tc<D, kXMixed, true, ALT>(m, p, grid, st);
  }
}

template <int D>
cudaError_t launch_ext_tc_d(const ExtTcMaps& m, const ExtTcParams& p, int vm, int grid, cudaStream_t st) {
  return p.nw > 0 ? launch_ext_tc_alt<D, true>(m, p, vm, grid, st) : launch_ext_tc_alt<D, false>(m, p, vm, grid, st);
}

}  // namespace ekv
