// prompt_tc05.cu -- causal attention of packed prompts, straight from the rows of the projection, on the
// fifth-generation tensor cores.
//
// For a prompt of rows row0 .. row0 + L - 1, query position s and query head hq of KV head h:
//   out = sum_k softmax_k(sm_scale q_s . k_k) v_k over max(0, s - window + 1) <= k <= s.
// 4 D FLOP a visible pair and head against 2 D bytes of a row of q, k, v or out: prompts of some hundred tokens
// are bound by HBM, longer ones by the tensor pipe, with the exponentials next.
//   * tiles: 128 query rows (the MMA's M), `heads` query heads of a KV head times 128 / heads tokens, row = token *
//     heads + head. heads = 1 takes 128 tokens of one head; heads = G fills a tile with short prompts.
//   * items: two tiles that follow each other and share every key block of 128 tokens, one tile's softmax under the
//     other's products. Persistent CTAs, one a SM.
//   * plan: the items of all prompts, heaviest first (short prompts in their order). An item's weight goes by its query block,
//     so the prompts are sorted by their number of query blocks (in shared memory, by every CTA for itself), and item x of the
//     list is found by a search over the places where a prompt joins in. The list is dealt in a snake, which balances a
//     sorted list about as well as a queue does, without one. Empty blocks of short prompts are not in it.
//     Prompts of one token, 4/2 heads of 64, and with a first one of 300, so that they are sorted: 1 prompt 9.3 / 11.3 us,
//     32 10.9 / 13.3, 256 19.1 / 23.0, 1,024 52 / 61, 4,096 195 / 224.
//   * roles: warp 0 loads queries, keys and values (TMA); warp 1 issues the MMAs; warp 2 owns tensor memory and posts the
//     items' descriptions up to four ahead (looked up by every role for itself, an item cost each 1,000 cycles); warp 3
//     zeroes the value rows past a prompt's end in its last block, so that weight 0 never meets what the next prompt
//     (or nobody) wrote there; warps 4-7 and 8-11 are the softmax of tile 0 and 1, a thread per row.
// Tensor memory of tile t: S and P at 256 t, O at 256 t + 128. The order of the MMAs and the lazily moved maximum are those
// of the prefill (prefill_tc05.cu); the reference of a row lies 2^kHeadroom below its maximum, so that fp16 weights keep
// their bits down to 2^-21 of the largest (extend_tc05.cuh). Every wait is bounded; a timeout is reported and
// every role winds down.
// What the steps towards this form gave (200 prompts of 1-300 tokens, 32/4 heads / 16 of 100-4,096, 32/8 heads, us): first
// form 207 / 461; registers split between the roles, no spills 193 / 449; descriptions, queries behind the first keys and results
// in whole 32-byte sectors 158 / 426; one elected region a step, descriptors outside it 158 / 418; masks tested bit by
// bit of one register instead of by compares, a quarter of the epilogue's code 154 / 408; the next item looked at early
// 147 / 408. Dropped: queries prefetched to L2 (166 / 432: TMA's rate, not DRAM, sets their 4,600 cycles), chunks of 32 keys
// that no row sees left out (152 / 414: the branches cost the full blocks more), the same with fewer MMA steps (156 / 434),
// items drawn from a counter (154 / 416).
#include "extend_tc05.cuh"
#include "prompt.cuh"

namespace ekv {

namespace {

using namespace xt;

constexpr int kPThreads = 384;
constexpr int kInOrderTokens = 256;                    // longest prompt of a batch that keeps its order (see make_plan)

template <int D>
struct PT {
  static constexpr int NB = D / 64;                    // 64-value slabs of a row
  static constexpr int QB = kTRows * D * 2;            // bytes of a query tile
  static constexpr int IB = kTKeys * D * 2;            // bytes of a K or V block
  static constexpr int NS = D == 128 ? 4 : 8;          // ring stages
};

constexpr int kItems = 4;                                 // descriptions of items
constexpr int kItemReaders = 3 + 2 * kTRows / 32;        // warps that read one: loads, zeros, MMAs and softmax

// One work item: two tiles of one prompt and `heads` query heads.
struct PromptItem {
  int row0, L, hg;         // the prompt's first row, its tokens; the group of heads
  int q0[2];               // [tile] first token
  int ja[2], jb[2];        // [tile] key blocks [ja, jb); none where the tile has no token
  int jlo, jhi;            // of either; jlo < 0: no item follows
};

template <int NS>
struct PromptBars {
  uint64_t q_full[2];            // [tile]: the tile's query rows of its next item landed
  uint64_t q_empty[2];           // [tile]: an item's last S has read the tile's query rows
  uint64_t kv_full[NS];          // a block landed (a prompt's last value block: and its end zeroed)
  uint64_t kv_empty[NS];         // the MMAs reading the stage have completed
  uint64_t v_raw[NS];            // a prompt's last value block landed
  uint64_t s_full[2];            // [tile]: S of the next block written
  uint64_t p_full[2];            // [tile]: P written, S read (one arrival per softmax warp)
  uint64_t pv_done[2];           // [tile]: an item's last O += P V completed
  uint64_t o_free[2];            // [tile]: an item's O read out (one arrival per softmax warp)
  uint64_t mma_final;            // every MMA issued has completed
  uint64_t item_full[kItems], item_empty[kItems];   // a description posted; read by its readers
  PromptItem item[kItems];
  int red[kPThreads / 32];
  uint32_t tmem_base;
  int abort;
};

// The plan, in shared memory: prompts as (query blocks << 12) | (4095 - prompt), and the places in the list of (prompt, query
// block) pairs. Sorted by falling number of blocks: from first[k - 1] on k prompts take part, a block each in turn.
// In the order of memory: prompt k's pairs begin at first[k].
struct alignas(16) Plan {
  uint32_t key[kMaxBatch];
  int first[kMaxBatch];
  int sorted;
};

template <int D>
constexpr int prompt_smem_bytes() {
  return 2 * PT<D>::QB + PT<D>::NS * PT<D>::IB + (int)sizeof(Plan) + (int)sizeof(PromptBars<PT<D>::NS>);
}

// Fills the plan; returns the number of (prompt, query block) pairs. All threads.
__device__ __forceinline__ int make_plan(const PromptParams& p, Plan& pl, int* red) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int step = 2 * p.tile_tokens;
  int n2 = 1, longest = 0;
  while (n2 < p.n) n2 <<= 1;
  for (int i = tid; i < n2; i += kPThreads) {
    uint32_t key = 0;
    if (i < p.n) {
      const int a = __ldg(p.cu + i), b = __ldg(p.cu + i + 1);
      const bool good = a >= 0 && b >= a && b <= p.total;
      if (!good && blockIdx.x == 0) report_error(p.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SEQ_LEN, i);
      const int blocks = good ? (b - a + step - 1) / step : 0;
      key = ((uint32_t)blocks << 12) | (uint32_t)(kMaxBatch - 1 - i);
      longest = max(longest, blocks);
    }
    pl.key[i] = key;
  }
  // Short prompts, all of about one weight, keep their order: the rows past a prompt's end that a tile loads are then the
  // next one's, wanted at about the same time, and not read from memory twice. 32/4 heads, sorted / in order: 200 prompts of 200 to
  // 256 tokens 209 / 188 us, 256 of 1 to 64 65.5 / 61.5; up to 512 tokens weights differ too much (16 of 1 to 512 37 / 41).
  const bool sorted = __syncthreads_or(longest * step > kInOrderTokens);
  for (int size = 2; sorted && size <= n2; size <<= 1)     // bitonic, falling
    for (int d = size >> 1; d > 0; d >>= 1) {
      for (int x = tid; x < n2 / 2; x += kPThreads) {
        const int i = ((x & ~(d - 1)) << 1) | (x & (d - 1)), j = i | d;
        const uint32_t a = pl.key[i], b = pl.key[j];
        if ((a < b) == ((i & size) == 0)) {
          pl.key[i] = b;
          pl.key[j] = a;
        }
      }
      __syncthreads();
    }
  // sorted: first[k - 1] = (blocks of the k first prompts) - k * (blocks of the k-th)
  const int each = (p.n + kPThreads - 1) / kPThreads, k0 = tid * each, k1 = min(k0 + each, p.n);
  int sum = 0;
  for (int k = k0; k < k1; ++k) sum += (int)(pl.key[k] >> 12);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) red[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < kPThreads / 32; ++w) {
    if (w < warp) before += red[w];
    total += red[w];
  }
  before += incl - sum;
  for (int k = k0; k < k1; ++k) {
    const int blocks = (int)(pl.key[k] >> 12);
    pl.first[k] = sorted ? before - k * blocks : before;
    before += blocks;
  }
  if (tid == 0) pl.sorted = sorted;
  __syncthreads();
  // prompts one behind the other have at most so many; lengths that go up and down may claim rows many times over
  if (total <= p.total / step + p.n) return total;
  if (blockIdx.x == 0 && tid == 0) report_error(p.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_SEQ_LEN, -1);
  return 0;
}

// Item w of the list (the whole warp).
__device__ __forceinline__ PromptItem prompt_item(const PromptParams& p, const Plan& pl, int w) {
  const int lane = threadIdx.x & 31, groups = p.Hq / p.heads;
  const int x = w / groups;
  PromptItem it;
  it.hg = w % groups;
  int lo = 0, n = p.n;                                     // the last k with first[k] <= x, of n from lo on
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool in = lane * step < n && pl.first[lo + lane * step] <= x;
    const int last = __popc(__ballot_sync(0xffffffffu, in)) - 1;
    lo += last * step;
    n = min(step, n - last * step);
  }
  const int off = x - pl.first[lo], turn = pl.sorted ? lo + 1 : 1;   // prompts that take part here
  const int qb = (int)(pl.key[lo] >> 12) - 1 - off / turn;
  const int i = kMaxBatch - 1 - (int)(pl.key[pl.sorted ? off % turn : lo] & 4095u);
  it.row0 = __ldg(p.cu + i);
  it.L = __ldg(p.cu + i + 1) - it.row0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.q0[t] = (2 * qb + t) * p.tile_tokens;
    const bool active = it.q0[t] < it.L;
    it.ja[t] = active && it.q0[t] >= p.window ? (it.q0[t] - p.window + 1) / kTKeys : 0;
    it.jb[t] = active ? (min(it.q0[t] + p.tile_tokens, it.L) + kTKeys - 1) / kTKeys : 0;
  }
  it.jlo = it.ja[0];
  it.jhi = max(it.jb[0], it.jb[1]);
  return it;
}

// The next item, as posted by warp 2, for a reader's warp; false: none follows, or a wait gave up (ok).
template <int NS>
__device__ __forceinline__ bool next_item(PromptBars<NS>* bars, int r, PromptItem& it, bool& ok) {
  const int s = r % kItems;
  ok = wait_warp(&bars->item_full[s], (uint32_t)(r / kItems) & 1u, &bars->abort);
  if (!ok) return false;
  it = bars->item[s];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&bars->item_empty[s]);
  return it.jlo >= 0;
}

// The r-th item of this CTA: dealt in rounds of gridDim.x, alternately forwards and backwards.
__device__ __forceinline__ int dealt(int r) {
  const int g = (int)gridDim.x, c = (int)blockIdx.x;
  return r * g + ((r & 1) ? g - 1 - c : c);
}

// The maximum of 32 scores.
__device__ __forceinline__ float max32(const uint32_t (&a)[32]) {
  float m8[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t* y = a + 8 * g;
    m8[g] = fmaxf(max3(max3(__uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2])), __uint_as_float(y[3]),
                       __uint_as_float(y[4])),
                  max3(__uint_as_float(y[5]), __uint_as_float(y[6]), __uint_as_float(y[7])));
  }
  return max3(m8[0], m8[1], fmaxf(m8[2], m8[3]));
}

// The S row of one key block, read from tensor memory into registers once; MASK: columns outside lc + 1 .. hc become
// -inf. Returns the row's maximum (raw score).
template <bool MASK>
__device__ __forceinline__ float prompt_row(uint32_t t_s, int lc, int hc, uint32_t (&a)[4][32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) tc05::ld32(t_s + 32 * c, a[c]);
  tc05::wait_ld();
  float mg[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (MASK) {                                            // a bit per column: 32 tests of one register
      const int h = hc - 32 * c, l = lc - 32 * c;
      const uint32_t upto = h >= 31 ? ~0u : h < 0 ? 0u : (2u << h) - 1u, below = l >= 31 ? ~0u : l < 0 ? 0u : (2u << l) - 1u;
      const uint32_t seen = upto & ~below;
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (!((seen >> e) & 1u)) a[c][e] = __float_as_uint(-INFINITY);
    }
    mg[c] = max32(a[c]);
  }
  return max3(mg[0], mg[1], fmaxf(mg[2], mg[3]));
}

// P = 2^(S qs + nm) of the row in registers, as fp16 pairs over the first 64 columns of S (read by then);
// returns the sum of the fp32 exponentials.
__device__ __forceinline__ float prompt_weights(uint32_t t_s, float qs, float nm, uint32_t (&a)[4][32]) {
  float la[4] = {0.f, 0.f, 0.f, 0.f}, lb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float a0, a1;
      ffma2(a0, a1, __uint_as_float(a[c][2 * e]), __uint_as_float(a[c][2 * e + 1]), qs, nm);
      const float p0 = ex2(a0), p1 = ex2(a1);
      fadd2(la[e & 3], lb[e & 3], p0, p1);
      a[c][e] = pack2(p0, p1);                             // (a[c][2 e] and a[c][2 e + 1] are read)
    }
    tst16(t_s + 16 * c, &a[c][0]);
  }
  fadd2(la[0], lb[0], la[2], lb[2]);
  fadd2(la[1], lb[1], la[3], lb[3]);
  return (la[0] + la[1]) + (lb[0] + lb[1]);
}

// 32 bytes to a 32-byte aligned place.
__device__ __forceinline__ void store32(void* dst, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kPThreads, 1)
prompt_tc05_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, const PromptParams p) {
  using C = PT<D>;
  constexpr int NS = C::NS, NB = C::NB;
  extern __shared__ __align__(1024) uint8_t sm_1k[];
  uint8_t* sQ = sm_1k;                                     // [2][NB][128 rows][128 B]
  uint8_t* sKV = sQ + 2 * C::QB;                           // [NS][NB][128 rows][128 B]
  Plan& pl = *reinterpret_cast<Plan*>(sKV + NS * C::IB);
  PromptBars<NS>* bars = reinterpret_cast<PromptBars<NS>*>(sKV + NS * C::IB + sizeof(Plan));
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_u32(sm_1k) & 1023u) {                           // the swizzled layouts would not hold
    if (threadIdx.x == 0) report_error(p.err, EKV_ERR_DEVICE_CHECK, EKV_DETAIL_TIMEOUT, -2);
    return;
  }

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], 1);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], kTRows / 32);
      mbar_init(&bars->pv_done[t], 1);
      mbar_init(&bars->o_free[t], kTRows / 32);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->kv_full[s], 1);
      mbar_init(&bars->kv_empty[s], 1);
      mbar_init(&bars->v_raw[s], 1);
    }
    mbar_init(&bars->mma_final, 1);
    for (int s = 0; s < kItems; ++s) {
      mbar_init(&bars->item_full[s], 1);
      mbar_init(&bars->item_empty[s], kItemReaders);
    }
    bars->abort = 0;
    fence_barrier_init();
#ifdef EKV_TEST_WAIT_TIMEOUT
    if (p.inject_timeout && blockIdx.x == 0) {             // test build only: 16 bytes that no copy delivers
      uint64_t* const waits[] = {&bars->q_full[0], &bars->kv_full[0], &bars->kv_full[1], &bars->v_raw[1], &bars->s_full[0],
                                 &bars->p_full[0], &bars->pv_done[0], &bars->kv_empty[0], &bars->q_empty[0],
                                 &bars->o_free[0]};
      mbar_expect_tx(waits[p.inject_timeout - 1], 16);
    }
#endif
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 2) tc05::tmem_alloc(&bars->tmem_base, 512);
  const int W = make_plan(p, pl, bars->red) * (p.Hq / p.heads);   // items
  tc05::fence_before_sync();
  __syncthreads();
  tc05::fence_after_sync();
  const uint32_t tbase = bars->tmem_base;
  const int TT = p.tile_tokens;

  // (each register split stands at the head of its roles' code: 80 and 208 a thread, the 168 of launch together)
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      int stage = 0, u = 0;
      uint32_t phase = 0, edges = 0;                         // edges: bit per stage whose last copy went to v_raw
      uint32_t raw_ph = 0;                                   // bit per stage: parity of v_raw's last phase begun
      uint32_t ql[2] = {0u, 0u};                             // query tiles loaded, per tile
      bool ok = true;
      PromptItem it;
      for (int r = 0; next_item(bars, r, it, ok); ++r) {
        const int h = it.hg * p.heads / p.G;
        const bool edge = it.L < it.jhi * kTKeys;          // the last block reaches past the prompt
        for (int x = 0; ok && x < 2 * (it.jhi - it.jlo); ++x) {   // K, V, K, V, ...
          if (u >= NS) ok = wait_warp(&bars->kv_empty[stage], phase ^ 1u, abort);
          if (!ok) break;
          const int j = it.jlo + x / 2;
          const bool is_v = x & 1, raw = is_v && edge && j == it.jhi - 1;
          uint64_t* bar = raw ? &bars->v_raw[stage] : &bars->kv_full[stage];
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, C::IB);
            tma_load_4d(sKV + stage * C::IB, is_v ? &tv : &tk, 0, it.row0 + j * kTKeys, 0, h, bar);
          }
          edges = raw ? edges | 1u << stage : edges & ~(1u << stage);
          if (raw) raw_ph ^= 1u << stage;
          ++u;
          if (++stage == NS) {
            stage = 0;
            phase ^= 1u;
          }
          if (x > 0) continue;
          // The query tiles come behind the first keys, which have a free stage before the tiles' last rows are read, and
          // before the values, which are wanted later: 32 KB take 700 cycles to arrive.
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || it.ja[t] >= it.jb[t]) continue;
            if (ql[t] > 0) ok = wait_warp(&bars->q_empty[t], (ql[t] - 1u) & 1u, abort);
            if (!ok) continue;
            if (lane == 0) {
              mbar_arrive_expect_tx(&bars->q_full[t], (uint32_t)(TT * p.heads * D * 2));
              for (int s = 0; s < NB; ++s)
                tma_load_5d(sQ + t * C::QB + s * kTRows * 128, &tq, 0, 0, s, it.hg, it.row0 + it.q0[t], &bars->q_full[t]);
            }
            ++ql[t];
          }
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) give_up(p.err, abort);
      // the copies still in flight land before the CTA can exit
      for (int v = u > NS ? u - NS : 0; v < u; ++v) {
        const int s = v % NS;
        if ((edges >> s) & 1u) drain(&bars->v_raw[s], ((raw_ph >> s) & 1u) ^ 1u);
        else drain(&bars->kv_full[s], (uint32_t)(v / NS) & 1u);
      }
      for (int t = 0; t < 2; ++t)
        if (ql[t] > 0) drain(&bars->q_full[t], (ql[t] - 1u) & 1u);
    } else if (warp == 2) {
      // ------------------------------------------ the items' descriptions, ahead of their readers
      bool ok = true;
      for (int r = 0; ok; ++r) {
        const int s = r % kItems;
        const bool none = dealt(r) >= W;
        PromptItem it;
        if (none) it.jlo = -1;
        else it = prompt_item(p, pl, dealt(r));
        if (r >= kItems) ok = wait_warp(&bars->item_empty[s], (uint32_t)(r / kItems - 1) & 1u, abort);
        if (!ok) break;
        if (lane == 0) {
          bars->item[s] = it;
          mbar_arrive(&bars->item_full[s]);
        }
        __syncwarp();
        if (none) break;
      }
      if (!ok && lane == 0) give_up(p.err, abort);
    } else if (warp == 3) {
      // ------------------------------------- value rows past a prompt's end: zeros
      int u = 0;                                             // blocks up to the item's end
      uint32_t raw_ph = 0;
      bool ok = true;
      PromptItem it;
      for (int r = 0; next_item(bars, r, it, ok); ++r) {
        u += 2 * (it.jhi - it.jlo);
        const int zr = it.L - (it.jhi - 1) * kTKeys;         // rows >= zr of the last block
        if (zr >= kTKeys) continue;
        const int s = (u - 1) % NS;
        ok = wait_warp(&bars->v_raw[s], (raw_ph >> s) & 1u, abort);
        raw_ph ^= 1u << s;
        if (!ok) break;
        uint8_t* dst = sKV + s * C::IB;
        const int per_slab = (kTKeys - zr) * 8;              // 16-byte chunks past the prompt
        for (int e = lane; e < per_slab * NB; e += 32) {
          const int slab = e / per_slab, rem = e % per_slab;
          *reinterpret_cast<uint4*>(dst + slab * kTKeys * 128 + (zr + rem / 8) * 128 + (rem % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->kv_full[s]);
      }
      if (!ok && lane == 0) give_up(p.err, abort);
    } else if (warp == 1) {
      // ------------------------------------------------------------- MMA issuer
      // The whole warp runs the control flow and computes the descriptors; one elected lane issues.
      constexpr uint32_t idS = tc05::idesc_f16_f32(kTRows, kTKeys, false);
      constexpr uint32_t idO = tc05::idesc_f16_f32(kTRows, D, true);
      constexpr uint32_t HI = tc05::sdesc_hi(1024);          // 8-row groups 1024 B apart
      const uint32_t q_lo = tc05::sdesc_lo(smem_u32(sQ), 16);
      const uint32_t k_lo = tc05::sdesc_lo(smem_u32(sKV), 16);
      const uint32_t v_lo = tc05::sdesc_lo(smem_u32(sKV), kTKeys * 128);
      int ks = 0, vs = 1;                                    // ring cursors of the K blocks and the V blocks
      uint32_t kp = 0, vp = 0;
      uint32_t qc[2] = {0u, 0u}, pc[2] = {0u, 0u}, oc[2] = {0u, 0u};   // phases taken: q_full, p_full; items with an O
      auto adv2 = [&](int& s, uint32_t& ph) {
        s += 2;
        if (s >= NS) {
          s -= NS;
          ph ^= 1u;
        }
      };
      auto commit_one = [&](uint64_t* bar) {
        if (tc05::elect_one()) tc05::commit(bar);
        __syncwarp();
      };
      bool ok = true;
      PromptItem it, after;
      bool go = next_item(bars, 0, after, ok);
      for (int r = 1; go; ++r) {
        it = after;
        // S_t of block j from stage ks, by one lane: over the P_t before it (read by an O_t += P_t V issued earlier: one
        // thread's MMAs run in order)
        auto issue_s = [&](int t, uint32_t ka, bool last) {
          const uint32_t qa = q_lo + t * (C::QB >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc05::mma_ss(tbase + t * 256, tc05::sdesc_join(qa + (((k >> 2) * (kTRows * 128) + (k & 3) * 32) >> 4), HI),
                         tc05::sdesc_join(ka + (((k >> 2) * (kTKeys * 128) + (k & 3) * 32) >> 4), HI), idS, k > 0);
          tc05::commit(&bars->s_full[t]);
          if (last) tc05::commit(&bars->q_empty[t]);
        };
        ok = wait_warp(&bars->kv_full[ks], kp, abort);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (ok && it.ja[t] == it.jlo && it.jlo < it.jb[t]) {
            ok = wait_warp(&bars->q_full[t], qc[t] & 1u, abort);
            ++qc[t];
            tc05::fence_after_sync();
            const uint32_t ka = k_lo + ks * (C::IB >> 4);
            const bool last = it.jlo + 1 == it.jb[t];
            if (ok && tc05::elect_one()) issue_s(t, ka, last);
            __syncwarp();
          }
        }
        if (!ok) break;
        commit_one(&bars->kv_empty[ks]);
        adv2(ks, kp);
        go = next_item(bars, r, after, ok);                // (there long before it is wanted)
        if (!ok) break;
        for (int j = it.jlo; ok && j < it.jhi; ++j) {
          const bool more = j + 1 < it.jhi;
          ok = wait_warp(&bars->kv_full[vs], vp, abort);
          if (ok && more) ok = wait_warp(&bars->kv_full[ks], kp, abort);
          if (!ok) break;
          const uint32_t va = v_lo + vs * (C::IB >> 4), ka = k_lo + ks * (C::IB >> 4);
          uint64_t *const v_free = &bars->kv_empty[vs], *const k_free = &bars->kv_empty[ks];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            // O_t += P_t V_j once the softmax has written P (and, for an item's first block, once the previous item's O_t
            // has been read out), and right behind it S_t of the next block
            const bool pv = j >= it.ja[t] && j < it.jb[t], sn = j + 1 >= it.ja[t] && j + 1 < it.jb[t];
            if (ok && pv) {
              ok = wait_warp(&bars->p_full[t], pc[t] & 1u, abort);
              ++pc[t];
              if (ok && j == it.ja[t] && oc[t] > 0) ok = wait_warp(&bars->o_free[t], (oc[t] - 1u) & 1u, abort);
            }
            if (ok && sn && j + 1 == it.ja[t]) {
              ok = wait_warp(&bars->q_full[t], qc[t] & 1u, abort);
              ++qc[t];
            }
            if (!ok) break;
            const bool acc0 = j > it.ja[t], last_pv = j + 1 == it.jb[t], last_s = j + 2 == it.jb[t];
            const uint32_t pa = tbase + t * 256, od = tbase + t * 256 + 128;
            tc05::fence_after_sync();
            if (tc05::elect_one()) {
              if (pv) {
#pragma unroll
                for (int k = 0; k < kTKeys / 16; ++k)
                  tc05::mma_ts(od, pa + 8 * k, tc05::sdesc_join(va + k * (2048 >> 4), HI), idO, acc0 || k > 0);
                if (last_pv) tc05::commit(&bars->pv_done[t]);
              }
              if (t == 1) tc05::commit(v_free);
              if (sn) issue_s(t, ka, last_s);
              if (t == 1 && more) tc05::commit(k_free);
            }
            __syncwarp();
          }
          if (!ok) break;
          adv2(vs, vp);
          if (more) adv2(ks, kp);
        }
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (it.ja[t] < it.jb[t]) ++oc[t];
      }
      if (!ok && lane == 0) give_up(p.err, abort);
      commit_one(&bars->mma_final);
      if (lane == 0) drain(&bars->mma_final, 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------- softmax, tile t
    const int t = (warp - 4) >> 2, r = threadIdx.x - 128 - t * kTRows;
    const uint32_t lanebase = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float qs = p.qscale;
    const uint32_t t_s = tbase + t * 256 + lanebase, t_o = tbase + t * 256 + 128 + lanebase;
    const int tok_t = r / p.heads;                         // this row's token within the tile
    // a row's results leave 32 bytes at a time, a whole sector, where out lies so
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
    uint32_t sc = 0, pvc = 0;                              // phases taken: s_full, pv_done
    bool ok = true;
    PromptItem it, after;                                  // the next item is looked at while this one's last product runs
    bool more = next_item(bars, 0, after, ok);
    for (int ri = 1; more; ++ri) {
      it = after;
      const int ja = t ? it.ja[1] : it.ja[0], jb = t ? it.jb[1] : it.jb[0], q0 = t ? it.q0[1] : it.q0[0];
      if (ja >= jb) {
        more = next_item(bars, ri, after, ok);
        continue;
      }
      const int pos = q0 + tok_t;
      const int lo = max(pos - p.window, -1);              // the row sees keys lo + 1 .. pos
      const int all_lo = min(q0 + TT, it.L) - 1 - p.window;   // every row sees keys above this and up to q0
      const bool valid = tok_t < TT && pos < it.L;
      float m_ref = -INFINITY, l = 0.f;
      for (int j = ja; j < jb; ++j) {
        // S of block j is there; O += P V of block j - 1 has completed too (its commit came first)
        ok = wait_warp(&bars->s_full[t], sc & 1u, abort);
        ++sc;
        if (!ok) break;
        tc05::fence_after_sync();
        const int k0 = j * kTKeys;
        uint32_t sv[4][32];
        float mx = k0 + kTKeys - 1 > q0 || k0 <= all_lo ? prompt_row<true>(t_s, lo - k0, pos - k0, sv) : prompt_row<false>(t_s, 0, 0, sv);
        mx = fmaf(mx, qs, -kHeadroom);
        const float m_new = fmaxf(m_ref, mx);
        const bool need = m_new > m_ref + 8.f;
        if (__any_sync(0xffffffffu, need)) {
          const float alpha = need ? ex2(m_ref - m_new) : 1.f;
          if (j > ja) {
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
        l += prompt_weights(t_s, qs, m_ref == -INFINITY ? 0.f : -m_ref, sv);
        tc05::wait_st();
        tc05::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[t]);
      }
      if (!ok) break;
      more = next_item(bars, ri, after, ok);
      if (!ok) break;
      ok = wait_warp(&bars->pv_done[t], pvc & 1u, abort);
      ++pvc;
      if (!ok) break;
      tc05::fence_after_sync();
      const bool none = l == 0.f;                          // every score -inf (a NaN goes on to the output)
      const float inv = none ? 0.f : 1.f / l;
      const size_t orow = (size_t)(it.row0 + pos) * p.Hq + it.hg * p.heads + r % p.heads;
#pragma unroll 1
      for (int x = 0; x < D / 32; ++x) {
        uint32_t o[32];
        tc05::ld32(t_o + 32 * x, o);
        tc05::wait_ld();
        if (x == D / 32 - 1) {                             // O is read out: the next item may overwrite it
          tc05::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->o_free[t]);
        }
        if (valid) {
          uint32_t w[16];
#pragma unroll
          for (int y = 0; y < 16; ++y) w[y] = none ? 0u : pack2(__uint_as_float(o[2 * y]) * inv, __uint_as_float(o[2 * y + 1]) * inv);
          __half* dst = p.out + orow * D + 32 * x;
          if (wide) {
            store32(dst, w);
            store32(dst + 16, w + 8);
          } else {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              *reinterpret_cast<uint4*>(dst + 8 * y) = make_uint4(w[4 * y], w[4 * y + 1], w[4 * y + 2], w[4 * y + 3]);
          }
        }
      }
      if (valid && p.lse) p.lse[orow] = none ? -INFINITY : (m_ref + log2f(l)) * 0.69314718055994531f;
    }
    if (!ok && lane == 0) give_up(p.err, abort);
  }
  tc05::fence_before_sync();
  __syncthreads();
  if (warp == 2) {
    tc05::fence_after_sync();
    tc05::tmem_free(tbase, 512);
  }
}

// Key or value rows: 4-D view (d mod 64, row, d / 64, head), `stride` values between rows; the box {64, 128, D / 64, 1}
// lands 128 rows of one head as [D / 64][128 rows][128 B], 128B swizzle. Rows past `rows` read as zeros.
bool encode_kv_map(CUtensorMap* tm, const void* base, int D, int heads, int rows, long long stride) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)(D / 64), (cuuint64_t)heads};
  cuuint64_t strides[3] = {(cuuint64_t)stride * 2, 128, (cuuint64_t)D * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)kTKeys, (cuuint32_t)(D / 64), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_prompt(const PromptParams& p, int num_sms, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  if (!encode_query_map(&tq, p.q, D, p.Hq / p.heads, p.heads, p.total, p.tile_tokens, p.q_stride) ||
      !encode_kv_map(&tk, p.k, D, p.Hkv, p.total, p.k_stride) || !encode_kv_map(&tv, p.v, D, p.Hkv, p.total, p.v_stride))
    return cudaErrorInvalidValue;
  constexpr int smem = prompt_smem_bytes<D>();
  static_assert(smem <= 232448, "shared memory of one CTA");
  static_assert(sizeof(Plan) % 16 == 0, "the barriers lie behind it");
  cudaError_t e = set_smem_attr(reinterpret_cast<const void*>(prompt_tc05_kernel<D>), smem);
  if (e != cudaSuccess) return e;
  // at most so many items: a CTA for each, and one a processor
  const long long items = ((long long)p.total / (2 * p.tile_tokens) + p.n) * (p.Hq / p.heads);
  prompt_tc05_kernel<D><<<(int)(items < num_sms ? items : num_sms), kPThreads, smem, st>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_tc05(PromptParams p, int D, int num_sms, cudaStream_t st) {
  // Packed heads fill the tiles of short prompts and keep the masked edges of a window short; a long prompt's tiles are full
  // either way, and with one head each the CTAs of a KV head read the same keys at about the same time. D 128, one head / packed:
  // 8 x 8,192 tokens 2,947 / 3,180 us, 4 x 8,192 1,503 / 1,512, under a window of 2,048 770 / 756, 16 prompts of 100 to
  // 4,096 426 / 408, 200 of 1 to 300 (G 8) 244 / 148. D 64: packed everywhere (4 x 8,192 541 / 535).
  // The mean length does not tell all cases apart: equal prompts below the threshold would do better with one head (32/8 heads, 64 x 512
  // 178 / 192, 32 x 1,024 264 / 276, 16 x 2,048 442 / 459), a single one of 4,096 packed (117 / 113); nor does the host know
  // that a window hides nothing (8 x 8,192 under one of 8,192: 3,515 us packed, 3,201 without) or that `total` counts rows of no prompt.
  p.heads = D == 128 && p.window == 0x7fffffff && p.total >= 4096ll * p.n ? 1 : p.G;
  p.tile_tokens = kTRows / p.heads;
  return D == 128 ? launch_prompt<128>(p, num_sms, st) : launch_prompt<64>(p, num_sms, st);
}

}  // namespace ekv
