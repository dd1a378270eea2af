// Softmax attention over a sliding window with first tokens that stay visible,
// backward:
//   P_ij = exp(s_ij - lse_i) where key j is visible to query i, else 0,
//   delta_i = dout_i . o_i,  dS = P (dout V^T - delta),
//   dq = scale dS K,  dk = scale dS^T Q,  dv = P^T dout.
//
// Launches per call:
//   1. prep : -delta and -lse log2(e) per query, padded to whole blocks of 128
//             (padding: 0 and -inf, so P = 0 there)
//   2. kv   : dK and dV of a block of 128 keys accumulate in TMEM over the blocks
//             of 128 queries that meet it; each bf16 dS tile leaves for the workspace
//   3. dq   : dQ of a block of 128 queries accumulates over its dS tiles and K blocks
//   4. join : where a key block's queries were dealt to several CTAs, the sum of
//             their parts in a fixed order
// Only pairs of blocks that meet are visited: the window's, and for the first
// tokens' blocks all queries behind them.  Where that is more than a CTA's share of
// all pairs, they go to several CTAs (and all blocks' do while the grid would not
// fill the GPU); parts are fp32 in the workspace.
//
// kv (persistent, one CTA per SM, 16 warps: 0 loads, 1 and 2 products, 4-11 softmax,
// 12-15 outputs): per pair of blocks the products go out in the order
//   S(n) dP(n) | P(n) ready: dV(n) S(n+1) | dS(n) ready: dK(n) dP(n+1)
// with S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q (M = 128 keys, P and
// dS as A operands in TMEM over S and dP), so P is formed while dP runs, dS while
// dV and the next S run.  n runs on across items: K and V of the next one arrive
// while the last pair of this one is worked on.  Per slot of dO, once dV has read
// it, the dS tile is staged there for its copy to the workspace, and behind an
// item's last pair dV and dK as bf16 rows.
// dq (persistent): dQ += dS K with A = dS^T tiles as they stand (queries contiguous)
// and B = K, into two accumulators in turn.
// Rows behind a sequence's last token are cleared in shared memory before a
// product sees them, so nothing there (NaN included) is looked at.
//
// 4 x 2048 tokens of 20 heads, window 512: 175 us.  prep 16: memory.  kv 112: a CTA has
// 43 pairs of blocks in 8 items.  A pair takes 2.0 us (windows of 512, 1024 and all keys:
// 112, 150, 170 us for 43, 61, 72 pairs), of which the four products are 1.05: S, the
// exponentials, dV and dP, dS, dK are two chains that depend on one another.  The other 27
// us are the changes of item: both accumulators and a slot of dO are handed on only when
// the output warps have dV and dK out of TMEM.  dq 45: memory, mostly the dS
// tiles, which are written once and read once (212 MB each; recomputing S and dP
// there would take three products in place of one).  What measured worse: dS tiles,
// dV and dK stored from registers (217 and 213 us in place of 194: a store of 32 rows
// is 32 transactions), items taken from a counter in memory and handed on through a
// ring (179 in place of 176; long items at the end of the list are left to one CTA).
#include <algorithm>

#include "window.cuh"

namespace abw {
namespace {

using namespace win;

constexpr int kThr = 384;        // dq kernel
constexpr int kKvThr = 512;      // kv kernel
constexpr long long kGroupBytes = 72 << 20;   // 4 x 2048 tokens of 20 heads, all keys: 24 MB 290, 48 265, 72 255, 96 255 us
constexpr int kTileBytes = kBlk * kBlk * 2;    // one dS^T tile: [2 query halves][128 keys][64 queries]

// Which blocks meet, and where their dS tiles stand within a head.
struct Grid {
  int nb;        // blocks of 128 tokens
  int wq;        // query blocks that a key block behind the first tokens' meets
  int first;     // key blocks of first tokens
  int window, sinks;
  __host__ __device__ int queries(int kb) const { return kb < first || nb - kb < wq ? nb - kb : wq; }
  // dS tiles in front of key block kb's
  __host__ __device__ long long tile0(int kb) const {
    const int a = kb < first ? kb : first;
    long long n = static_cast<long long>(a) * nb - static_cast<long long>(a) * (a - 1) / 2;
    if (kb <= first) return n;
    int e = nb - wq > first ? nb - wq : first;   // from here on fewer than wq follow
    if (e > kb) e = kb;
    n += static_cast<long long>(e - first) * wq;
    const long long k = kb - e;
    return n + k * (nb - e) - k * (k - 1) / 2;
  }
  // a query block's key blocks: lead of first tokens, then lo .. m
  __host__ __device__ int lo(int m) const {
    const int x = m * kBlk - window + 1;
    return x > 0 ? x / kBlk : 0;
  }
  __host__ __device__ int lead(int m) const { return first < lo(m) ? first : lo(m); }
};

Grid grid_of(int T, int window, int sinks) {
  Grid g;
  g.nb = (T + kBlk - 1) / kBlk;
  g.window = std::min(window, T);
  g.sinks = std::min(sinks, T);
  g.wq = std::min(g.nb, 1 + (g.window + kBlk - 2) / kBlk);
  g.first = (g.sinks + kBlk - 1) / kBlk;
  return g;
}

struct BwdParams {
  const __nv_bfloat16 *o, *dout;
  const float *lse;
  const int *lengths;
  float *ndelta, *nlse2;          // [B][Hq][Tp]
  __nv_bfloat16 *ds;              // [B][Hq][tiles]
  float *parts;                   // [units][slots][2: dV, dK][D / 4][128 keys][4]
  __nv_bfloat16 *dq, *dk, *dv;
  int B, T, Tp, Hq, Hkv, G;
  long long o_stride, dout_stride, dk_stride, dv_stride, tiles;
  Grid g;
  int first_parts, parts_each;    // CTAs per key block: first tokens', others
  int per_unit, slots;            // items (without the first tokens') and part slots per (batch, KV head)
  int items, dq_items;
  int units, group;               // (batch, KV head)s, in scheduling groups
  int lead_items, lead_rounds, lead_rest, span, rounds;   // see kv_nth
  Div by_units, by_group, by_width, by_last;  // units, items of a group, its units (the last one's)
  Div by_dq_group, by_dq_width, by_dq_last;   // the same of the dq kernel's items, heads
  Div by_hkv, by_first, by_each, by_hq, by_chunks, by_g;   // Hkv, first_parts, parts_each, ..
  float scale;
  WaitCtl wait;
};

// ---------------------------------------------------------------------- prep
// A block per 32 (64) tokens of a head, heads next to one another: what runs at one
// time reads o and dout in order, and the statistics are written in whole lines.  A
// row per kD / 8 lanes, two rows each.
constexpr int kPrepThr = 256, kPrepRows = 2;
template <int kD>
constexpr int kPrepTokens = kPrepRows * kPrepThr * 8 / kD;

__device__ __forceinline__ float dot8(uint4 a, uint4 g) {
  return bf16_lo(a.x) * bf16_lo(g.x) + bf16_hi(a.x) * bf16_hi(g.x) + bf16_lo(a.y) * bf16_lo(g.y) +
         bf16_hi(a.y) * bf16_hi(g.y) + bf16_lo(a.z) * bf16_lo(g.z) + bf16_hi(a.z) * bf16_hi(g.z) +
         bf16_lo(a.w) * bf16_lo(g.w) + bf16_hi(a.w) * bf16_hi(g.w);
}

template <int kD>
__global__ void __launch_bounds__(kPrepThr) window_prep_kernel(const __grid_constant__ BwdParams p) {
  constexpr int kL = kD / 8;   // lanes of a row
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int sub = threadIdx.x % kL;
  int h = blockIdx.x;
  int b = p.by_hq(h);          // a quotient; h becomes the remainder
  int chunk = b;
  b = p.by_chunks(chunk);
  const int n = tokens_of(p.lengths, b, p.T), t0 = chunk * kPrepTokens<kD> + threadIdx.x / kL;
  const size_t row = static_cast<size_t>(b) * p.Hq + h;
  uint4 x[kPrepRows], y[kPrepRows];
  float l[kPrepRows];
#pragma unroll
  for (int k = 0; k < kPrepRows; ++k) {
    const int t = t0 + k * (kPrepThr / kL);
    x[k] = y[k] = make_uint4(0, 0, 0, 0);
    l[k] = INFINITY;           // padding: P = 2^(s - inf) = 0
    if (t < n) {
      const long long tok = static_cast<long long>(b) * p.T + t;
      x[k] = *reinterpret_cast<const uint4 *>(p.o + tok * p.o_stride + static_cast<size_t>(h) * kD + 8 * sub);
      y[k] = *reinterpret_cast<const uint4 *>(p.dout + tok * p.dout_stride + static_cast<size_t>(h) * kD + 8 * sub);
      if (sub == 0) l[k] = p.lse[row * p.T + t];
    }
  }
#pragma unroll
  for (int k = 0; k < kPrepRows; ++k) {
    const int t = t0 + k * (kPrepThr / kL);
    float v = dot8(x[k], y[k]);
#pragma unroll
    for (int d = kL / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);   // within the row's lanes
    if (sub == 0 && t < p.Tp) {
      p.ndelta[row * p.Tp + t] = -v;
      p.nlse2[row * p.Tp + t] = -l[k] * kLog2e;
    }
  }
}

// ------------------------------------------------------------------------ kv
template <int kD>
struct KvSmem {
  static constexpr int kIn = kBlk * kD * 2;                  // one block of Q, K, V or dO
  static constexpr int kQs = 3, kDOs = 2;
  static constexpr int kDOPitch = kTileBytes;                // a dO slot also stages a dS tile
  static constexpr int kK = 0, kV = kIn, kQ = 2 * kIn, kDO = kQ + kQs * kIn;
  static constexpr int kLse = kDO + kDOs * kDOPitch;         // 512 B per Q slot
  static constexpr int kDelta = kLse + kQs * 512;            // 512 B per dO slot
  static constexpr int kBar = kDelta + kDOs * 512;
  enum {
    kKFull = 0, kVFull, kKEmpty, kVEmpty, kQFull, kQEmpty = kQFull + kQs, kDOFull = kQEmpty + kQs,
    kDOEmpty = kDOFull + kDOs, kSFull = kDOEmpty + kDOs, kDPFull, kPFull, kDSFull, kDSRead, kDVDone, kDKFinal = kDVDone + kDOs,
    kAccFree, kRaw, kFinal, kBars
  };
  static constexpr int kTmem = kBar + kBars * 8, kAbort = kTmem + 4;
  static constexpr int kBytes = kAbort + 4;                  // the kernel checks that the base is aligned
  static_assert(kBytes <= 232448, "kv kernel shared memory");
};

// nth_item for the kv kernel, whose items are first the first tokens' blocks of keys,
// dealt in turn, then the others, block of keys by block of keys through the units of
// a group, so that the short ones, whose queries end with the sequence, come last.
// `lead_rest` CTAs have one of the long items more; while they work on it the others
// take `span` of the others.  (With the long items cut to the others' length and dealt
// among them, 4 x 2048 tokens of 20 heads, window 512, took 194 us, this way 176.)
__device__ __forceinline__ int kv_nth(const BwdParams &p, int r) {
  const int c = blockIdx.x, n = gridDim.x, rest = p.lead_rest;
  const int lead = p.lead_rounds + (c < rest);
  if (r < lead) return c + r * n;
  r -= lead;
  int from = p.lead_items;
  if (rest > 0) {
    if (c >= rest) {
      if (r < p.span) return from + r * (n - rest) + c - rest;
      r -= p.span;
    }
    from += p.span * (n - rest);
  }
  return from + nth_item(r);
}

struct KvItem {
  int b, kvh, kb, part, nparts, n, qn;   // tokens, live query blocks per head
  int it0, it1;                          // its pairs: (head, query block) = it / qn, it % qn
  long long slot;                        // of its part (nparts > 1)
};

__device__ __noinline__ KvItem kv_item(const BwdParams &p, int idx) {
  KvItem r;
  const bool lead = idx < p.lead_items;
  int unit, head = 0;                       // slots in front of the place's
  if (lead) {
    r.part = p.by_units(idx);
    unit = idx;
  } else {
    idx -= p.lead_items;
    unit = p.by_group(idx) * p.group;       // idx becomes the place in the group
    r.part = unit + p.group <= p.units ? p.by_width(idx) : p.by_last(idx);
    unit += idx;
    if (p.first_parts > 1) head = p.g.first * p.first_parts;
  }
  r.kvh = unit;
  r.b = p.by_hkv(r.kvh);
  r.slot = static_cast<long long>(unit) * p.slots + head + r.part;
  const Div &div = lead ? p.by_first : p.by_each;
  r.kb = div(r.part) + (lead ? 0 : p.g.first);
  r.nparts = div.d;
  r.n = tokens_of(p.lengths, r.b, p.T);
  const int live = (r.n + kBlk - 1) / kBlk;
  r.qn = max(0, min(r.kb + p.g.queries(r.kb), live) - r.kb);
  int extra = p.G * r.qn;                   // the first `extra` parts have one more
  const int each = div(extra);
  r.it0 = r.part * each + min(r.part, extra);
  r.it1 = r.it0 + each + (r.part < extra);
  return r;
}

// The pairs of a CTA's items, one after the other.
struct KvStream {
  KvItem w;
  int round, it, h, qb;       // pair `it` of the item: query head h, block qb of queries
  bool valid;
  __device__ __forceinline__ void find(const BwdParams &p) {
    valid = false;
    for (; !valid && round < p.rounds; ++round) {
      const int idx = kv_nth(p, round);
      if (idx >= p.items) continue;
      w = kv_item(p, idx);
      if (w.it0 == w.it1) continue;
      it = w.it0;
      h = it / w.qn;
      qb = w.kb + it - h * w.qn;
      h += w.kvh * p.G;
      valid = true;
    }
  }
  __device__ __forceinline__ void begin(const BwdParams &p) {
    round = 0;
    find(p);
  }
  __device__ __forceinline__ void next(const BwdParams &p) {
    if (++it == w.it1) return find(p);
    if (++qb == w.kb + w.qn) qb = w.kb, ++h;
  }
  __device__ __forceinline__ bool opens() const { return it == w.it0; }
  __device__ __forceinline__ bool closes() const { return it == w.it1 - 1; }
};

template <int kD>
__global__ void __launch_bounds__(kKvThr, 1)
    window_kv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmdK, const __grid_constant__ CUtensorMap tmdV,
                     const __grid_constant__ BwdParams p) {
  using M = KvSmem<kD>;
  constexpr int kHalves = kD / 64;
  constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 256 + kD;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (sb & 1023) {
    if (tid == 0) atomicOr(p.wait.err, kErrSmemAlign);
    return;
  }
  auto bar = [&](int i) -> uint32_t { return sb + M::kBar + i * 8; };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + M::kAbort);
  const Waits wts{sb + M::kBar, abort_flag, &p.wait, kSiteWinKv};
  auto wtw = [&](int slot, uint32_t parity) -> bool { return wait_warp(wts, slot, parity); };

  if (tid == 0) {
    for (int i = 0; i < M::kBars; ++i) {
      int count = 1;
      if (i == M::kPFull || i == M::kDSFull) count = 256;                            // softmax threads
      if (i == M::kDSRead || i == M::kAccFree) count = 128;                          // output threads
      if (i == M::kDOEmpty || i == M::kDOEmpty + 1) count = 4;                       // output warps
      if (i == M::kFinal) count = 2;
      mbar_init(bar(i), count);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2) tc::tmem_alloc(sb + M::kTmem, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(smem + M::kTmem), 0);

  if (warp == 0) {
    // ============================ loads ================================
    if (lane == 0) {
      prefetch_tensormap(&tmK);
      prefetch_tensormap(&tmQ);
      prefetch_tensormap(&tmV);
      prefetch_tensormap(&tmDO);
    }
    int raw = 0, nq = 0, nd = 0, nk = 0, nv = 0;   // copies so far: repaired, Q, dO, K, V
    // one block of 128 rows (and 512 B of row statistics), rows from `live` on cleared
    auto load = [&](const CUtensorMap *map, uint32_t off, int h, int row0, int b, int live, uint32_t full, uint32_t stat_off,
                    const float *stat) {
      const bool repair = live < kBlk && row0 + live < p.T;
      const uint32_t fb = repair ? bar(M::kRaw) : full;
      if (lane == 0) {
        mbar_arrive_expect_tx(fb, M::kIn + (stat ? 512 : 0));
        for (int hx = 0; hx < kHalves; ++hx) tma_load_4d(sb + off + hx * 16384, map, hx * 64, h, row0, b, fb);
        if (stat) bulk_load(sb + stat_off, stat, 512, fb);
      }
      if (repair) clear_tail<kHalves>(wts, smem + off, live, M::kRaw, raw++ & 1, full);
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the statistics come from prep
    KvStream s;
    for (s.begin(p); s.valid; s.next(p)) {
      const KvItem &w = s.w;
      const int h = s.h, q0 = s.qb * kBlk, k0 = w.kb * kBlk;
      const int qs = nq % M::kQs, ds = nd % M::kDOs;
      const size_t ro = (static_cast<size_t>(w.b) * p.Hq + h) * p.Tp + q0;
      if (s.opens()) {
        if (!wtw(M::kKEmpty, (nk & 1) ^ 1)) break;
        load(&tmK, M::kK, w.kvh, k0, w.b, w.n - k0, bar(M::kKFull), 0, nullptr);
        ++nk;
      }
      if (!wtw(M::kQEmpty + qs, ((nq / M::kQs) & 1) ^ 1)) break;
      load(&tmQ, M::kQ + qs * M::kIn, h, q0, w.b, w.n - q0, bar(M::kQFull + qs), M::kLse + qs * 512, p.nlse2 + ro);
      ++nq;
      if (s.opens()) {
        if (!wtw(M::kVEmpty, (nv & 1) ^ 1)) break;
        load(&tmV, M::kV, w.kvh, k0, w.b, w.n - k0, bar(M::kVFull), 0, nullptr);
        ++nv;
      }
      if (!wtw(M::kDOEmpty + ds, ((nd / M::kDOs) & 1) ^ 1)) break;
      load(&tmDO, M::kDO + ds * M::kDOPitch, h, q0, w.b, w.n - q0, bar(M::kDOFull + ds), M::kDelta + ds * 512, p.ndelta + ro);
      ++nd;
    }
    // The last copy of every slot has landed before the CTA may end, whoever gives up
    // and when (otherwise this finds every phase complete).
    for (int i = max(nq - M::kQs, 0); i < nq; ++i) wait_landed(bar(M::kQFull + i % M::kQs), (i / M::kQs) & 1);
    for (int i = max(nd - M::kDOs, 0); i < nd; ++i) wait_landed(bar(M::kDOFull + i % M::kDOs), (i / M::kDOs) & 1);
    if (nk > 0) wait_landed(bar(M::kKFull), (nk - 1) & 1);
    if (nv > 0) wait_landed(bar(M::kVFull), (nv - 1) & 1);
  } else if (warp < 3) {
    // ============================ products =============================
    // Warp 1 issues S and dV, which share TMEM columns with P, warp 2 dP and dK.
    // Between two products an issuer waits and looks things up for some 400 cycles;
    // two of them do so in turn (one for both measured the same, within 1 %).
    constexpr uint32_t id_sdp = tc::idesc_bf16_f32(128, 128, 0, 0);   // S^T, dP^T
    constexpr uint32_t id_kv = tc::idesc_bf16_f32(128, kD, 0, 1);     // dV, dK (A from TMEM)
    int gave_up = 0;
    auto wti = [&](int slot, uint32_t parity) -> bool { return wait_issuer(wts, slot, parity, gave_up); };
    const bool first = warp == 1;
    // The first's operands: K, Q (K-major B of S^T), dO (MN-major B of dV); the
    // second's: V, dO, Q.
    const uint64_t dA = tc::sdesc_sw128(sb + (first ? M::kK : M::kV), 16, 1024);
    const uint64_t dBk = tc::sdesc_sw128(sb + (first ? M::kQ : M::kDO), 16, 1024);
    const uint64_t dBm = tc::sdesc_sw128(sb + (first ? M::kDO : M::kQ), 16384, 1024);
    const uint32_t tX = tmem + (first ? kColS : kColDP), tY = tmem + (first ? kColDV : kColDK);
    auto qoff = [](int n) -> uint64_t { return static_cast<uint64_t>((n % M::kQs) * M::kIn) >> 4; };
    auto dooff = [](int n) -> uint64_t { return static_cast<uint64_t>((n % M::kDOs) * M::kDOPitch) >> 4; };
    int items = 0, na = 0;                  // items whose output was begun; K (V) blocks waited for
    // pairs of the next item that has some; 0: there is none
    int round = 0;
    auto next_item = [&]() -> int {
      int pairs = 0;
      for (; pairs == 0 && round < p.rounds; ++round) {
        const int idx = kv_nth(p, round);
        if (idx >= p.items) continue;
        const KvItem w = kv_item(p, idx);
        pairs = __shfl_sync(0xffffffffu, w.it1 - w.it0, 0);
      }
      return pairs;
    };
    // `left` pairs of the item from this one on, `then` from the next one on (of the
    // next item behind the last); n = -1: only S and dP of pair 0
    int left = 1, then = next_item();
    bool opens = false, ok = may_wait(p.wait, abort_flag, kSiteWinKv, M::kKFull);
#pragma unroll 1
    for (int n = -1; ok && left > 0; ++n) {
      const bool closes = left == 1;
      if (n >= 0) {                         // dV += P^T dO (dK += dS^T Q)
        // the accumulators of the item before have been read
        if (opens && !wti(M::kAccFree, (items++ & 1) ^ 1)) break;
        if (!wti(first ? M::kDOFull + n % M::kDOs : M::kQFull + n % M::kQs, (n / (first ? M::kDOs : M::kQs)) & 1)) break;
        if (!wti(first ? M::kPFull : M::kDSFull, n & 1)) break;
        tc::fence_after_sync();
        if (tc::elect()) {
          tc::product_ts<2, 32>(tY, tX, dBm + (first ? dooff(n) : qoff(n)), id_kv, !opens);
          tc::commit(bar(first ? M::kDVDone + n % M::kDOs : M::kQEmpty + n % M::kQs));
          if (closes && !first) tc::commit(bar(M::kDKFinal));
        }
        __syncwarp();
      }
      const int m = n + 1;                  // S^T = K Q^T (dP^T = V dO^T) of the next pair
      if (then > 0) {
        if (closes && !wti(first ? M::kKFull : M::kVFull, na++ & 1)) break;
        if (!wti(first ? M::kQFull + m % M::kQs : M::kDOFull + m % M::kDOs, (m / (first ? M::kQs : M::kDOs)) & 1)) break;
        if (!first && n >= 0 && !wti(M::kDSRead, n & 1)) break;   // the dS tile has been read for the workspace
        tc::fence_after_sync();
        if (tc::elect()) {
          tc::product_k<kD>(tX, dA, dBk + (first ? qoff(m) : dooff(m)), id_sdp);
          tc::commit(bar(first ? M::kSFull : M::kDPFull));
          if (then == 1) tc::commit(bar(first ? M::kKEmpty : M::kVEmpty));
        }
        __syncwarp();
      }
      opens = closes;
      left = then;
      then = left == 1 ? next_item() : left - 1;
    }
    tc::commit_w(bar(M::kFinal));
    report_issuer(wts, gave_up);
    wait_landed(bar(M::kFinal), 0);   // every product of both has completed
  } else if (warp >= 4 && warp < 12) {
    // ============================ softmax ================================
    // Warp w: keys 32 (w % 4) .. of the block (thread = key), half (w - 4) / 4 of its
    // 128 queries.
    const int qd = warp & 3, ch = (warp - 4) >> 2;
    const int j = 32 * qd + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
    const float sl2 = p.scale * kLog2e;
    const float2 sl22 = make_float2(sl2, sl2);
    const uint32_t tS = tmem + lanes + kColS + 64 * ch, tD = tmem + lanes + kColDP + 64 * ch;
    KvStream s;
    int n = 0;
    for (s.begin(p); s.valid; s.next(p), ++n) {
      const int k0 = s.w.kb * kBlk, key = k0 + j, qblk = s.qb * kBlk, q0 = qblk + 64 * ch;
      const float *nl = reinterpret_cast<const float *>(smem + M::kLse + (n % M::kQs) * 512) + 64 * ch;
      const float *nd = reinterpret_cast<const float *>(smem + M::kDelta + (n % M::kDOs) * 512) + 64 * ch;
      // this half's queries that see the key; all of them where the block is whole
      uint32_t see[2] = {0xffffffffu, 0xffffffffu};
      if (!(qblk > k0 && (qblk + kBlk - 1 - k0 < p.g.window || p.g.sinks - k0 >= kBlk))) {
        const int first = key - q0, end = key < p.g.sinks ? 64 : first + p.g.window;
#pragma unroll
        for (int x = 0; x < 2; ++x) see[x] = below(end - 32 * x) & ~below(first - 32 * x);
      }
      // ---- P = 2^(S scale log2 e - lse log2 e)
      float2 P[32];
      if (!wtw(M::kSFull, n & 1)) break;
      tc::fence_after_sync();
      {
        float(&lo)[32] = *reinterpret_cast<float(*)[32]>(&P[0]);
        float(&hi)[32] = *reinterpret_cast<float(*)[32]>(&P[16]);
        tc::ld32x2_wait(tS, tS + 32, lo, hi);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {   // chunk c of 16 queries: columns 32 (c / 2) + 8 (c % 2)
        uint32_t pk[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float4 l4 = *reinterpret_cast<const float4 *>(nl + 16 * c + 2 * e);
          float2 &a = P[8 * c + e], &b = P[8 * c + e + 1];
          a = fma2(a, sl22, make_float2(l4.x, l4.y));
          b = fma2(b, sl22, make_float2(l4.z, l4.w));
          const uint32_t m = see[c >> 1] >> ((16 * c + 2 * e) & 31);
          a = make_float2(m & 1u ? ex2(a.x) : 0.f, m & 2u ? ex2(a.y) : 0.f);
          b = make_float2(m & 4u ? ex2(b.x) : 0.f, m & 8u ? ex2(b.y) : 0.f);
          pk[e] = pack_bf16(a.x, a.y);
          pk[e + 1] = pack_bf16(b.x, b.y);
        }
        tc::st8_async(tS + (c >> 1) * 32 + (c & 1) * 8, pk);
      }
      tc::wait_st();
      tc::fence_before_sync();
      mbar_arrive(bar(M::kPFull));
      // ---- dS = P (dP - delta), over dP
      if (!wtw(M::kDPFull, n & 1)) break;
      tc::fence_after_sync();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float d[32];
        tc::ld32_wait(tD + 32 * half, d);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int i = 16 * c + 2 * e;
            const float4 d4 = *reinterpret_cast<const float4 *>(nd + 32 * half + i);
            const float2 x = add2(make_float2(d[i], d[i + 1]), make_float2(d4.x, d4.y));
            const float2 y = add2(make_float2(d[i + 2], d[i + 3]), make_float2(d4.z, d4.w));
            const float2 a = P[16 * half + i / 2], b = P[16 * half + i / 2 + 1];
            pk[e] = pack_bf16(a.x * x.x, a.y * x.y);
            pk[e + 1] = pack_bf16(b.x * y.x, b.y * y.y);
          }
          tc::st8_async(tD + 32 * half + 8 * c, pk);
        }
      }
      tc::wait_st();
      tc::fence_before_sync();
      mbar_arrive(bar(M::kDSFull));
    }
    tc::wait_st();
  } else if (warp >= 12) {
    // ============================ outputs ================================
    // Warp w: keys 32 (w % 4) .. (thread = key).  Each pair's dS^T goes from TMEM
    // through the pair's dO slot, once dV has read that, to the workspace; behind an
    // item's last pair dV and dK go the same way as bf16 rows (or, a part, as fp32).
    // A warp's rows are 4 KB of each half, which it writes and sends by itself.
    const int qd = warp & 3, j = 32 * qd + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
    KvStream s;
    int n = 0, items = 0;
    for (s.begin(p); s.valid; s.next(p), ++n) {
      const KvItem &w = s.w;
      const uint32_t off = M::kDO + (n % M::kDOs) * M::kDOPitch;
      unsigned char *rows = smem + off + j * 128;        // of half 0; half 1 is 16 KB behind
      if (!wtw(M::kDSFull, n & 1)) break;
      tc::fence_after_sync();
      uint32_t u[64];                                    // 128 queries, two to a register
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::ld16_wait(tmem + lanes + kColDP + 32 * c, *reinterpret_cast<uint32_t(*)[16]>(&u[16 * c]));
      tc::fence_before_sync();
      mbar_arrive(bar(M::kDSRead));
      // per slot: dV may be a pair ahead of this warp, but not of this slot
      if (!wtw(M::kDVDone + n % M::kDOs, (n / M::kDOs) & 1)) break;
#pragma unroll
      for (int x = 0; x < 16; ++x)
        *reinterpret_cast<uint4 *>(rows + (x >> 3) * 16384 + (((x & 7) ^ (j & 7)) << 4)) =
            make_uint4(u[4 * x], u[4 * x + 1], u[4 * x + 2], u[4 * x + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        unsigned char *dst = reinterpret_cast<unsigned char *>(p.ds) +
                             ((static_cast<long long>(w.b) * p.Hq + s.h) * p.tiles + p.g.tile0(w.kb) + s.qb - w.kb) * kTileBytes +
                             qd * 4096;
        bulk_store(dst, sb + off + qd * 4096, 4096);
        bulk_store(dst + 16384, sb + off + 16384 + qd * 4096, 4096);
        bulk_commit_group();
      }
      bool ok = true;
      if (s.closes()) {
        tc::fence_after_sync();
        float4 *part = reinterpret_cast<float4 *>(p.parts) + w.slot * 2 * (kD / 4) * kBlk + j;
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {                    // dV, dK
          if (x == 1) {
            ok = wtw(M::kDKFinal, items & 1);
            if (!ok) break;
            tc::fence_after_sync();
          }
          const float f = x == 0 ? 1.f : p.scale;
          const uint32_t from = tmem + lanes + (x == 0 ? kColDV : kColDK);
          if (w.nparts == 1) {
#pragma unroll
            for (int c = 0; c < kD; c += 32) {
              float v[32];
              tc::ld32_wait(from + c, v);
#pragma unroll
              for (int e = 0; e < 16; ++e) u[c / 2 + e] = pack_bf16(v[2 * e] * f, v[2 * e + 1] * f);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < kD; c += 32) {
              float v[32];
              tc::ld32_wait(from + c, v);
#pragma unroll
              for (int e = 0; e < 8; ++e)                // a warp's 32 keys next to one another
                part[(x * (kD / 4) + c / 4 + e) * kBlk] = make_float4(v[4 * e] * f, v[4 * e + 1] * f, v[4 * e + 2] * f, v[4 * e + 3] * f);
            }
          }
          if (x == 1) {                                  // the next item's products may begin
            tc::fence_before_sync();
            mbar_arrive(bar(M::kAccFree));
          }
          if (w.nparts > 1) continue;
          if (lane == 0) bulk_wait_group_read0();        // the copies out of the rows have read them
          __syncwarp();
#pragma unroll
          for (int e = 0; e < kD / 8; ++e)
            *reinterpret_cast<uint4 *>(rows + (e >> 3) * 16384 + (((e & 7) ^ (j & 7)) << 4)) =
                make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          const int row0 = w.kb * kBlk + 32 * qd;
          if (lane == 0 && row0 < p.T) {                 // rows past T are not written
            for (int hx = 0; hx < kHalves; ++hx)
              tma_store_4d(x == 0 ? &tmdV : &tmdK, sb + off + hx * 16384 + qd * 4096, hx * 64, w.kvh, row0, w.b);
            bulk_commit_group();
          }
        }
        if (!ok) break;
        ++items;
      }
      if (lane == 0) {
        bulk_wait_group_read0();
        mbar_arrive(bar(M::kDOEmpty + n % M::kDOs));
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait_group0();
    // key blocks that no query meets (behind the sequence): 0
    for (int idx = blockIdx.x; idx < p.items; idx += gridDim.x) {
      const KvItem w = kv_item(p, idx);
      if (w.it0 < w.it1 || w.nparts > 1 || w.kb * kBlk + j >= p.T) continue;
      const long long tok = static_cast<long long>(w.b) * p.T + w.kb * kBlk + j;
      const size_t c = static_cast<size_t>(w.kvh) * kD;
#pragma unroll 1
      for (int u = 0; u < kD / 8; ++u) {
        reinterpret_cast<uint4 *>(p.dv + tok * p.dv_stride + c)[u] = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4 *>(p.dk + tok * p.dk_stride + c)[u] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 2) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------- join
// Parts of the key blocks that went to several CTAs, summed in their order: four
// components of dV or dK per thread, with all its loads under way at one time (a block
// for each 32 keys that goes through them took 11 us of a layer's 33, this 5 of 28).  Runs
// beside the dq kernel, which lets it start once the kv kernel has completed.
constexpr int kJoinThr = 256;
template <int kD>
constexpr int kJoinBlocks = 4 * 2 * 32 * (kD / 4) / kJoinThr;   // per (batch, KV head, key block)

template <int kD>
__global__ void __launch_bounds__(kJoinThr) window_join_kernel(const __grid_constant__ BwdParams p) {
  const int nk = p.parts_each > 1 ? p.g.nb : p.g.first;   // key blocks with parts
  const int sub = blockIdx.x % kJoinBlocks<kD>, block = blockIdx.x / kJoinBlocks<kD>;
  const int unit = block / nk, kb = block - unit * nk;
  const int group = unit / p.group * p.group, width = min(p.group, p.units - group);
  const int idx = kb < p.g.first ? kb * p.first_parts * p.units + unit
                                 : p.lead_items + group * p.per_unit + (kb - p.g.first) * p.parts_each * width + unit - group;
  const KvItem w = kv_item(p, idx);
  // of fewer pairs than parts only the first parts have one and were written
  const int all = p.G * w.qn;
  const int e = sub * kJoinThr + threadIdx.x, r = e % kBlk, c = e / kBlk % (kD / 4), x = e / kBlk / (kD / 4);
  const int tok = kb * kBlk + r;
  if (tok < p.T) {
    const float4 *src = reinterpret_cast<const float4 *>(p.parts) + ((w.slot * 2 + x) * (kD / 4) + c) * kBlk + r;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const int n = min(w.nparts, all);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float4 v = __ldcg(src + static_cast<size_t>(i) * 2 * (kD / 4) * kBlk);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const long long at = static_cast<long long>(w.b) * p.T + tok;
    __nv_bfloat16 *dst = (x == 0 ? p.dv + at * p.dv_stride : p.dk + at * p.dk_stride) + static_cast<size_t>(w.kvh) * kD + 4 * c;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
  }
  // what follows on the stream follows the dq kernel too
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------------ dq
template <int kD>
struct DqSmem {
  static constexpr int kK = kBlk * kD * 2, kStage = kK + kTileBytes, kStages = 3;
  static constexpr int kOut = kStages * kStage;              // 4 KB per epilogue warp
  static constexpr int kBar = kOut + 8 * 4096;
  enum { kFull = 0, kEmpty = kStages, kAccFull = 2 * kStages, kAccEmpty = kAccFull + 2, kRaw = kAccEmpty + 2, kFinal, kBars };
  static constexpr int kTmem = kBar + kBars * 8, kAbort = kTmem + 4;
  static constexpr int kBytes = kAbort + 4 + 1024;
  static_assert(kBytes <= 232448, "dq kernel shared memory");
};

struct DqItem {
  int b, h, m, n, lo, lead, steps;
  __device__ __forceinline__ int block(int x) const { return x < lead ? x : lo + (x - lead); }
};
__device__ __forceinline__ DqItem dq_item(const BwdParams &p, int idx) {
  DqItem r;
  idx = p.dq_items - 1 - idx;
  const int unit = p.by_dq_group(idx) * p.group;   // idx becomes the place in the group
  r.m = unit + p.group <= p.units ? p.by_dq_width(idx) : p.by_dq_last(idx);
  r.h = unit * p.G + idx;
  r.b = p.by_hq(r.h);
  r.n = tokens_warp(p.lengths, r.b, p.T);
  r.lo = p.g.lo(r.m);
  r.lead = p.g.lead(r.m);
  r.steps = r.m * kBlk < r.n ? r.lead + r.m - r.lo + 1 : 0;
  return r;
}

template <int kD>
__global__ void __launch_bounds__(kThr, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmdQ,
                     const __grid_constant__ BwdParams p) {
  using M = DqSmem<kD>;
  constexpr int kHalves = kD / 64;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  auto bar = [&](int i) -> uint32_t { return sb + M::kBar + i * 8; };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + M::kAbort);
  const Waits wts{sb + M::kBar, abort_flag, &p.wait, kSiteWinDq};
  auto wtw = [&](int slot, uint32_t parity) -> bool { return wait_warp(wts, slot, parity); };

  if (tid == 0) {
    for (int i = 0; i < M::kBars; ++i) mbar_init(bar(i), i == M::kAccEmpty || i == M::kAccEmpty + 1 ? 128 * kHalves : 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2) tc::tmem_alloc(sb + M::kTmem, 2 * kD);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(smem + M::kTmem), 0);

  if (warp == 0) {
    // ============================ loads ================================
    if (lane == 0) prefetch_tensormap(&tmK);
    const uint64_t keep = l2_evict_last(), stream = l2_evict_first();
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the dS tiles come from the kv kernel
    // the join may start beside this kernel: what it reads is there, and it waits for
    // this grid behind its work
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int g = 0, raw = 0;
    bool ok = true;
    for (int round = 0, idx = nth_item(0); ok && round * static_cast<int>(gridDim.x) < p.dq_items; idx = nth_item(++round)) {
      if (idx >= p.dq_items) continue;
      const DqItem w = dq_item(p, idx);
      int rest = w.h;
      const int kvh = p.by_g(rest);
      const unsigned char *tiles = reinterpret_cast<const unsigned char *>(p.ds) +
                                   (static_cast<long long>(w.b) * p.Hq + w.h) * p.tiles * kTileBytes;
      for (int x = 0; x < w.steps; ++x, ++g) {
        const int s = g % M::kStages, kb = w.block(x);
        ok = wtw(M::kEmpty + s, ((g / M::kStages) & 1) ^ 1);
        if (!ok) break;
        const uint32_t st = sb + s * M::kStage;
        const int live = w.n - kb * kBlk;
        const bool repair = live < kBlk && w.n < p.T;      // rows of K behind the last token: cleared
        const uint32_t fb = bar(repair ? M::kRaw : M::kFull + s);
        if (lane == 0) {
          mbar_arrive_expect_tx(fb, M::kStage);
          for (int hx = 0; hx < kHalves; ++hx)
            tma_load_4d_hint(st + hx * 16384, &tmK, hx * 64, kvh, kb * kBlk, w.b, fb, keep);
          bulk_load_hint(st + M::kK, tiles + (p.g.tile0(kb) + (w.m - kb)) * kTileBytes, kTileBytes, fb, stream);
        }
        if (repair) clear_tail<kHalves>(wts, smem + s * M::kStage, live, M::kRaw, raw++ & 1, bar(M::kFull + s));
      }
    }
    // the last copy of every slot has landed before the CTA may end
    for (int i = max(g - M::kStages, 0); i < g; ++i)
      wait_landed(bar(M::kFull + i % M::kStages), (i / M::kStages) & 1);
  } else if (warp == 1) {
    // ============================ products =============================
    constexpr uint32_t id = tc::idesc_bf16_f32(128, kD, 1, 1);              // dQ += dS K, both MN-major
    const uint64_t dS = tc::sdesc_sw128(sb + M::kK, kTileBytes / 2, 1024);  // queries contiguous
    const uint64_t dK = tc::sdesc_sw128(sb, 16384, 1024);
    int g = 0, j = 0, gave_up = 0;
    auto wti = [&](int slot, uint32_t parity) -> bool { return wait_issuer(wts, slot, parity, gave_up); };
    bool ok = may_wait(p.wait, abort_flag, kSiteWinDq, M::kFull);
    for (int round = 0, idx = nth_item(0); ok && round * static_cast<int>(gridDim.x) < p.dq_items; idx = nth_item(++round)) {
      if (idx >= p.dq_items) continue;
      const DqItem w = dq_item(p, idx);
      if (w.steps == 0) continue;
      const int a = j & 1;
      if (!wti(M::kAccEmpty + a, ((j >> 1) & 1) ^ 1)) break;
      tc::fence_after_sync();
      for (int x = 0; x < w.steps; ++x, ++g) {
        const int s = g % M::kStages;
        ok = wti(M::kFull + s, (g / M::kStages) & 1);
        if (!ok) break;
        tc::fence_after_sync();
        const uint64_t so = static_cast<uint64_t>(s * M::kStage) >> 4;
        if (tc::elect()) {
          tc::product_mn(tmem + a * kD, dS + so, dK + so, id, x > 0);
          tc::commit(bar(M::kEmpty + s));
          if (x == w.steps - 1) tc::commit(bar(M::kAccFull + a));
        }
        __syncwarp();
      }
      ++j;
    }
    tc::commit_w(bar(M::kFinal));
    report_issuer(wts, gave_up);
    wait_landed(bar(M::kFinal), 0);   // every product has completed
  } else if (warp >= 4 && warp < 4 + 4 * kHalves) {
    // ============================ epilogue ================================
    // Warp w: queries 32 (w % 4) .. of the block, 64 components
    const int qd = warp & 3, hx = (warp - 4) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
    unsigned char *stage = smem + M::kOut + (warp - 4) * 4096;
    int j = 0;
    for (int round = 0, idx = nth_item(0); round * static_cast<int>(gridDim.x) < p.dq_items; idx = nth_item(++round)) {
      if (idx >= p.dq_items) continue;
      const DqItem w = dq_item(p, idx);
      const int a = j & 1, row = w.m * kBlk + 32 * qd + lane;
      if (w.steps > 0) {
        if (!wtw(M::kAccFull + a, (j >> 1) & 1)) break;
        tc::fence_after_sync();
        ++j;
      }
      float v[2][32];
      if (w.steps > 0) {
        tc::ld32x2_wait(tmem + lanes + a * kD + 64 * hx, tmem + lanes + a * kD + 64 * hx + 32, v[0], v[1]);
        tc::fence_before_sync();
        mbar_arrive(bar(M::kAccEmpty + a));
      }
      if (lane == 0) bulk_wait_group_read0();              // the copy before has read the buffer
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float *y = &v[u >> 2][8 * (u & 3)];
        uint4 x = make_uint4(pack_bf16(y[0] * p.scale, y[1] * p.scale), pack_bf16(y[2] * p.scale, y[3] * p.scale),
                             pack_bf16(y[4] * p.scale, y[5] * p.scale), pack_bf16(y[6] * p.scale, y[7] * p.scale));
        if (row >= w.n) x = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) = x;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && w.m * kBlk + 32 * qd < p.T) {
        tma_store_4d(&tmdQ, sb + M::kOut + (warp - 4) * 4096, hx * 64, w.h, w.m * kBlk + 32 * qd, w.b);
        bulk_commit_group();
      }
    }
    if (lane == 0) bulk_wait_group_read0();
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 2) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 2 * kD);
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Sizes that the launch and the workspace share.
struct BwdSizes {
  Grid g;
  int Tp, first_parts, parts_each, per_unit, slots;
  long long tiles, first_pairs, each_pairs;   // dS tiles per head; pairs of an item, at most
  size_t stats, ds, parts;   // bytes
};

BwdSizes bwd_sizes(int B, int T, int Hq, int Hkv, int D, int window, int sinks) {
  BwdSizes s;
  s.g = grid_of(T, window, sinks);
  const Grid &g = s.g;
  const int G = Hq / Hkv;
  const long long units = static_cast<long long>(B) * Hkv;
  s.Tp = g.nb * kBlk;
  s.tiles = g.tile0(g.nb);
  // Pairs per item: a key block's own while there are items enough to fill 152 SMs
  // twice, else an equal share of all pairs, at least 2.  The first tokens' blocks
  // have more pairs and are cut to an equal share of all.
  const long long each = static_cast<long long>(G) * std::min(g.nb, g.wq), total = units * G * s.tiles;
  const long long share = std::max(2LL, (total + 151) / 152), most = units * g.nb >= 304 ? each : std::min(each, share);
  s.parts_each = static_cast<int>((each + most - 1) / most);
  s.first_pairs = static_cast<long long>(G) * g.nb;
  s.first_parts = static_cast<int>((s.first_pairs + share - 1) / share);
  s.each_pairs = (each + s.parts_each - 1) / s.parts_each;
  s.first_pairs = (s.first_pairs + s.first_parts - 1) / s.first_parts;
  s.per_unit = (g.nb - g.first) * s.parts_each;
  s.slots = (s.first_parts > 1 ? g.first * s.first_parts : 0) + (s.parts_each > 1 ? (g.nb - g.first) * s.parts_each : 0);
  s.stats = up256(static_cast<size_t>(B) * Hq * s.Tp * 4);
  s.ds = static_cast<size_t>(B) * Hq * s.tiles * kTileBytes;
  s.parts = static_cast<size_t>(units) * s.slots * 2 * kBlk * D * 4;
  return s;
}

template <int kD>
cudaError_t launch(const WindowArgs &a, BwdParams &p, const BwdSizes &s, int sms, cudaStream_t st, const char **why) {
  CUtensorMap q, dout, k, v, dq, dk, dv;
  if (!token_map(&q, a.q, a.Hq, a.T, a.B, kD, a.q_stride, kBlk, why) ||
      !token_map(&dout, a.dout, a.Hq, a.T, a.B, kD, a.dout_stride, kBlk, why) ||
      !token_map(&k, a.k, a.Hkv, a.T, a.B, kD, a.k_stride, kBlk, why) ||
      !token_map(&v, a.v, a.Hkv, a.T, a.B, kD, a.v_stride, kBlk, why) ||
      !token_map(&dq, a.dq, a.Hq, a.T, a.B, kD, a.dq_stride, 32, why) ||
      !token_map(&dk, a.dk, a.Hkv, a.T, a.B, kD, a.dk_stride, 32, why) ||
      !token_map(&dv, a.dv, a.Hkv, a.T, a.B, kD, a.dv_stride, 32, why))
    return cudaErrorInvalidValue;
  const void *kv_fn = reinterpret_cast<const void *>(window_kv_kernel<kD>);
  const void *dq_fn = reinterpret_cast<const void *>(window_dq_kernel<kD>);
  cudaError_t e = ensure_dynamic_smem(kv_fn, KvSmem<kD>::kBytes);
  if (e == cudaSuccess) e = ensure_dynamic_smem(dq_fn, DqSmem<kD>::kBytes);
  if (e != cudaSuccess) return e;
  const int chunks = s.Tp / kPrepTokens<kD>;   // whole ones: Tp is a multiple of 128
  p.by_chunks = Div::by(chunks);
  const long long blocks = static_cast<long long>(a.B) * chunks * a.Hq;
  if (blocks > 0x7fffffffLL) {
    *why = "grid too large";
    return cudaErrorNotSupported;
  }
  window_prep_kernel<kD><<<static_cast<unsigned>(blocks), kPrepThr, 0, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kKvThr);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(std::min(p.items, sms));
  cfg.dynamicSmemBytes = KvSmem<kD>::kBytes;
  e = cudaLaunchKernelEx(&cfg, window_kv_kernel<kD>, q, dout, k, v, dk, dv, p);
  if (e != cudaSuccess) return e;
  cfg.blockDim = dim3(kThr);
  cfg.gridDim = dim3(std::min(p.dq_items, sms));
  cfg.dynamicSmemBytes = DqSmem<kD>::kBytes;
  e = cudaLaunchKernelEx(&cfg, window_dq_kernel<kD>, k, dq, p);
  if (e != cudaSuccess) return e;
  if (s.slots > 0) {
    const int nk = s.parts_each > 1 ? s.g.nb : s.g.first;
    cfg.gridDim = dim3(a.B * a.Hkv * nk * kJoinBlocks<kD>);
    cfg.blockDim = dim3(kJoinThr);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, window_join_kernel<kD>, p);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

// The dS tiles of a call may be more than a card holds (one sequence of 131,072 tokens, 32
// heads, window 1024: 10 GB; all keys: 550 GB), so a call goes through its (batch, KV head)s
// in slabs of at most this much: whole sequences, or KV heads of one.  Calls of 2.1 to 8.3 GB,
// us at 256 MB, 512 MB, 1 GB, 2 GB and in one go: 1 x 8192 tokens of 32 heads, all keys, 1727,
// 1318, 1210, 1202, 1210; 1 x 32768 of 32, window 4096, 5630, 5225, 4700, 4550, 4590; 1 x 65536
// of 16, window 1024, 1990, 1832, 1725, 1689, 1681: a slab's last CTAs end alone.
constexpr long long kSlabBytes = 2LL << 30;

struct Slab {
  int seqs, heads;   // sequences with all KV heads, or KV heads of one sequence
};
Slab slab_of(int B, int T, int Hq, int Hkv, int window, int sinks) {
  const Grid g = grid_of(T, window, sinks);
  const long long head = g.tile0(g.nb) * kTileBytes * (Hq / Hkv), fit = std::max(1LL, kSlabBytes / head);
  auto even = [](long long n, long long most) {   // of as many slabs of at most `most` as it takes, the size of one
    const long long slabs = (n + most - 1) / most;
    return static_cast<int>((n + slabs - 1) / slabs);
  };
  return fit >= Hkv ? Slab{even(B, fit / Hkv), Hkv} : Slab{1, even(Hkv, fit)};
}

// The call on sequences b .. b + seqs - 1 and KV heads h .. h + heads - 1 (all of them, or one sequence).
WindowArgs part_of(const WindowArgs &a, long long b, long long seqs, long long h, long long heads) {
  const int G = a.Hq / a.Hkv;
  const long long tok = b * a.T, qh = h * G;
  auto at = [&](const void *x, long long stride, long long head) {
    return static_cast<const __nv_bfloat16 *>(x) + tok * stride + head * a.D;
  };
  auto out = [&](void *x, long long stride, long long head) { return const_cast<__nv_bfloat16 *>(at(x, stride, head)); };
  WindowArgs r = a;
  r.q = at(a.q, a.q_stride, qh), r.dout = at(a.dout, a.dout_stride, qh);
  r.k = at(a.k, a.k_stride, h), r.v = at(a.v, a.v_stride, h);
  r.o = out(a.o, a.o_stride, qh), r.dq = out(a.dq, a.dq_stride, qh);
  r.dk = out(a.dk, a.dk_stride, h), r.dv = out(a.dv, a.dv_stride, h);
  r.lse = a.lse + (b * a.Hq + qh) * a.T;
  if (a.lengths) r.lengths = a.lengths + b;
  r.B = static_cast<int>(seqs), r.Hq = static_cast<int>(heads * G), r.Hkv = static_cast<int>(heads);
  return r;
}

cudaError_t launch_slab(const WindowArgs &a, const WaitCtl &w, int sms, cudaStream_t st, const char **why) {
  const BwdSizes s = bwd_sizes(a.B, a.T, a.Hq, a.Hkv, a.D, a.window, a.sinks);
  const long long units = static_cast<long long>(a.B) * a.Hkv, lead_items = units * s.g.first * s.first_parts;
  const long long items = lead_items + units * s.per_unit;
  const long long dq_items = static_cast<long long>(a.B) * a.Hq * s.g.nb;
  if (items > 0x03ffffffLL || dq_items > 0x1fffffffLL) {   // the join's grid is up to 32 times the items
    *why = "grid too large";
    return cudaErrorNotSupported;
  }
  BwdParams p;
  p.o = static_cast<const __nv_bfloat16 *>(a.o), p.dout = static_cast<const __nv_bfloat16 *>(a.dout);
  p.lse = a.lse, p.lengths = a.lengths;
  unsigned char *ws = static_cast<unsigned char *>(a.ws);
  ws += (256 - (reinterpret_cast<uintptr_t>(ws) & 255)) & 255;
  p.ndelta = reinterpret_cast<float *>(ws);
  p.nlse2 = reinterpret_cast<float *>(ws + s.stats);
  p.ds = reinterpret_cast<__nv_bfloat16 *>(ws + 2 * s.stats);
  p.parts = reinterpret_cast<float *>(ws + 2 * s.stats + s.ds);
  p.dq = static_cast<__nv_bfloat16 *>(a.dq);
  p.dk = static_cast<__nv_bfloat16 *>(a.dk), p.dv = static_cast<__nv_bfloat16 *>(a.dv);
  p.B = a.B, p.T = a.T, p.Tp = s.Tp, p.Hq = a.Hq, p.Hkv = a.Hkv, p.G = a.Hq / a.Hkv;
  p.o_stride = a.o_stride, p.dout_stride = a.dout_stride, p.dk_stride = a.dk_stride, p.dv_stride = a.dv_stride;
  p.tiles = s.tiles;
  p.g = s.g;
  p.first_parts = s.first_parts, p.parts_each = s.parts_each, p.per_unit = s.per_unit, p.slots = s.slots;
  p.items = static_cast<int>(items), p.dq_items = static_cast<int>(dq_items);
  p.units = static_cast<int>(units), p.lead_items = static_cast<int>(lead_items);
  const int grid = std::min(p.items, sms);
  p.lead_rounds = p.lead_items / grid, p.lead_rest = p.lead_items % grid;
  p.span = static_cast<int>(std::min((s.first_pairs + s.each_pairs / 2) / s.each_pairs, 1LL * (p.items / grid + 1)));
  p.rounds = p.lead_rounds + 1 + p.span + (p.items - p.lead_items + grid - 1) / grid;
  // Units of a group: what the blocks of keys that are worked on at one time meet of
  // q and dout is to stay in L2
  const long long meets = static_cast<long long>(p.G) * (s.g.wq + 1) * kBlk * a.D * 4;
  p.group = p.items <= grid ? 1 : static_cast<int>(std::max(1LL, std::min<long long>(p.units, kGroupBytes / meets)));
  const int last = (p.units - 1) % p.group + 1;
  p.by_units = Div::by(p.units), p.by_group = Div::by(std::max(1, p.group * s.per_unit)), p.by_width = Div::by(p.group), p.by_last = Div::by(last);
  p.by_dq_group = Div::by(p.group * p.G * s.g.nb), p.by_dq_width = Div::by(p.group * p.G), p.by_dq_last = Div::by(last * p.G);
  p.by_hkv = Div::by(a.Hkv);
  p.by_first = Div::by(s.first_parts), p.by_each = Div::by(s.parts_each);
  p.by_hq = Div::by(a.Hq), p.by_g = Div::by(p.G);
  p.scale = a.scale;
  p.wait = w;
  return a.D == 64 ? launch<64>(a, p, s, sms, st, why) : launch<128>(a, p, s, sms, st, why);
}

}  // namespace

size_t window_bwd_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int window, int sinks) {
  const Slab s = slab_of(B, T, Hq, Hkv, window, sinks);
  const int G = Hq / Hkv;
  size_t most = 0;
  for (int seqs : {s.seqs, (B - 1) % s.seqs + 1})                     // a slab, the last one
    for (int heads : {s.heads, (Hkv - 1) % s.heads + 1}) {
      const BwdSizes z = bwd_sizes(seqs, T, heads * G, heads, D, window, sinks);
      most = std::max(most, 256 + 2 * z.stats + z.ds + z.parts);
    }
  return most;
}

cudaError_t launch_window_bwd(const WindowArgs &a, const WaitCtl &w, cudaStream_t st, const char **why) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const Slab s = slab_of(a.B, a.T, a.Hq, a.Hkv, a.window, a.sinks);
  for (long long b = 0; b < a.B; b += s.seqs)
    for (long long h = 0; e == cudaSuccess && h < a.Hkv; h += s.heads)
      e = launch_slab(part_of(a, b, std::min<long long>(s.seqs, a.B - b), h, std::min<long long>(s.heads, a.Hkv - h)), w, sms, st, why);
  return e;
}

}  // namespace abw
