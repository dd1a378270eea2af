// Softmax attention over a sliding window with first tokens that stay visible,
// forward: query i sees key j where j <= i and (j > i - window or j < sinks).
//
// Per query row, over blocks of 128 keys: m = running max, l = running sum of
// 2^(s - m) (base-2 units, fp32), O = running sum of 2^(s - m) v in TMEM.  The
// rescale is lazy: m moves only when a block's max exceeds it by more than 8, so
// P <= 2^8 between rescales.  O / l and (m + log2 l) ln 2 come out.
//
// One persistent CTA per SM works on two tiles of 128 queries at once, in turn:
// while the softmax warps of one form P, the tensor core runs the products of the
// other.  The tiles share their K and V blocks: two heads of a KV head where the
// group is even, else two neighbouring blocks of queries.  Only blocks that a
// tile meets are multiplied: the window's, and the first tokens' in front of it.
//   S = Q K^T   M=128 queries, N=128 keys      (TMEM [0,128) and [128,256))
//   O += P V    M=128 queries, N=D, A = P in TMEM over S   (behind [256, ..))
// Order of the products, block after block: per tile PV of its last block, then
// S of the next, so S (and Q, O) need one buffer per tile; the order runs on
// over the CTA's items.
// Warps: 0 loads (K, V through a ring, Q per tile), 1 issues products, 4-7 and 8-11
// softmax of tile 0 and 1, 12-15 outputs (thread = query row).
// Padding behind a sequence is not looked at: its keys are never visible, and
// its rows of V, which meet weights of 0, are cleared in shared memory.
//
// 8192 tokens of 32 heads, window 1024: 136 us, 950 TFLOP/s of the visible pairs; all
// keys 390 us, 1400 TFLOP/s.  What bounds it is the softmax warps' chain.  A block of 128
// x 128 at D = 128 is 1024 cycles of products and 512 of exponentials (32 a cycle and SM),
// which run beside one another: the first call's 125 blocks a CTA are 68 us of the one
// and 34 of the other at 1.9 GHz.  A whole block more takes 0.81 us, some 1,500 cycles
// (the two calls' difference): its scores come out of TMEM one and a half times (128
// registers a thread do not hold a row of them), are converted and go back, each step
// behind a wait.  34 of the 136 us are what cut blocks' masks and the changes of item
// cost on top.  (With the softmax taken out the kernel took 100 us, with the products
// out 124: each with the other waits still in place.)  What measured no better: an
// issuer per tile, eight softmax warps per tile, cut blocks 32 columns at a time,
// prefetches of the next queries into L2, outputs read out of TMEM before they are staged.
#include <algorithm>

#include "window.cuh"

namespace abw {
namespace {

using namespace win;

constexpr int kThr = 512;
constexpr float kRescale = 8.f;       // lazy-rescale threshold (base-2 units)
// K and V that a scheduling group's tiles meet at one time: many head units, so that the
// CTAs' sums come out alike (8192 tokens of 32 heads, all keys: 36 MB 666, 72 480, 144 389
// us), but not all of them (16 x 4096 tokens: 144 MB 1.73, no groups 1.81 ms).
constexpr long long kGroupBytes = 144 << 20;

template <int kD>
struct FwdSmem {
  static constexpr int kTile = kBlk * kD * 2;               // one block of Q, K or V
  static constexpr int kStages = kD == 128 ? 4 : 8;
  static constexpr int kQ = 0;                              // two tiles
  static constexpr int kRing = 2 * kTile;
  static constexpr int kOut = kRing + kStages * kTile;      // 4 KB per output warp: 32 rows x 64 components
  static constexpr int kStat = kOut + 4 * 4096;             // [tile][128] (m, l)
  static constexpr int kBar = kStat + 2048;
  enum {
    kQFull = 0, kQEmpty = 2, kSFull = 4, kOFull = 6, kPFull = 8, kOEmpty = 10, kLFull = 12, kLEmpty = 14, kRaw = 16,
    kFinal = 17, kKVFull = 18,
    kKVEmpty = kKVFull + kStages, kBars = kKVEmpty + kStages
  };
  static constexpr int kTmem = kBar + kBars * 8, kAbort = kTmem + 4;
  static constexpr int kBytes = kAbort + 4 + 1024;          // + alignment slack
  static_assert(kBytes <= 232448, "forward kernel shared memory");
};

struct FwdParams {
  float *lse;
  const int *lengths;
  int B, T, Hq, Hkv, G, nqb, per_head, units, group, items;
  Div by_group, by_width, by_last, by_heads, by_g;   // items of a scheduling group, its width (the last one's), head units, G
  int pair_heads;         // tiles: 1 two heads of a group, 0 two blocks of queries
  int window, sinks, sink_blocks;
  float scale;
  WaitCtl wait;
};

// A tile and its blocks of keys, in the order of the products: `lead` blocks of
// first tokens in front of the window's, lo .. hi; hi < 0: no block.
struct Tile {
  int h, q0, lo, hi, lead;
  bool exists;
  __device__ __forceinline__ int steps() const { return hi < 0 ? 0 : lead + hi - lo + 1; }
  __device__ __forceinline__ int block(int x) const { return x < lead ? x : lo + (x - lead); }
  __device__ __forceinline__ bool meets(int n) const { return n <= hi && (n >= lo || n < lead); }
};
struct Unit {
  int b, u, m, n;   // batch, head unit, place along the queries, tokens
};

__device__ __forceinline__ Unit unit_of(const FwdParams &p, int it) {
  // (batch, head unit) in groups; in a group the late blocks of queries first, so that
  // what runs at one time shares K and V in L2 and the short items come last
  Unit r;
  const int first = p.by_group(it) * p.group;   // `it` becomes the place in the group
  const int m = first + p.group <= p.units ? p.by_width(it) : p.by_last(it);
  r.m = p.per_head - 1 - m;
  r.u = first + it;
  r.b = p.by_heads(r.u);
  r.n = tokens_warp(p.lengths, r.b, p.T);
  return r;
}
__device__ __forceinline__ Tile tile_of(const FwdParams &p, const Unit &w, int t) {
  Tile x;
  const int blk = p.pair_heads ? w.m : 2 * w.m + t;
  x.h = p.pair_heads ? 2 * w.u + t : w.u;
  x.q0 = blk * kBlk;
  x.exists = blk < p.nqb;
  x.hi = x.exists && x.q0 < w.n ? blk : -1;
  x.lo = max(0, x.q0 - p.window + 1) / kBlk;
  x.lead = min(p.sink_blocks, x.lo);
  return x;
}
// The blocks of both tiles: tile 1 meets all that tile 0 meets in front of the
// window's, and no window begins more than a block behind the other's.
__device__ __forceinline__ Tile both_tiles(const Tile &a, const Tile &b) {
  Tile x = a;
  if (b.hi >= 0) {
    x.hi = b.hi;            // where b is there, so is a, and not behind it
    x.lo = min(a.lo, b.lo);
    x.lead = min(a.lead, b.lead);
  }
  return x;
}

template <int kD>
__global__ void __launch_bounds__(kThr, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                      const __grid_constant__ FwdParams p) {
  using M = FwdSmem<kD>;
  constexpr int kHalves = kD / 64;
  constexpr uint32_t kColO = 256;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  auto bar = [&](int i) -> uint32_t { return sb + M::kBar + i * 8; };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + M::kAbort);
  const Waits wts{sb + M::kBar, abort_flag, &p.wait, kSiteWinFwd};
  auto wtw = [&](int slot, uint32_t parity) -> bool { return wait_warp(wts, slot, parity); };

  if (tid == 0) {
    for (int i = 0; i < M::kBars; ++i)
      mbar_init(bar(i), i >= M::kPFull && i < M::kRaw ? 128 : 1);   // threads of a warpgroup
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(sb + M::kTmem, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(smem + M::kTmem), 0);

  if (warp < 4) {
    if (warp == 0) {
      // ============================ loads ================================
      if (lane == 0) {
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
      }
      int r = 0, raw = 0, nq[2] = {0, 0};   // ring position, repaired blocks, Q tiles so far
      bool ok = true;
      for (int rd = 0; ok; ++rd) {
        const int it = nth_item(rd);
        if (it >= p.items) break;
        const Unit w = unit_of(p, it);
        const Tile t0 = tile_of(p, w, 0), t1 = tile_of(p, w, 1), all = both_tiles(t0, t1);
        int rest = t0.h;
        const int kvh = p.by_g(rest);
        auto load = [&](const CUtensorMap *map, int n, bool value) -> bool {
          const int s = r % M::kStages;
          if (!wtw(M::kKVEmpty + s, ((r / M::kStages) & 1) ^ 1)) return false;
          const uint32_t dst = sb + M::kRing + s * M::kTile;
          // rows of V behind the sequence's last token: cleared before the products see them
          const int live = w.n - n * kBlk;
          const bool repair = value && live < kBlk && w.n < p.T;
          const uint32_t fb = bar(repair ? M::kRaw : M::kKVFull + s);
          if (lane == 0) {
            mbar_arrive_expect_tx(fb, M::kTile);
            for (int hx = 0; hx < kHalves; ++hx) tma_load_4d(dst + hx * 16384, map, hx * 64, kvh, n * kBlk, w.b, fb);
          }
          ++r;
          if (repair)
            clear_tail<kHalves>(wts, smem + M::kRing + s * M::kTile, live, M::kRaw, raw++ & 1, bar(M::kKVFull + s));
          return true;
        };
        for (int x = 0; ok && x < all.steps(); ++x) {
          const int n = all.block(x);
          ok = load(&tmK, n, false);
          for (int t = 0; ok && x == 0 && t < 2; ++t) {
            const Tile &tile = t == 0 ? t0 : t1;
            if (tile.hi < 0) continue;
            ok = wtw(M::kQEmpty + t, (nq[t] & 1) ^ 1);
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(bar(M::kQFull + t), M::kTile);
              for (int hx = 0; hx < kHalves; ++hx)
                tma_load_4d(sb + M::kQ + t * M::kTile + hx * 16384, &tmQ, hx * 64, tile.h, tile.q0, w.b, bar(M::kQFull + t));
            }
            ++nq[t];
          }
          if (ok) ok = load(&tmV, n, true);
        }
      }
      // The last copy of every slot has landed before the block may end, whoever gives
      // up and when (otherwise this finds every phase complete).
      for (int i = max(r - M::kStages, 0); i < r; ++i)
        wait_landed(bar(M::kKVFull + i % M::kStages), (i / M::kStages) & 1);
      for (int t = 0; t < 2; ++t)
        if (nq[t] > 0) wait_landed(bar(M::kQFull + t), (nq[t] - 1) & 1);
    } else if (warp == 1) {
      // ============================ products =============================
      // S = Q K^T, both K-major; -Q K^T where the scale is negative
      const uint32_t id_s = tc::idesc_bf16_f32(128, 128, 0, 0) | (p.scale < 0.f ? tc::kNegateA : 0u);
      constexpr uint32_t id_o = tc::idesc_bf16_f32(128, kD, 0, 1);    // O += P V, V MN-major
      const uint64_t dQ = tc::sdesc_sw128(sb + M::kQ, 16, 1024);
      const uint64_t dK = tc::sdesc_sw128(sb + M::kRing, 16, 1024);
      const uint64_t dV = tc::sdesc_sw128(sb + M::kRing, 16384, 1024);
      int gave_up = 0;
      auto wti = [&](int slot, uint32_t parity) -> bool { return wait_issuer(wts, slot, parity, gave_up); };
      auto slot = [](int r) -> uint64_t { return static_cast<uint64_t>((r % M::kStages) * M::kTile) >> 4; };
      int r = 0;                    // ring position of the next K block; its V block follows
      int vr = 0;                   // ring position of the V block that the PV products to come read
      // bit t: a PV product of tile t is to come, it is its output's first, its last;
      // and the parities of its P tiles, outputs and Q tiles
      uint32_t pend = 0, opens = 0, closes = 0, np = 0, ni = 0, nq = 0;
      bool ok = may_wait(p.wait, abort_flag, kSiteWinFwd, M::kQFull);
      int rd = 0, x = 0;
      Unit w = {};
      Tile ta = {}, tb = {}, all = {};
      all.hi = -1;
      uint32_t begun = 0;
      // Steps: the blocks of the items, one after the other, and a last one for the
      // products that are still to come.  In each, per tile: PV of the tile's block
      // before, then S of this one.
      for (bool more = true; ok && more;) {
        if (x >= all.steps()) {
          x = 0;
          begun = 0;
          const int it = nth_item(rd++);
          more = it < p.items;
          all.hi = -1;
          if (more) {
            w = unit_of(p, it);
            ta = tile_of(p, w, 0);
            tb = tile_of(p, w, 1);
            all = both_tiles(ta, tb);
            if (all.hi < 0) continue;
          }
        }
        const int n = more ? all.block(x) : 0;
#pragma unroll 1
        for (int t = 0; ok && t < 2; ++t) {
          const uint32_t bit = 1u << t;
          const int hi = t ? tb.hi : ta.hi;
          if (pend & bit) {         // O_t += P_t V
            ok = wti(M::kKVFull + vr % M::kStages, (vr / M::kStages) & 1) &&
                 (!(opens & bit) || wti(M::kOEmpty + t, ((ni >> t) & 1) ^ 1)) && wti(M::kPFull + t, (np >> t) & 1);
            if (!ok) break;
            tc::fence_after_sync();
            if (tc::elect()) {
              tc::product_ts<8, 0>(tmem + kColO + t * kD, tmem + t * 128 + 64, dV + slot(vr), id_o, !(opens & bit));
              if (closes & bit) tc::commit(bar(M::kOFull + t));
              // both tiles are through with the V block
              if (t == 1 || !(pend & 2u)) tc::commit(bar(M::kKVEmpty + vr % M::kStages));
            }
            __syncwarp();
            np ^= bit;
            if (closes & bit) ni ^= bit;
            pend &= ~bit;
          }
          if (!more || !(t ? tb : ta).meets(n)) continue;
          const bool first = !(begun & bit);
          ok = (!first || wti(M::kQFull + t, (nq >> t) & 1)) && wti(M::kKVFull + r % M::kStages, (r / M::kStages) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          if (tc::elect()) {
            tc::product_k<kD>(tmem + t * 128, dQ + (static_cast<uint64_t>(t * M::kTile) >> 4), dK + slot(r), id_s);
            tc::commit(bar(M::kSFull + t));
            if (n == hi) tc::commit(bar(M::kQEmpty + t));
            // both tiles are through with the K block
            if (t == 1 || !tb.meets(n)) tc::commit(bar(M::kKVEmpty + r % M::kStages));
          }
          __syncwarp();
          pend |= bit;
          opens = first ? opens | bit : opens & ~bit;
          begun |= bit;
          if (first) nq ^= bit;
          closes = n == hi ? closes | bit : closes & ~bit;
        }
        if (!ok || !more) break;
        vr = r + 1;
        r += 2;
        ++x;
      }
      tc::commit_w(bar(M::kFinal));
      report_issuer(wts, gave_up);
      wait_landed(bar(M::kFinal), 0);   // every product has completed
    }
  } else if (warp < 12) {
    // ============================ softmax ================================
    const int t = (warp >> 2) - 1;                      // tile
    const int qd = warp & 3;                            // TMEM lane quarter
    const int row = 32 * qd + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
    const uint32_t tS = tmem + lanes + t * 128, tO = tmem + lanes + kColO + t * kD;
    const float sl2 = fabsf(p.scale) * kLog2e;          // scores in base-2 units
    float2 *stat = reinterpret_cast<float2 *>(smem + M::kStat) + t * 128 + row;
    int ns = 0, no = 0;                                 // S tiles, outputs so far
    bool ok = true;
    for (int rd = 0; ok; ++rd) {
        const int it = nth_item(rd);
        if (it >= p.items) break;
      const Unit w = unit_of(p, it);
      const Tile x = tile_of(p, w, t);
      const int i = x.q0 + row;
      float m = -INFINITY, l = 0.f;
      const int steps = x.steps();
      if (steps == 0) continue;
      for (int step = 0; step < steps; ++step) {
        const int n = x.block(step), k0 = n * kBlk;
        // every key of the block is visible to every query of the tile
        const bool full = k0 + kBlk - 1 <= x.q0 && (k0 > x.q0 + kBlk - 1 - p.window || p.sinks - k0 >= kBlk);
        ok = wtw(M::kSFull + t, ns & 1);
        if (!ok) break;
        ++ns;
        tc::fence_after_sync();
        // 64 columns at a time, in loops of their own for whole blocks and for cut ones,
        // whose halves that no row of the warp sees are left out
        float s[64];
        uint32_t see[2];
        auto load = [&](int half) {
          float(&lo)[32] = *reinterpret_cast<float(*)[32]>(&s[0]);
          float(&hi)[32] = *reinterpret_cast<float(*)[32]>(&s[32]);
          tc::ld32x2_wait(tS + 64 * half, tS + 64 * half + 32, lo, hi);
        };
        auto load_cut = [&](int half) -> bool {
          const int end = i - k0 + 1 - 64 * half, first = end - p.window, stay = min(p.sinks - k0 - 64 * half, end);
#pragma unroll
          for (int wd = 0; wd < 2; ++wd)
            see[wd] = (below(end - 32 * wd) & ~below(first - 32 * wd)) | below(stay - 32 * wd);
          if (!__any_sync(0xffffffffu, (see[0] | see[1]) != 0)) return false;
          load(half);
          return true;
        };
        auto masked = [&](int c, float v) -> float { return see[c >> 5] & (1u << (c & 31)) ? v : -INFINITY; };
        float top = -INFINITY;
        if (full) {
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            load(half);
            float u[4] = {top, s[0], s[1], s[2]};
#pragma unroll
            for (int c = 3; c + 1 < 64; c += 2) u[(c >> 1) & 3] = max3(u[(c >> 1) & 3], s[c], s[c + 1]);
            top = max3(max3(u[0], u[1], s[63]), u[2], u[3]);
          }
        } else {
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            if (!load_cut(half)) continue;
            float u[2] = {top, -INFINITY};
#pragma unroll
            for (int c = 0; c < 64; c += 2) u[(c >> 1) & 1] = max3(u[(c >> 1) & 1], masked(c, s[c]), masked(c + 1, s[c + 1]));
            top = fmaxf(u[0], u[1]);
          }
        }
        if (top > -INFINITY) top *= sl2;
        const bool need = top > m + kRescale;
        if (__any_sync(0xffffffffu, need)) {
          const float mn = need ? top : m;
          const float f = m == -INFINITY ? 0.f : ex2(m - mn);
          l *= f;
          m = mn;
          // O holds the blocks before this one: their PV came before this S
          if (step > 0) {
#pragma unroll 1
            for (int c = 0; c < kD; c += 8) {
              uint32_t o[8];
              tc::ld8_wait(tO + c, o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tc::st8_async(tO + c, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m;     // nothing seen yet: 2^(-inf - 0) = 0
        const float2 b2 = make_float2(-base, -base);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 a2 = make_float2(sl2, sl2);
        // P of keys 2 c, 2 c + 1 in column 64 + c, from the last keys to the first:
        // what it overwrites has been read for the last time
        if (full) {
#pragma unroll 1
          for (int half = 1;; half = 0) {
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              uint32_t pk[16];
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const float2 e = fma2(make_float2(s[32 * part + c], s[32 * part + c + 1]), a2, b2);
                const float2 v = make_float2(ex2(e.x), ex2(e.y));
                sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], v);
                pk[c / 2] = pack_bf16(v.x, v.y);
              }
              tc::st16_async(tS + 64 + 32 * half + 16 * part, pk);
            }
            if (half == 0) break;
            load(0);
          }
        } else {
#pragma unroll 1
          for (int half = 1;; half = 0) {
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              uint32_t pk[16];
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const int k = 32 * part + c;
                const float2 e = fma2(make_float2(s[k], s[k + 1]), a2, b2);
                const float2 v = make_float2(ex2(masked(k, e.x)), ex2(masked(k + 1, e.y)));
                sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], v);
                pk[c / 2] = pack_bf16(v.x, v.y);
              }
              tc::st16_async(tS + 64 + 32 * half + 16 * part, pk);
            }
            if (half == 0) break;
            load_cut(0);
          }
        }
        const float2 both = add2(sum[0], sum[1]);
        l += both.x + both.y;
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(bar(M::kPFull + t));
      }
      if (!ok) break;
      ok = wtw(M::kLEmpty + t, (no & 1) ^ 1);
      if (!ok) break;
      ++no;
      *stat = make_float2(m, l);
      mbar_arrive(bar(M::kLFull + t));
    }
    tc::wait_st();                                       // P on its way when this warp gave up
  } else {
    // ============================ outputs ================================
    // O / l as bf16 rows, lse = (m + log2 l) ln 2, of the tiles in turn, while the
    // softmax warps work on the next ones (thread = query row)
    const int qd = warp & 3, row = 32 * qd + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
    unsigned char *stage = smem + M::kOut + qd * 4096;
    uint32_t no = 0;                                     // parities of the tiles' outputs so far
    bool ok = true;
    for (int rd = 0; ok; ++rd) {
        const int it = nth_item(rd);
        if (it >= p.items) break;
      const Unit w = unit_of(p, it);
#pragma unroll 1
      for (int t = 0; ok && t < 2; ++t) {
        const Tile x = tile_of(p, w, t);
        if (!x.exists) continue;
        const uint32_t tO = tmem + lanes + kColO + t * kD;
        const int i = x.q0 + row;
        float2 ml = make_float2(0.f, 1.f);
        if (x.hi >= 0) {
          const uint32_t parity = (no >> t) & 1;
          no ^= 1u << t;
          ok = wtw(M::kLFull + t, parity) && wtw(M::kOFull + t, parity);
          if (!ok) break;
          tc::fence_after_sync();
          ml = reinterpret_cast<const float2 *>(smem + M::kStat)[t * 128 + row];
          mbar_arrive(bar(M::kLEmpty + t));
        }
        const bool live = i < w.n;
        const float inv = 1.f / ml.y;
#pragma unroll 1
        for (int hx = 0; hx < kHalves; ++hx) {
          if (lane == 0) bulk_wait_group_read0();        // the copy before has read the buffer
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            float o[32];
            if (x.hi >= 0) tc::ld32_wait(tO + 64 * hx + c, o);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float *y = o + 8 * u;
              uint4 v = make_uint4(pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv),
                                   pack_bf16(y[4] * inv, y[5] * inv), pack_bf16(y[6] * inv, y[7] * inv));
              if (!live) v = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4 *>(stage + lane * 128 + (((c / 8 + u) ^ (lane & 7)) << 4)) = v;
            }
          }
          if (hx == kHalves - 1 && x.hi >= 0) {
            tc::fence_before_sync();
            mbar_arrive(bar(M::kOEmpty + t));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && x.q0 + 32 * qd < p.T) {       // rows past T are not written
            tma_store_4d(&tmO, sb + M::kOut + qd * 4096, hx * 64, x.h, x.q0 + 32 * qd, w.b);
            bulk_commit_group();
          }
        }
        if (i < p.T)
          p.lse[(static_cast<size_t>(w.b) * p.Hq + x.h) * p.T + i] = live ? (ml.x + __log2f(ml.y)) * kLn2 : -INFINITY;
        __syncwarp();
      }
    }
    if (lane == 0) bulk_wait_group_read0();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int kD>
cudaError_t launch(const WindowArgs &a, const FwdParams &p, int grid, cudaStream_t st, const char **why) {
  CUtensorMap q, k, v, o;
  if (!token_map(&q, a.q, a.Hq, a.T, a.B, kD, a.q_stride, kBlk, why) ||
      !token_map(&k, a.k, a.Hkv, a.T, a.B, kD, a.k_stride, kBlk, why) ||
      !token_map(&v, a.v, a.Hkv, a.T, a.B, kD, a.v_stride, kBlk, why) ||
      !token_map(&o, a.o, a.Hq, a.T, a.B, kD, a.o_stride, 32, why))
    return cudaErrorInvalidValue;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(window_fwd_kernel<kD>), FwdSmem<kD>::kBytes);
  if (e != cudaSuccess) return e;
  window_fwd_kernel<kD><<<grid, kThr, FwdSmem<kD>::kBytes, st>>>(q, k, v, o, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_fwd(const WindowArgs &a, const WaitCtl &w, cudaStream_t st, const char **why) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  FwdParams p;
  p.lse = a.lse, p.lengths = a.lengths;
  p.B = a.B, p.T = a.T, p.Hq = a.Hq, p.Hkv = a.Hkv, p.G = a.Hq / a.Hkv;
  p.nqb = (a.T + kBlk - 1) / kBlk;
  p.pair_heads = p.G % 2 == 0;
  p.per_head = p.pair_heads ? p.nqb : (p.nqb + 1) / 2;
  const long long units = static_cast<long long>(a.B) * (p.pair_heads ? a.Hq / 2 : a.Hq);
  const long long items = units * p.per_head;
  if (items > 0x7fff0000LL) {
    *why = "grid too large";
    return cudaErrorNotSupported;
  }
  p.units = static_cast<int>(units), p.items = static_cast<int>(items);
  p.window = std::min(a.window, a.T), p.sinks = std::min(a.sinks, a.T);
  p.sink_blocks = (p.sinks + kBlk - 1) / kBlk;
  p.scale = a.scale;
  p.wait = w;
  // what the tiles that are worked on at one time meet of K and V is to stay in L2
  const long long meets = static_cast<long long>(std::min(p.nqb, (p.window + kBlk - 1) / kBlk + 2)) * kBlk * a.D * 4;
  p.group = static_cast<int>(std::max(1LL, std::min(units, kGroupBytes / meets * (p.pair_heads ? p.G / 2 : p.G))));
  p.by_group = Div::by(p.group * p.per_head);
  p.by_width = Div::by(p.group);
  p.by_last = Div::by((p.units - 1) % p.group + 1);
  p.by_heads = Div::by(p.pair_heads ? a.Hq / 2 : a.Hq);
  p.by_g = Div::by(p.G);
  const int grid = static_cast<int>(std::min<long long>(items, sms));
  return a.D == 64 ? launch<64>(a, p, grid, st, why) : launch<128>(a, p, grid, st, why);
}

}  // namespace abw
