// Serving side of the softmax attention: a paged cache of keys and values,
// attention of one new token per sequence over it, and the eviction of the
// tokens that got the least attention.
//
// Cache: k_pages, v_pages [n_pages][page_size][Hkv][D] bf16; position p of
// sequence b stands in row p % page_size of page block_table[b][p / page_size].
// Every entry is tested against n_pages before it becomes an address.
//
// attn_decode_paged, two launches:
//   split : the visible positions of all sequences and heads as one list of
//           16-token tiles, cut into equal runs, one per CTA, whatever the
//           sequences' lengths.  A run's part of one (sequence, KV head) is a
//           piece; a piece that is the whole of it leaves as output, another as
//           (max, sum, unnormalised output) in the workspace.
//   finish: joins the pieces of each (sequence, head) that was cut, and with
//           weight sums adds 2^(score - lse) of every position.
// Per query row the softmax statistics run along (max m, sum l, output O, all
// fp32): a tile with a larger max rescales l and O by 2^(m_old - m_new).
//
// The bound is the cache's bytes.  A warp copies (cp.async) its tile's rows whole, two
// 256-byte rows an instruction, into a ring of two tiles (16 KB at D = 128) of its
// own, each 16-byte unit to where the lane that feeds it to the tensor core reads it:
// no barrier between warps, no bank conflict.  (With each lane copying its own units,
// 64 bytes of eight rows an instruction, the copies alone ran at 5.3 of 7.2 TB/s.)
// The units are fragments as they stand, because the contraction index of k q and the
// row index of v p may be permuted at will (m16n8k16, lane = 4 g + t):
//   S^T = K Q^T (rows = 16 keys, columns = 8 query heads): lane (g, t) reads keys g and
//     g + 8, components 32 c + 8 t .. + 7, whose pairs are the k indices (2t, 2t+1,
//     2t+8, 2t+9) of two steps; Q is laid out to match.
//   O^T = V^T P^T (rows = components, columns = heads): lane (g, t) reads keys 2t, 2t+1,
//     2t+8, 2t+9, components 64 c + 8 g .. + 7; a byte permutation pairs the keys.
//     P's fragment is the transpose of S's (movmatrix).
// P enters as bf16 terms (two of them for bf16 outputs, three for fp32), fp32
// queries as three, so nothing but the output is rounded to bf16.  The maximum is
// lazy: it moves only when a score exceeds it by more than 8 (base 2).
//
// 8 sequences of up to 32768 tokens, 32 / 8 heads of 128, with weight sums: 128 us for
// 668 MB of pages and 21 MB of scores (5.4 TB/s; the split alone 6.1).  64 sequences of
// up to 1024, 20 / 5 heads: 31 us for 125 MB: a CTA has 33 tiles, and its launch, its
// search for its place and the first copies take half as long as they do.
#include <math.h>

#include <algorithm>

#include "abw_host.h"

namespace abw {
namespace {

// ------------------------------------------------------------------- writing
// One block per `tpb` tokens; 16-byte units, up to four of k and of v in
// flight per thread.  Bound by the bytes: 4 x up to 2048 tokens of 20 heads of 128 in 22
// us (5.1 TB/s; two in flight 28, eight 29, pages looked up beside the rows 23); a step
// of 64 tokens is a launch, 2.6 us.
constexpr int kWrThr = 256;
constexpr int kWrUnroll = 4;

struct WriteParams {
  const uint4 *k, *v;
  uint4 *kp, *vp;
  const int *table, *starts, *lengths;
  long long ntok, k_stride, v_stride;   // strides in 16-byte units
  int T, units, tpb, n_pages, page_size, max_pages;
};

__global__ void __launch_bounds__(kWrThr) kv_pages_write_kernel(const __grid_constant__ WriteParams p) {
  const long long t0 = static_cast<long long>(blockIdx.x) * p.tpb;
  const int total = p.units * static_cast<int>(min(static_cast<long long>(p.tpb), p.ntok - t0));
  for (int e0 = threadIdx.x; e0 < total; e0 += kWrThr * kWrUnroll) {
    uint4 a[kWrUnroll], c[kWrUnroll];
    long long to[kWrUnroll];
#pragma unroll
    for (int i = 0; i < kWrUnroll; ++i) {
      const int e = e0 + i * kWrThr;
      to[i] = -1;
      if (e >= total) continue;
      const int rel = e / p.units, unit = e - rel * p.units;
      const long long tok = t0 + rel;
      const int b = static_cast<int>(tok / p.T), t = static_cast<int>(tok - static_cast<long long>(b) * p.T);
      if (p.lengths && t >= p.lengths[b]) continue;
      const long long pos = static_cast<long long>(p.starts[b]) + t;
      if (pos < 0 || pos >= static_cast<long long>(p.page_size) * p.max_pages) continue;
      const int at = static_cast<int>(pos), pg = at / p.page_size;
      const int page = p.table[static_cast<long long>(b) * p.max_pages + pg];
      if (page < 0 || page >= p.n_pages) continue;
      to[i] = (static_cast<long long>(page) * p.page_size + (at - pg * p.page_size)) * p.units + unit;
      a[i] = p.k[tok * p.k_stride + unit];
      c[i] = p.v[tok * p.v_stride + unit];
    }
#pragma unroll
    for (int i = 0; i < kWrUnroll; ++i)
      if (to[i] >= 0) {
        p.kp[to[i]] = a[i];
        p.vp[to[i]] = c[i];
      }
  }
}

// -------------------------------------------------------------------- decode
// Warps per CTA, two CTAs per SM: a tile's chain of waits and products takes some 1,500
// cycles, so more warps with two tiles each under way beat fewer with three (4 x 3
// stages 164 us, 6 x 2 138 us for 8 long sequences with weight sums).  fp32 queries
// of wide groups take the registers of four.
constexpr int dec_warps(bool f32, bool wide) { return f32 && wide ? 4 : 6; }
constexpr int kDecStages = 2;
constexpr int kTile = 16;            // positions per tile
constexpr int kMinTiles = 8;         // tiles a CTA takes at least, while there are few
constexpr int kDecCtas = 304;        // two per SM
// Blocks of the weight sums: as many for each sequence and KV head as give a full table
// kWtPos positions a block, one at least, while that makes no more than kWtBlocks.
constexpr int kWtPos = 1024, kWtBlocks = 1216;
constexpr int kWtUnroll = 4;
constexpr uint32_t kNoRow = 0xffffffffu;
constexpr float kLazy = 8.f;         // base-2 units a score may exceed the running maximum by

struct DecParams {
  const void *q;
  void *o;
  const __nv_bfloat16 *kp, *vp;
  const int *table, *lengths;
  float *weight_sums;
  float *slots;        // [2 per CTA][rows * (D + 4)]: O [rows][D], m [rows], l [rows]
  float2 *stats;       // [B][Hq] (m, l) of what one CTA had whole (with weight sums)
  float *scores;       // [B][Hq][score_stride] scores in base-2 units (with weight sums)
  long long score_stride;
  int B, Hq, Hkv, D, G, ng, rows;    // ng groups of up to 16 query heads per KV head, rows = min(G, 16)
  int n_pages, page_size, page_shift, max_pages, cap, window, sinks;
  int q_bf16, ctas, wt_chunks, wt_len;
  float sl2;           // scale * log2(e)
};

// Visible positions of a sequence: [0, s) and [lo, n); index x of them.
struct Seq {
  int n, lo, s, vis;
};
__device__ __forceinline__ Seq seq_of(const DecParams &p, int b) {
  Seq r;
  r.n = min(max(p.lengths[b], 0), p.cap);
  r.lo = p.window > 0 ? max(0, r.n - p.window) : 0;
  r.s = min(p.sinks, r.lo);
  r.vis = r.s + r.n - r.lo;
  return r;
}
__device__ __forceinline__ int tiles_of(const Seq &s) { return (s.vis + kTile - 1) / kTile; }
__device__ __forceinline__ int position(const Seq &s, int x) { return x < s.s ? x : x - s.s + s.lo; }

// The list of tiles: sequence by sequence, in it unit by unit (KV head, group
// of query heads), in it tile by tile.  Thread i of a block holds the counts of
// sequences first(i) .. first(i + 1) - 1: `before` tiles stand ahead of them.
struct Share {
  long long total, before, mine;
  int b0, b1;
};
template <int kThreads>
__device__ Share share_of(const DecParams &p) {
  __shared__ long long warp_sum_s[kThreads / 32];
  const int per = (p.B + kThreads - 1) / kThreads;
  Share r;
  r.b0 = min(p.B, static_cast<int>(threadIdx.x) * per);
  r.b1 = min(p.B, r.b0 + per);
  r.mine = 0;
  for (int b = r.b0; b < r.b1; ++b) r.mine += tiles_of(seq_of(p, b));
  r.mine *= static_cast<long long>(p.Hkv) * p.ng;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = r.mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) warp_sum_s[warp] = incl;
  __syncthreads();
  long long ahead = 0;
  r.total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) ahead += warp_sum_s[w];
    r.total += warp_sum_s[w];
  }
  __syncthreads();
  r.before = ahead + incl - r.mine;
  return r;
}

// Runs of the tile list: CTA c takes tiles start(c) .. start(c + 1) - 1.
struct Runs {
  long long each, extra;
  int n;
  __device__ Runs(long long total, int ctas) {
    const long long want = (total + kMinTiles - 1) / kMinTiles;
    n = static_cast<int>(min(static_cast<long long>(ctas), max(want, 1LL)));
    each = total / n;
    extra = total - each * n;
  }
  __device__ long long start(int c) const { return c * each + min(static_cast<long long>(c), extra); }
  __device__ int owner(long long x) const {   // the CTA of tile x
    const long long big = extra * (each + 1);
    return static_cast<int>(x < big ? x / (each + 1) : extra + (x - big) / each);
  }
};

// The sequence, unit and tile of tile x of the list, found by the thread whose
// share holds it; all threads get it (x < total).
struct Place {
  int b, u, tile;
  long long seg;   // index of the unit's first tile
};
__device__ __forceinline__ Place place_of(const DecParams &p, const Share &sh, long long x) {
  __shared__ Place found;
  if (x >= sh.before && x < sh.before + sh.mine) {
    long long at = sh.before;
    for (int b = sh.b0; b < sh.b1; ++b) {
      const int tiles = tiles_of(seq_of(p, b));
      const long long all = static_cast<long long>(tiles) * p.Hkv * p.ng;
      if (x < at + all) {
        const long long rel = x - at;
        found.b = b;
        found.u = static_cast<int>(rel / tiles);
        found.tile = static_cast<int>(rel - static_cast<long long>(found.u) * tiles);
        found.seg = at + static_cast<long long>(found.u) * tiles;
        break;
      }
      at += all;
    }
  }
  __syncthreads();
  const Place r = found;
  __syncthreads();
  return r;
}

// A walk over the pieces of a CTA's run, the tiles of each dealt to the warps.
struct Walk {
  Seq s;
  int b, u, tiles, tile0, tend;
  long long left;      // tiles of the run behind this piece
  __device__ __forceinline__ void begin(const DecParams &p, const Place &at, long long count) {
    b = at.b;
    u = at.u;
    s = seq_of(p, b);
    tiles = tiles_of(s);
    tile0 = at.tile;
    tend = static_cast<int>(min(static_cast<long long>(tiles), tile0 + count));
    left = count - (tend - tile0);
  }
  // the next piece; false behind the last one
  __device__ __forceinline__ bool next(const DecParams &p) {
    if (left <= 0) return false;
    if (++u == p.Hkv * p.ng) {
      u = 0;
      do {
        ++b;
        s = seq_of(p, b);
        tiles = tiles_of(s);
      } while (tiles == 0);
    }
    tile0 = 0;
    tend = static_cast<int>(min(static_cast<long long>(tiles), left));
    left -= tend;
    return true;
  }
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit elements.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool there) {
  const int bytes = there ? 16 : 0;   // 0: the slot is filled with zeros and nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}
// bf16 terms of a pair of fp32 values, largest first.
template <int kN>
__device__ __forceinline__ void terms(float x, float y, uint32_t (&out)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    out[i] = bf2(x, y);
    if (i + 1 < kN) {
      x -= bf16_lo(out[i]);
      y -= bf16_hi(out[i]);
    }
  }
}

constexpr int dec_smem(int D, int warps) {
  return warps * kDecStages * kTile * D * 4 + warps * 4 * (D + 4) * 4 + warps * 8 * 4;
}
static_assert(2 * (dec_smem(128, 6) + 1024) <= 228 * 1024, "two CTAs per SM");

// kF32: fp32 queries and outputs; kWide: more than 8 query heads per KV head;
// kScores: scores are kept for the weight sums.
template <int kD, bool kF32, bool kWide, bool kScores>
__global__ void __launch_bounds__(32 * dec_warps(kF32, kWide), 2) decode_split_kernel(const __grid_constant__ DecParams p) {
  constexpr int kDecWarps = dec_warps(kF32, kWide), kDecThr = 32 * kDecWarps;
  constexpr int kQT = kF32 ? 3 : 1, kPT = kF32 ? 3 : 2;   // terms of q and of p
  constexpr int kC = kD / 32, kV = kD / 64;               // 64-byte pieces of a k row, 128-byte pieces of a v row
  constexpr int kR = kWide ? 2 : 1;                       // row halves
  extern __shared__ __align__(128) unsigned char smem[];
  float *mo = reinterpret_cast<float *>(smem + kDecWarps * kDecStages * kTile * kD * 4);   // [warps][4][kD + 4]
  float *ms = mo + kDecWarps * 4 * (kD + 4);              // [warps][4 max, 4 sum]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const Share sh = share_of<kDecThr>(p);
  // rows that see nothing
  for (int b = blockIdx.x; b < p.B; b += gridDim.x)
    if (seq_of(p, b).vis == 0) {
      const size_t bytes = static_cast<size_t>(p.Hq) * kD * (kF32 ? 4 : 2);
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<unsigned char *>(p.o) + b * bytes);
      for (size_t i = tid; i < bytes / 16; i += kDecThr) dst[i] = make_uint4(0, 0, 0, 0);
    }
  if (sh.total == 0) return;
  const Runs runs(sh.total, p.ctas);
  const int cta = blockIdx.x;
  if (cta >= runs.n) return;
  const long long r0 = runs.start(cta), count = runs.start(cta + 1) - r0;
  if (count == 0) return;
  const Place at = place_of(p, sh, r0);

  Walk now, ahead;
  now.begin(p, at, count);
  ahead = now;
  const unsigned char *ring_p = smem + warp * (kDecStages * kTile * kD * 4);
  // copies: lane -> unit `q` of row `hi` of the kRows that an instruction takes
  constexpr int kUnits = kD / 8, kRows = 32 / kUnits;
  const int hi = lane / kUnits, q = lane % kUnits;
  const uint32_t to_k = smem_u32(ring_p) + (hi * 4 + (q & 3)) * 16 + (q >> 2) * 512;
  const uint32_t to_v = smem_u32(ring_p) + (2 * kC + (hi & 1) * kV + (q >> 3)) * 512 + (hi >> 1) * 128 + (q & 7) * 16;

  // ---- loads: tile `lt` of the piece `ahead`, whose rows `row` holds (lanes 0 .. 15)
  int lt = ahead.tile0 + warp;
  bool more = true;
  uint32_t row = kNoRow;
  auto settle = [&]() {   // moves on to a piece that has a tile for this warp
    while (more && lt >= ahead.tend) {
      more = ahead.next(p);
      lt = warp;
    }
  };
  auto look_up = [&]() {
    row = kNoRow;
    if (!more || lane >= kTile) return;
    const int x = lt * kTile + lane;
    if (x >= ahead.s.vis) return;
    const int pos = position(ahead.s, x);
    const int pg = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page_size;
    const int page = p.table[static_cast<long long>(ahead.b) * p.max_pages + pg];
    if (page >= 0 && page < p.n_pages)
      row = static_cast<uint32_t>(page) * static_cast<uint32_t>(p.page_size) + static_cast<uint32_t>(pos - pg * p.page_size);
  };
  static_assert(kDecStages == 2, "a word of its own for each stage");
  uint32_t seen0 = 0, seen1 = 0;   // positions of each tile under way that are there
  auto issue = [&](int stage) {
    const uint32_t there_all = __ballot_sync(0xffffffffu, row != kNoRow);
    if (stage == 0) seen0 = there_all;
    if (stage == 1) seen1 = there_all;
    if (more) {
      const size_t unit = static_cast<size_t>(ahead.u / p.ng) * kD + 8 * q;
      const size_t pitch = static_cast<size_t>(p.Hkv) * kD;
      const __nv_bfloat16 *nothing = static_cast<const __nv_bfloat16 *>(p.q);   // an address that no byte is read from
      const uint32_t st = stage * (kTile * kD * 4);
#pragma unroll
      for (int i = 0; i < kTile; i += kRows) {
        const uint32_t r = __shfl_sync(0xffffffffu, row, i + hi);
        const bool there = r != kNoRow;
        const size_t at = r * pitch + unit;
        cp_async16(to_k + st + (i >> 3) * kC * 512 + (i & 7) * 64, there ? p.kp + at : nothing, there);
        cp_async16(to_v + st + 2 * (i >> 3) * kV * 512 + (i >> 1 & 3) * 128, there ? p.vp + at : nothing, there);
      }
      lt += kDecWarps;
      settle();
      look_up();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  settle();
  look_up();
#pragma unroll
  for (int i = 0; i < kDecStages; ++i) issue(i);

  int stage = 0;
  bool first = true;
  do {
    // ---- this piece's queries, as fragments: head g of each eight
    const int kvh = now.u / p.ng, grp = now.u - kvh * p.ng;
    const int h0 = kvh * p.G + grp * 16, nrows = min(16, p.G - grp * 16);
    uint32_t qf[kQT][kR][kC][4];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const bool live = g + 8 * r < nrows;
      const size_t src = (static_cast<size_t>(now.b) * p.Hq + h0 + (live ? g + 8 * r : 0)) * kD + 8 * t;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        if constexpr (kF32) {
          const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + src + 32 * c);
          const float4 z = make_float4(0.f, 0.f, 0.f, 0.f), x = live ? f[0] : z, y = live ? f[1] : z;
          const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t tm[kQT];
            terms<kQT>(v[2 * i], v[2 * i + 1], tm);
#pragma unroll
            for (int k = 0; k < kQT; ++k) qf[k][r][c][i] = tm[k];
          }
        } else {
          const uint4 x = live ? *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + src + 32 * c)
                               : make_uint4(0, 0, 0, 0);
          qf[0][r][c][0] = x.x;
          qf[0][r][c][1] = x.y;
          qf[0][r][c][2] = x.z;
          qf[0][r][c][3] = x.w;
        }
      }
    }
    // of heads 2 t and 2 t + 1 (of each eight): maximum, this lane's sum, outputs of
    // components 64 c + 8 g + 2 j (elements 0, 1) and + 1 (2, 3)
    float m[kR][2], l[kR][2], O[kR][kV][4][4];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      m[r][0] = m[r][1] = -INFINITY;
      l[r][0] = l[r][1] = 0.f;
#pragma unroll
      for (int c = 0; c < kV; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) O[r][c][j][e] = 0.f;
    }

    for (int tile = now.tile0 + warp; tile < now.tend; tile += kDecWarps) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kDecStages - 1) : "memory");
      __syncwarp();                        // the other lanes' copies too
      const unsigned char *src = ring_p + stage * (kTile * kD * 4);
      const uint32_t mask = stage == 0 ? seen0 : seen1;
      // ---- S^T = K Q^T, in two chains
      float S[kR][2][4];
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[r][0][e] = S[r][1][e] = 0.f;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const uint4 a = *reinterpret_cast<const uint4 *>(src + c * 512 + lane * 16);
        const uint4 b = *reinterpret_cast<const uint4 *>(src + (kC + c) * 512 + lane * 16);
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
          for (int x = 0; x < kQT; ++x) {
            mma16816(S[r][0], a.x, b.x, a.y, b.y, qf[x][r][c][0], qf[x][r][c][1]);
            mma16816(S[r][1], a.z, b.z, a.w, b.w, qf[x][r][c][2], qf[x][r][c][3]);
          }
      }
      // ---- running softmax of each head over the 16 positions
      uint32_t pf[kR][kPT][2];             // [term][keys 2t, 2t+1 | 2t+8, 2t+9] of head g
      const bool in0 = mask >> g & 1u, in1 = mask >> (g + 8) & 1u;
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float s[4];                        // (key g, head 2t), (g, 2t+1), (g + 8, 2t), (g + 8, 2t+1)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = (e < 2 ? in0 : in1) ? (S[r][0][e] + S[r][1][e]) * p.sl2 : -INFINITY;
        if constexpr (kScores) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int head = 8 * r + 2 * t + x;
            if (head < nrows) {
              float *dst = p.scores + (static_cast<size_t>(now.b) * p.Hq + h0 + head) * p.score_stride +
                           static_cast<size_t>(tile) * kTile + g;
              dst[0] = s[x];
              dst[8] = s[2 + x];
            }
          }
        }
        float top[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
        if (__any_sync(0xffffffffu, top[0] > m[r][0] + kLazy || top[1] > m[r][1] + kLazy)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], d));
            const float mn = fmaxf(m[r][x], top[x]);
            const float f = mn == -INFINITY ? 1.f : ex2(m[r][x] - mn);
            m[r][x] = mn;
            l[r][x] *= f;
#pragma unroll
            for (int c = 0; c < kV; ++c)
#pragma unroll
              for (int j = 0; j < 4; ++j) O[r][c][j][x] *= f, O[r][c][j][2 + x] *= f;
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float base = m[r][x] == -INFINITY ? 0.f : m[r][x];   // nothing seen yet: 2^(-inf - 0) = 0
          s[x] = ex2(s[x] - base);
          s[2 + x] = ex2(s[2 + x] - base);
          l[r][x] += s[x] + s[2 + x];
        }
        uint32_t lo[kPT], up[kPT];
        terms<kPT>(s[0], s[1], lo);
        terms<kPT>(s[2], s[3], up);
#pragma unroll
        for (int k = 0; k < kPT; ++k) pf[r][k][0] = transposed(lo[k]), pf[r][k][1] = transposed(up[k]);
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int c = 0; c < kV; ++c) {
        uint32_t v[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {      // keys 2t, 2t+1, 2t+8, 2t+9
          const uint4 x = *reinterpret_cast<const uint4 *>(src + (2 * kC + n * kV + c) * 512 + (8 * t + g) * 16);
          v[n][0] = x.x, v[n][1] = x.y, v[n][2] = x.z, v[n][3] = x.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a0 = __byte_perm(v[0][j], v[1][j], 0x5410), a1 = __byte_perm(v[0][j], v[1][j], 0x7632);
          const uint32_t a2 = __byte_perm(v[2][j], v[3][j], 0x5410), a3 = __byte_perm(v[2][j], v[3][j], 0x7632);
#pragma unroll
          for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int k = 0; k < kPT; ++k) mma16816(O[r][c][j], a0, a1, a2, a3, pf[r][k][0], pf[r][k][1]);
        }
      }
      __syncwarp();                        // every lane has read the tile
      issue(stage);
      stage = stage + 1 == kDecStages ? 0 : stage + 1;
    }

    // ---- the warps' parts of the piece, joined through shared memory, four rows at a time
    // (with eight two CTAs do not fit an SM)
    const bool whole = now.tile0 == 0 && now.tend == now.tiles;
    float *slot = p.slots + (static_cast<size_t>(cta) * 2 + (first ? 0 : 1)) * p.rows * (kD + 4);
#pragma unroll
    for (int rx = 0; rx < 2 * kR; ++rx) {
      const int r = rx >> 1, x = rx & 1;                 // heads 8 r + 2 t + x
      {
        float sum = l[r][x];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (g == 0) {
          ms[warp * 8 + t] = m[r][x];
          ms[warp * 8 + 4 + t] = sum;
        }
#pragma unroll
        for (int c = 0; c < kV; ++c) {
          float *dst = mo + (warp * 4 + t) * (kD + 4) + 64 * c + 8 * g;
#pragma unroll
          for (int j = 0; j < 4; j += 2)
            *reinterpret_cast<float4 *>(dst + 2 * j) =
                make_float4(O[r][c][j][x], O[r][c][j][2 + x], O[r][c][j + 1][x], O[r][c][j + 1][2 + x]);
        }
      }
      __syncthreads();
      for (int e = tid; e < 4 * kD / 4; e += kDecThr) {
        const int rr = e / (kD / 4), d = (e - rr * (kD / 4)) * 4, hrow = 8 * r + 2 * rr + x;
        if (hrow >= nrows) continue;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, ms[w * 8 + rr]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float mw = ms[w * 8 + rr];
          const float f = mw == -INFINITY ? 0.f : ex2(mw - M);
          const float4 y = *reinterpret_cast<const float4 *>(mo + (w * 4 + rr) * (kD + 4) + d);
          L = fmaf(f, ms[w * 8 + 4 + rr], L);
          acc.x = fmaf(f, y.x, acc.x), acc.y = fmaf(f, y.y, acc.y);
          acc.z = fmaf(f, y.z, acc.z), acc.w = fmaf(f, y.w, acc.w);
        }
        if (whole) {
          const float inv = L > 0.f ? 1.f / L : 0.f;
          const size_t dst = (static_cast<size_t>(now.b) * p.Hq + h0 + hrow) * kD + d;
          if constexpr (kF32)
            *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + dst) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
          else
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.o) + dst) =
                make_uint2(bf2(acc.x * inv, acc.y * inv), bf2(acc.z * inv, acc.w * inv));
          if (kScores && d == 0) p.stats[static_cast<size_t>(now.b) * p.Hq + h0 + hrow] = make_float2(M, L);
        } else {
          *reinterpret_cast<float4 *>(slot + hrow * kD + d) = acc;
          if (d == 0) {
            slot[p.rows * kD + hrow] = M;
            slot[p.rows * (kD + 1) + hrow] = L;
          }
        }
      }
      __syncthreads();
    }
    first = false;
  } while (now.next(p));
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Blocks 0 .. ctas - 1: block c joins the unit that begins in CTA c's run and
// goes on behind it.  Blocks behind them, with weight sums: wt_len visible positions
// of a sequence and KV head each, wt_chunks blocks for the table's capacity (so a short
// sequence in a wide table is left to its first blocks).
constexpr int kFinThr = 256;

// Slot of the i-th piece of a unit whose first tile is `seg`.
__device__ __forceinline__ const float *piece_slot(const DecParams &p, const Runs &runs, long long seg, int c0, int i) {
  const int second = i == 0 && seg != runs.start(c0);
  return p.slots + (static_cast<size_t>(c0 + i) * 2 + second) * p.rows * (p.D + 4);
}

// Max and sum of row `row` of a unit over its pieces, by one warp.
__device__ __forceinline__ float2 joined_stats(const DecParams &p, const Runs &runs, long long seg, int c0, int pieces,
                                               int row) {
  const int lane = threadIdx.x & 31;
  float M = -INFINITY, L = 0.f;
  for (int i = lane; i < pieces; i += 32) {
    const float *s = piece_slot(p, runs, seg, c0, i) + p.rows * p.D;
    const float m = s[row], l = s[p.rows + row], mn = fmaxf(M, m);
    if (mn == -INFINITY) continue;
    L = L * ex2(M - mn) + l * ex2(m - mn);
    M = mn;
  }
  const float top = warp_max(M);
  L = warp_sum(top == -INFINITY || M == -INFINITY ? 0.f : L * ex2(M - top));
  return make_float2(top, L);
}

__global__ void __launch_bounds__(kFinThr) decode_finish_kernel(const __grid_constant__ DecParams p) {
  __shared__ float2 st[16];
  __shared__ long long wt_before;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Share sh = share_of<kFinThr>(p);
  // every block waits, also one without work: what follows on the stream then
  // finds the launch before this one complete
  if (sh.total == 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const Runs runs(sh.total, p.ctas);
  if (static_cast<int>(blockIdx.x) < p.ctas) {
    const int c = blockIdx.x;
    const long long r0 = runs.start(min(c, runs.n - 1)), r1 = runs.start(min(c, runs.n - 1) + 1);
    const Place at = place_of(p, sh, r1 - 1);
    const int tiles = tiles_of(seq_of(p, at.b));
    const long long end = at.seg + tiles;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c >= runs.n || end <= r1 || at.seg < r0) return;
    const int pieces = runs.owner(end - 1) - c + 1;
    const int kvh = at.u / p.ng, grp = at.u - kvh * p.ng;
    const int h0 = kvh * p.G + grp * 16, nrows = min(16, p.G - grp * 16);
    for (int r = warp; r < nrows; r += kFinThr / 32) {
      const float2 x = joined_stats(p, runs, at.seg, c, pieces, r);
      if (lane == 0) st[r] = x;
    }
    __syncthreads();
    for (int e = tid; e < nrows * (p.D / 4); e += kFinThr) {
      const int r = e / (p.D / 4), d = (e - r * (p.D / 4)) * 4;
      const float M = st[r].x, L = st[r].y;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < pieces; ++i) {
        const float *s = piece_slot(p, runs, at.seg, c, i);
        const float m = s[p.rows * p.D + r];
        const float4 x = *reinterpret_cast<const float4 *>(s + r * p.D + d);
        const float f = m == -INFINITY ? 0.f : ex2(m - M);
        acc.x = fmaf(f, x.x, acc.x), acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z), acc.w = fmaf(f, x.w, acc.w);
      }
      const float inv = L > 0.f ? 1.f / L : 0.f;
      const size_t dst = (static_cast<size_t>(at.b) * p.Hq + h0 + r) * p.D + d;
      if (p.q_bf16)
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.o) + dst) =
            make_uint2(bf2(acc.x * inv, acc.y * inv), bf2(acc.z * inv, acc.w * inv));
      else
        *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + dst) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
    return;
  }
  // ---- weight sums
  const long long w = static_cast<long long>(blockIdx.x) - p.ctas;
  const int chunk = static_cast<int>(w % p.wt_chunks);
  const int kvh = static_cast<int>(w / p.wt_chunks % p.Hkv), b = static_cast<int>(w / p.wt_chunks / p.Hkv);
  const Seq s = seq_of(p, b);
  if (b >= sh.b0 && b < sh.b1) {   // tiles ahead of this sequence
    long long at = 0;
    for (int i = sh.b0; i < b; ++i) at += tiles_of(seq_of(p, i));
    wt_before = sh.before + at * p.Hkv * p.ng;
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int x0 = static_cast<int>(min(static_cast<long long>(chunk) * p.wt_len, static_cast<long long>(s.vis)));
  const int x1 = static_cast<int>(min(static_cast<long long>(x0) + p.wt_len, static_cast<long long>(s.vis)));
  if (x0 >= x1) return;
  const int tiles = tiles_of(s);
  float *dst = p.weight_sums + (static_cast<size_t>(b) * p.Hkv + kvh) * p.cap;
  for (int grp = 0; grp < p.ng; ++grp) {
    const long long seg = wt_before + (static_cast<long long>(kvh) * p.ng + grp) * tiles;
    const int c0 = runs.owner(seg), c1 = runs.owner(seg + tiles - 1);
    const int h0 = kvh * p.G + grp * 16, nrows = min(16, p.G - grp * 16);
    __syncthreads();
    for (int r = warp; r < nrows; r += kFinThr / 32) {
      const float2 x = c0 == c1 ? p.stats[static_cast<size_t>(b) * p.Hq + h0 + r]
                                : joined_stats(p, runs, seg, c0, c1 - c0 + 1, r);
      if (lane == 0) st[r] = x.y > 0.f ? make_float2(x.x, 1.f / x.y) : make_float2(0.f, 0.f);
    }
    __syncthreads();
    const float *sc = p.scores + (static_cast<size_t>(b) * p.Hq + h0) * p.score_stride;
    for (int x = x0 + tid; x < x1; x += kFinThr * kWtUnroll) {
      float acc[kWtUnroll], old[kWtUnroll];
#pragma unroll
      for (int i = 0; i < kWtUnroll; ++i) {
        acc[i] = 0.f;
        old[i] = x + i * kFinThr < x1 ? dst[position(s, x + i * kFinThr)] : 0.f;
      }
#pragma unroll 4
      for (int r = 0; r < nrows; ++r) {
        const float M = st[r].x, inv = st[r].y;          // 0, 0 where nothing is seen
#pragma unroll
        for (int i = 0; i < kWtUnroll; ++i)
          if (x + i * kFinThr < x1) acc[i] = fmaf(ex2(sc[r * p.score_stride + x + i * kFinThr] - M), inv, acc[i]);
      }
#pragma unroll
      for (int i = 0; i < kWtUnroll; ++i)
        if (x + i * kFinThr < x1 && acc[i] > 0.f) dst[position(s, x + i * kFinThr)] = old[i] + acc[i];
    }
  }
}

// ------------------------------------------------------------------ eviction
// One block per (sequence, KV head) finds the tokens to keep: their weights become
// unsigned keys of the same order (0: absent page; the largest: kept whatever its
// weight), a radix select over the keys' bits (11, 11 and 10 at a time, from the top)
// gives the key of the last one kept and how many equal ones go with it, and a walk in
// the order of the positions, a stretch per warp, writes them down.  A second launch
// moves the rows.  The keys stay in shared memory where all positions fit (8192 of
// them in each of 128 blocks: 16 us, 26 us without), else each step forms them
// again from the weights.
constexpr int kEvThr = 1024, kEvWarps = kEvThr / 32;
constexpr int kEvBins = 2048;
constexpr int kEvCached = 40960;      // positions whose keys fit shared memory
constexpr uint32_t kKeyHeld = 0xffffffffu;   // above every weight's

struct EvictParams {
  uint4 *kp, *vp;
  const int *table, *lengths, *new_table;
  const float *sums;
  int *kept, *new_lengths;
  float *new_sums;
  int B, Hkv, units;                  // units: 16-byte units of a head's row
  int n_pages, page_size, page_shift, max_pages, cap, new_max_pages, new_cap, budget, sinks, recent;
};

// Order of the weights as unsigned numbers: larger weight, larger number, from
// 0x007fffff (-infinity, and NaN) to 0xff800000; -0 counts as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w != w ? -INFINITY : w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <bool kCache>
__global__ void __launch_bounds__(kEvThr, 1) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ int hist[kEvBins], warp_a[kEvWarps], warp_b[kEvWarps];
  __shared__ int digit_s, need_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n = min(max(p.lengths[b], 0), p.cap);
  const int late = max(n - p.recent, 0);   // positions from here on are recent
  const float *sums = p.sums + static_cast<size_t>(blockIdx.x) * p.cap;
  int *kept = p.kept + static_cast<size_t>(blockIdx.x) * p.budget;
  float *new_sums = p.new_sums + static_cast<size_t>(blockIdx.x) * p.new_cap;
  auto form = [&](int j) -> uint32_t {
    const int pg = p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
    const int page = p.table[static_cast<long long>(b) * p.max_pages + pg];
    if (page < 0 || page >= p.n_pages) return 0u;
    return j < p.sinks || j >= late ? kKeyHeld : weight_key(sums[j]);
  };
  auto key = [&](int j) -> uint32_t { return kCache ? keys[j] : form(j); };

  int here = 0;
#pragma unroll 4
  for (int j = tid; j < n; j += kEvThr) {
    const uint32_t k = form(j);
    if (kCache) keys[j] = k;
    here += k != 0u;
  }
  here = __reduce_add_sync(0xffffffffu, here);
  if (lane == 0) warp_a[warp] = here;
  __syncthreads();
  here = __reduce_add_sync(0xffffffffu, warp_a[lane]);
  const int m = min(here, p.budget);
  // the smallest key that is kept, and how many of its equals (the first ones); those
  // that are held are at most sinks + recent <= budget
  uint32_t least = 1u;
  int ties = n;
  if (here > p.budget) {
    int need = m;
    uint32_t prefix = 0u;
    for (int step = 0; step < 3; ++step) {
      const int shift = step == 0 ? 21 : step == 1 ? 10 : 0, bits = step == 2 ? 10 : 11;
      __syncthreads();
      for (int i = tid; i < kEvBins; i += kEvThr) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int j = tid; j < n; j += kEvThr) {
        const uint32_t k = key(j);
        if (step == 0 || (k >> (shift + bits)) == (prefix >> (shift + bits))) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1);
      }
      __syncthreads();
      // thread i: bins 2 i and 2 i + 1; what is above them in its warp, then in others
      const int lo = hist[2 * tid], hi = hist[2 * tid + 1];
      int above = lo + hi;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_down_sync(0xffffffffu, above, d);
        if (lane + d < 32) above += o;
      }
      if (lane == 0) warp_a[warp] = above;
      __syncthreads();
      above += __reduce_add_sync(0xffffffffu, lane > warp ? warp_a[lane] : 0) - lo - hi;
      if (above < need && above + hi >= need) {
        digit_s = 2 * tid + 1;
        need_s = need - above;
      } else if (above + hi < need && above + hi + lo >= need) {
        digit_s = 2 * tid;
        need_s = need - above - hi;
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(digit_s) << shift;
      need = need_s;
    }
    least = prefix;
    ties = need;
  }
  // ---- in the order of the positions: warp w takes a stretch of them
  const int stretch = ((n + kEvThr - 1) / kEvThr) * 32;
  const int j0 = min(n, warp * stretch), j1 = min(n, j0 + stretch);
  int more = 0, equal = 0;                 // above `least` and equal to it
  for (int j = j0 + lane; j - lane < j1; j += 32) {
    const uint32_t k = j < j1 ? key(j) : 0u;
    more += __popc(__ballot_sync(0xffffffffu, k > least));
    equal += __popc(__ballot_sync(0xffffffffu, k == least && k != 0u));
  }
  // with `least` 1 (all are kept) no key equals it: weights' keys begin higher
  __syncthreads();
  if (lane == 0) warp_a[warp] = more, warp_b[warp] = equal;
  __syncthreads();
  more = __reduce_add_sync(0xffffffffu, lane < warp ? warp_a[lane] : 0);
  equal = __reduce_add_sync(0xffffffffu, lane < warp ? warp_b[lane] : 0);
  int out = more + min(equal, ties);
  const uint32_t before = (1u << lane) - 1u;
  for (int j = j0 + lane; j - lane < j1; j += 32) {
    const uint32_t k = j < j1 ? key(j) : 0u;
    const uint32_t eq = __ballot_sync(0xffffffffu, k == least);
    const bool keep = k > least || (k == least && equal + __popc(eq & before) < ties);
    const uint32_t ks = __ballot_sync(0xffffffffu, keep);
    const int at = out + __popc(ks & before);
    if (keep && at < m) {
      kept[at] = j;
      new_sums[at] = sums[j];
    }
    equal += __popc(eq);
    out += __popc(ks);
  }
  for (int i = m + tid; i < p.budget; i += kEvThr) kept[i] = -1;
  for (int i = m + tid; i < p.new_cap; i += kEvThr) new_sums[i] = 0.f;
  if (h == 0 && tid == 0) p.new_lengths[b] = m;
}

// Rows of the kept tokens, 16 bytes per thread and step; consecutive threads
// take the units of a row, then its heads.  Rows of 256 bytes from anywhere, each read and
// written once and so streamed past L2: 16 x 8192 tokens of 8 heads to 2048 take 55 us a
// call (60 with ordinary loads and stores), one sequence of 1025 to 512 8.8 us (9.8
// with four steps of a thread under way in place of two).
constexpr int kMvThr = 256, kMvUnroll = 2;

__global__ void __launch_bounds__(kMvThr) evict_move_kernel(const __grid_constant__ EvictParams p, long long total) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per_tok = p.Hkv * p.units;
  for (long long e0 = static_cast<long long>(blockIdx.x) * kMvThr * kMvUnroll + threadIdx.x; e0 < total;
       e0 += static_cast<long long>(gridDim.x) * kMvThr * kMvUnroll) {
    uint4 a[kMvUnroll], c[kMvUnroll];
    long long to[kMvUnroll];
#pragma unroll
    for (int i = 0; i < kMvUnroll; ++i) {
      to[i] = -1;
      const long long e = e0 + i * kMvThr;
      if (e >= total) continue;
      const long long tok = e / per_tok;
      const int in_tok = static_cast<int>(e - tok * per_tok), h = in_tok / p.units;
      const int b = static_cast<int>(tok / p.budget), slot = static_cast<int>(tok - static_cast<long long>(b) * p.budget);
      const int j = p.kept[(static_cast<long long>(b) * p.Hkv + h) * p.budget + slot];
      if (j < 0) continue;
      const int np = slot / p.page_size, op = j / p.page_size;
      const int dst = p.new_table[static_cast<long long>(b) * p.new_max_pages + np];
      const int src = p.table[static_cast<long long>(b) * p.max_pages + op];
      if (dst < 0 || dst >= p.n_pages || src < 0 || src >= p.n_pages) continue;
      const long long from = (static_cast<long long>(src) * p.page_size + (j - op * p.page_size)) * per_tok + in_tok;
      to[i] = (static_cast<long long>(dst) * p.page_size + (slot - np * p.page_size)) * per_tok + in_tok;
      a[i] = __ldcs(p.kp + from);
      c[i] = __ldcs(p.vp + from);
    }
#pragma unroll
    for (int i = 0; i < kMvUnroll; ++i)
      if (to[i] >= 0) {
        __stcs(p.kp + to[i], a[i]);
        __stcs(p.vp + to[i], c[i]);
      }
  }
}

// log2 of a power of two, else -1
int shift_of(int x) {
  for (int i = 0; i < 31; ++i)
    if (x == 1 << i) return i;
  return -1;
}
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Sizes of a decode call that its launch and its workspace share.
struct DecSizes {
  int ctas, rows, ng, wt_chunks;
  long long score_stride;
  size_t slots, stats, scores;   // bytes, multiples of 16
};
DecSizes dec_sizes(int B, int Hq, int Hkv, int D, long long tokens, bool weights) {
  DecSizes s;
  const int G = Hq / Hkv;
  s.rows = std::min(G, 16);
  s.ng = (G + 15) / 16;
  const long long tiles = ceil_div(tokens, kTile);
  s.ctas = static_cast<int>(std::max(1LL, std::min<long long>(kDecCtas, ceil_div(tiles * B * Hkv * s.ng, kMinTiles))));
  s.score_stride = tiles * kTile;
  s.wt_chunks = !weights ? 0 : static_cast<int>(std::min(ceil_div(std::max(tokens, 1LL), kWtPos),
                                                         std::max<long long>(1, kWtBlocks / (static_cast<long long>(B) * Hkv))));
  s.slots = static_cast<size_t>(s.ctas) * 2 * s.rows * (D + 4) * 4;
  s.stats = weights ? (static_cast<size_t>(B) * Hq * 8 + 15) / 16 * 16 : 0;
  s.scores = weights ? static_cast<size_t>(B) * Hq * s.score_stride * 4 : 0;
  return s;
}

template <int kD, bool kF32, bool kWide, bool kScores>
cudaError_t launch_split(const DecParams &p, cudaStream_t st) {
  constexpr int warps = dec_warps(kF32, kWide), smem = dec_smem(kD, warps);
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(decode_split_kernel<kD, kF32, kWide, kScores>), smem);
  if (e != cudaSuccess) return e;
  decode_split_kernel<kD, kF32, kWide, kScores><<<p.ctas, 32 * warps, smem, st>>>(p);
  return cudaGetLastError();
}
template <int kD, bool kF32>
cudaError_t launch_split(const DecParams &p, cudaStream_t st) {
  if (p.G > 8)
    return p.weight_sums ? launch_split<kD, kF32, true, true>(p, st) : launch_split<kD, kF32, true, false>(p, st);
  return p.weight_sums ? launch_split<kD, kF32, false, true>(p, st) : launch_split<kD, kF32, false, false>(p, st);
}

// Launches `kernel` so that it may start while the launch before it drains; it
// waits (griddepcontrol.wait) before it reads what that one writes.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), unsigned grid, unsigned block, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_pages_write(const PagesArgs &a, const void *k, const void *v, const int *starts, int T,
                                  long long k_stride, long long v_stride, cudaStream_t st) {
  WriteParams p;
  p.k = static_cast<const uint4 *>(k), p.v = static_cast<const uint4 *>(v);
  p.kp = static_cast<uint4 *>(a.k_pages), p.vp = static_cast<uint4 *>(a.v_pages);
  p.table = a.table, p.starts = starts, p.lengths = a.lengths;
  p.ntok = static_cast<long long>(a.B) * T;
  p.k_stride = k_stride / 8, p.v_stride = v_stride / 8;
  p.T = T;
  p.units = a.Hkv * a.D / 8;
  p.n_pages = a.n_pages, p.page_size = a.page_size, p.max_pages = a.max_pages;
  // as many tokens per block as give each thread kWrUnroll units, fewer while
  // the grid would not fill the GPU
  p.tpb = static_cast<int>(std::max(1LL, std::min<long long>(kWrThr * kWrUnroll / p.units, ceil_div(p.ntok, 1216))));
  const long long blocks = ceil_div(p.ntok, p.tpb);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kv_pages_write_kernel<<<static_cast<unsigned>(blocks), kWrThr, 0, st>>>(p);
  return cudaGetLastError();
}

size_t decode_paged_workspace_bytes(int B, int Hq, int Hkv, int D, long long tokens, bool weights) {
  const DecSizes s = dec_sizes(B, Hq, Hkv, D, tokens, weights);
  return s.slots + s.stats + s.scores;
}

cudaError_t launch_attn_decode_paged(const PagesArgs &a, const void *q, int bf16, float *weight_sums, void *o, int Hq,
                                     int window, int sinks, float scale, void *ws, cudaStream_t st) {
  long long tokens = static_cast<long long>(a.page_size) * a.max_pages;
  DecParams p;
  p.cap = static_cast<int>(tokens);
  if (window > 0) tokens = std::min(tokens, static_cast<long long>(window) + sinks);
  const DecSizes s = dec_sizes(a.B, Hq, a.Hkv, a.D, tokens, weight_sums != nullptr);
  p.q = q, p.o = o;
  p.kp = static_cast<const __nv_bfloat16 *>(a.k_pages), p.vp = static_cast<const __nv_bfloat16 *>(a.v_pages);
  p.table = a.table, p.lengths = a.lengths;
  p.weight_sums = weight_sums;
  unsigned char *w = static_cast<unsigned char *>(ws);
  p.slots = reinterpret_cast<float *>(w);
  p.stats = reinterpret_cast<float2 *>(w + s.slots);
  p.scores = reinterpret_cast<float *>(w + s.slots + s.stats);
  p.score_stride = s.score_stride;
  p.B = a.B, p.Hq = Hq, p.Hkv = a.Hkv, p.D = a.D, p.G = Hq / a.Hkv, p.ng = s.ng, p.rows = s.rows;
  p.n_pages = a.n_pages, p.page_size = a.page_size, p.max_pages = a.max_pages;
  p.page_shift = shift_of(a.page_size);
  p.window = window, p.sinks = sinks;
  p.q_bf16 = bf16, p.ctas = s.ctas, p.wt_chunks = s.wt_chunks;
  p.wt_len = s.wt_chunks ? static_cast<int>(ceil_div(std::max(tokens, 1LL), s.wt_chunks)) : 0;
  p.sl2 = scale * 1.4426950408889634f;
  const long long blocks = p.ctas + static_cast<long long>(s.wt_chunks) * a.B * a.Hkv;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaError_t e = a.D == 64 ? (bf16 ? launch_split<64, false>(p, st) : launch_split<64, true>(p, st))
                            : (bf16 ? launch_split<128, false>(p, st) : launch_split<128, true>(p, st));
  if (e != cudaSuccess) return e;
  return launch_dependent(decode_finish_kernel, static_cast<unsigned>(blocks), kFinThr, st, p);
}

cudaError_t launch_kv_pages_evict(const PagesArgs &a, const float *weight_sums, const int *new_table, int *kept,
                                  int *new_lengths, float *new_weight_sums, int new_max_pages, int budget, int sinks,
                                  int recent, cudaStream_t st) {
  EvictParams p;
  p.kp = static_cast<uint4 *>(a.k_pages), p.vp = static_cast<uint4 *>(a.v_pages);
  p.table = a.table, p.lengths = a.lengths, p.new_table = new_table;
  p.sums = weight_sums;
  p.kept = kept, p.new_lengths = new_lengths, p.new_sums = new_weight_sums;
  p.B = a.B, p.Hkv = a.Hkv, p.units = a.D / 8;
  p.n_pages = a.n_pages, p.page_size = a.page_size, p.max_pages = a.max_pages;
  p.cap = a.page_size * a.max_pages;
  p.new_max_pages = new_max_pages, p.new_cap = a.page_size * new_max_pages;
  p.budget = budget, p.sinks = sinks, p.recent = recent;
  const long long blocks = static_cast<long long>(a.B) * a.Hkv;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  p.page_shift = shift_of(a.page_size);
  const bool cached = p.cap <= kEvCached;
  auto select = cached ? evict_select_kernel<true> : evict_select_kernel<false>;
  const int smem = cached ? p.cap * 4 : 0;
  cudaError_t e = cached ? ensure_dynamic_smem(reinterpret_cast<const void *>(select), kEvCached * 4) : cudaSuccess;
  if (e != cudaSuccess) return e;
  select<<<static_cast<unsigned>(blocks), kEvThr, smem, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.n_pages == 0 || a.max_pages == 0) return e;
  const long long total = blocks * budget * p.units;
  const long long grid = std::min<long long>(ceil_div(total, kMvThr * kMvUnroll), 152 * 32);
  return launch_dependent(evict_move_kernel, static_cast<unsigned>(grid), kMvThr, st, p, total);
}

}  // namespace abw
