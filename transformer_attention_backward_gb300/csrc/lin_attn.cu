// Linear attention with a decay for each KV head: chunked forward and
// backward over whole sequences, and the recurrent form for single tokens.
//
//   S_t = a S_(t-1) + k_t v_t^T,   o_t = scale S_t^T q_t,   a = exp(log_decay)
//
// Over a chunk of 128 tokens that starts with the state S (local t, j; L
// valid tokens):
//   o_t = sum_(j<=t) scale a^(t-j) (q_t . k_j) v_j  +  scale a^(t+1) S^T q_t
//   S' = a^L S + sum_j a^(L-1-j) k_j v_j^T
// and for the gradients, with R the gradient of the state behind the chunk:
//   dq_t = sum_(j<=t) scale a^(t-j) (do_t . v_j) k_j  +  scale a^(t+1) S do_t
//   dk_j = sum_(t>=j) scale a^(t-j) (v_j . do_t) q_t  +  a^(L-1-j) R v_j
//   dv_j = sum_(t>=j) scale a^(t-j) (k_j . q_t) do_t  +  a^(L-1-j) R^T k_j
//   R' = a^L R + sum_t scale a^(t+1) q_t do_t^T        (towards earlier chunks)
// So o, dq, dk and dv are one operation, out = mask(A B^T) C + row factor
// (A S), on other operands, and S and R are one recurrence on other operands
// and in the other direction.  Two launches:
//   lin_state : walks the chunks of one (batch, KV head) and leaves the state
//               that enters each of them as a bf16 tile in the workspace
//   lin_out   : one item per 128 output rows; everything it needs is there,
//               so items run in any order (lin_grad, where every query head has
//               a KV head of its own: dq, dk and dv of a chunk in one item)
// Short sequences without states at their ends take the second alone: an item
// goes through the products of the chunks before it (behind it) as well, which
// for a few chunks costs less than the walk and its launch.
// Decay powers are a^0 and below, so strong decays underflow to 0 and never
// overflow; next to the diagonal alone a row's factor may be above 1 (a^-31 at
// most, where that fits, MaskWeights).
#include <math.h>

#include "abw_host.h"
#include "tcgen05.cuh"

namespace abw {
namespace {

constexpr int kC = 128;               // tokens per chunk
constexpr int kSub = 64;              // tokens per TMA box: half a chunk
// Most chunks whose outputs are formed without states; a group of query heads
// shares its KV head's states, so fewer where there are groups.  GPU time in us
// of forward / backward, with the walk and directly: 2 x 512 tokens of 20/5 heads
// 11.9 / 21.0, 9.7 / 21.0 (and a launch less); 2 x 640 13.2 / 23.5, 11.6 / 27.0; 8 x
// 768 of 16/4 25.7 / 59, 31.3 / 72; 4 x 768 of 20/20 31 / 59, 23 / 54; 4 x 1024
// 39 / 73, 32 / 82; 1 x 1280 of 32/32 19.3 / 39, 20.4 / 49.
constexpr int direct_chunks(bool backward, int G) {
  return G == 1 ? (backward ? 6 : 8) : (backward ? 4 : 5);
}

__device__ __forceinline__ uint32_t lpack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

// 2^x to 2 ulp; results below the normal range are 0.
__device__ __forceinline__ float lexp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2 of the decay, held above -1e30 so that 0 * log2 a is 0 for a = 0.
__device__ __forceinline__ float log2_decay(float log_decay) {
  const float l2 = log_decay * 1.4426950408889634f;
  return l2 < -1e30f ? -1e30f : l2;
}

// a^n for the decay of a step of n tokens: the float below it, and what it misses
// of it.  A head that hardly decays collects that over some 1 / (1 - a^n) steps
// (one float alone: 1.7e-5 of the state after 100,000 tokens in chunks, 1.8e-4
// after 4,000 single ones), so 1 - a^n is what is formed to fp32; stronger decays
// forget sooner, and take strong(), a^n as one float.
template <typename F>
__device__ __forceinline__ float2 step_decay(float log_decay, int n, F strong) {
  const float m = -expm1f(log_decay * static_cast<float>(n));
  if (!(m < 0.5f)) return make_float2(strong(), 0.f);
  const float a = __fsub_rd(1.f, m);
  return make_float2(a, (1.f - a) - m);                       // (both differences are exact)
}
// Chunks after which the state makes up for what they missed, in one
// multiplication (with each chunk 108 us for 8192 tokens of 32 heads, as the walk
// has few issue slots to spare; so 105, with no more than one float 104).  What
// joined the state since the last time is moved by less than kOwed 2^-24.
constexpr int kOwed = 16;

__device__ __forceinline__ int seq_len(const int *lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

// Waits of the two tensor-core kernels.  A barrier that has completed costs one
// access: shared memory is busy, and each access of a warp that has little
// else to do stands in its queue.
__device__ __forceinline__ bool lin_wait_slow(uint32_t br, uint32_t parity, uint32_t bars, volatile int *abort_flag,
                                              unsigned int kernel, unsigned int *err, unsigned long long limit_ns) {
  if (*abort_flag) return false;      // a wait has run out: all others return
  if (mbar_wait_bounded(br, parity, limit_ns)) return true;
  *abort_flag = 1;
  report_timeout(err, kernel, (br - bars) / 8);
  return false;
}
struct LinWait {
  uint32_t bars;                      // shared address of barrier 0
  volatile int *abort_flag;
  unsigned int kernel;
  const WaitCtl &ctl;

  __device__ __forceinline__ uint32_t bar(int i) const { return bars + i * 8; }
  // the MMA warps, before their first wait, which is on barrier i
  __device__ __forceinline__ bool start(int i) const { return may_wait(ctl, abort_flag, kernel, i); }
  // one thread, or each lane for its own barrier
  __device__ __forceinline__ bool one(uint32_t br, uint32_t parity) const {
    return mbar_try_wait(br, parity) || lin_wait_slow(br, parity, bars, abort_flag, kernel, ctl.err, ctl.limit_ns);
  }
  // a whole warp
  __device__ __forceinline__ bool warp(uint32_t br, uint32_t parity) const {
    return __all_sync(0xffffffffu, mbar_try_wait(br, parity)) ||
           __all_sync(0xffffffffu, lin_wait_slow(br, parity, bars, abort_flag, kernel, ctl.err, ctl.limit_ns));
  }
};

struct LinSizes {
  int B, T, Hq, Hkv, G, NC;
  float scale;
  const float *log_decay;             // [Hkv]
  const int *lengths;                 // [B] or null
};

// ---------------------------------------------------------------------------
// lin_state: the recurrence over the chunks of one (batch, KV head, 32 columns
// of the state).  Role F: X = K, Y = V, weights a^(L-1-j), chunks in order.
// Role R: X = Q, Y = dO of every query head of the group, weights
// scale a^(t+1), chunks from the last to the first.  In steps of 64 tokens:
//   U = X^T (w o Y)    M = D state rows, N = 32 columns a term, K = 64 tokens
// The fp32 product w o Y enters the tensor core as a sum of NS bf16 terms
// (each the rounding of what the ones before leave), side by side as N: two
// terms are good to 2^-17, which is far below the rounding of the bf16 state
// tiles; three are good to 2^-25, for a state that leaves in fp32.  The state
// itself stays in fp32 registers, and each step's U is added there: sums over
// steps or terms inside the tensor core would cut off bits of the
// accumulator's size at every one (measured: 5 times the error).
// Bound by shared memory: a step moves 20 KB into it by TMA, 16 KB for the
// weighted rows (read, formed, written) and 28 KB out of it to the tensor core,
// some 500 of the 650 cycles that a step takes.  What hides the rest is steps
// under way: a ring of 6 (X, Y) slots, four buffers of weighted rows, filled in
// turn by three groups of warps, two MMA warps and two buffers of U.  The walk
// takes 54 us for 8192 tokens of 32 heads with states (48 where none leaves: two
// terms) and 80 for 640 chains of 2048 tokens.  Tried, against what it took at the
// time: two groups 59 and four 58 (55); deeper rings no change; 64 columns a CTA,
// half as many chains, 95 and 81 (52 and 76); X once for all CTAs of a chain, by
// multicast, 57 and 85 (55 and 79).
// Warps: 0 TMA, 1 and 18 MMA, 2-13 weights, 14-17 state.
// ---------------------------------------------------------------------------
constexpr int kSGroups = 3;                          // groups of four warps that form weighted rows
constexpr int kSThr = 64 + kSGroups * 128 + 128 + 32;
constexpr int kSMma2 = kSThr / 32 - 1;               // the second MMA warp
constexpr int kCW = 32;

// A slot: X (two 64-column parts of 8 KB) | Y (32 columns, 4 KB); the weighted
// rows, which live from their forming to their product only, have buffers of
// their own (two terms of 32 columns to an 8 KB part).
template <int NS>
struct StateShape {
  static constexpr int kN = NS * kCW;                // columns of U
  static constexpr int kSlot = 2 * 8192 + 4096;
  // A group comes back to the slots it has waited for before: loads complete in
  // any order, and with slots that change hands a wait could take the phase
  // before the last for the one it waits for.
  static constexpr int kRing = 6;
  static_assert(kRing % kSGroups == 0, "a slot belongs to one group");
  static constexpr int kWSlot = (kN + 63) / 64 * 8192, kWRing = 4;
  static_assert(kWRing >= kSGroups, "every group has a buffer to work on");
  static constexpr int kOffW = kRing * kSlot;
  static constexpr int kOffBar = kOffW + kWRing * kWSlot;
  static constexpr int kFull = 0, kDone = kRing, kW = 2 * kRing, kUEmpty = kW + kWRing, kFinal = kUEmpty + 2;
  static constexpr int kOffTmem = kOffBar + (kFinal + 2) * 8, kOffAbort = kOffTmem + 4;
  static constexpr int kSmem = kOffBar + 256 + 1024;                   // + alignment slack
  static_assert(kOffAbort + 4 <= kOffBar + 256 && kSmem <= 232448 && kOffW % 1024 == 0, "state kernel shared memory");
};

struct LinStateParams {
  LinSizes z;
  int first_role, nroles;             // 0 F, 1 R
  __nv_bfloat16 *tiles[2];            // [B][Hkv][NC][D * D], 128B-swizzled
  const float *start[2];              // initial_state, dfinal_state (or null)
  float *end[2];                      // final_state, dinitial_state (or null)
  WaitCtl wait;
};

template <int D, int NS>
__global__ void __launch_bounds__(kSThr, 1)
    lin_state_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV32,
                     const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO32,
                     const __grid_constant__ LinStateParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  using Z = StateShape<NS>;
  constexpr int NH = D / 64, NP = D / kCW;
  const int part = blockIdx.x % NP, unit = blockIdx.x / NP;   // kCW columns of the state
  const int nbh = p.z.B * p.z.Hkv;
  const int role = p.first_role + unit / nbh, bh = unit % nbh;
  const int b = bh / p.z.Hkv, kv = bh % p.z.Hkv;
  const int len = seq_len(p.z.lengths, b, p.z.T);
  const int ncb = (len + kC - 1) / kC;                        // chunks that hold tokens
  const int nst = p.end[role] ? ncb : max(ncb - 1, 0);        // chunks to add
  const int gi = role ? 2 * p.z.G : 2;                        // steps per chunk: heads x halves
  const float l2 = log2_decay(p.z.log_decay[kv]);
  auto chunk = [&](int m) -> int { return role ? ncb - 1 - m : m; };

  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Z::kOffAbort);
  const LinWait lw{sb + Z::kOffBar, abort_flag, kSiteLinState, p.wait};
  auto bar = [&](int i) -> uint32_t { return lw.bar(i); };
  auto wt = [&](uint32_t br, uint32_t parity) -> bool { return lw.one(br, parity); };
  auto wtw = [&](uint32_t br, uint32_t parity) -> bool { return lw.warp(br, parity); };

  if (tid == 0) {
    for (int s = 0; s < Z::kRing; ++s) {
      mbar_init(bar(Z::kFull + s), 1);
      mbar_init(bar(Z::kDone + s), 1);
    }
    for (int s = 0; s < Z::kWRing; ++s) mbar_init(bar(Z::kW + s), 128);
    for (int s = 0; s < 2; ++s) mbar_init(bar(Z::kUEmpty + s), 128);
    for (int s = 0; s < 2; ++s) mbar_init(bar(Z::kFinal + s), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(sb + Z::kOffTmem, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + Z::kOffTmem);
  // the output kernel's CTAs may start on SMs that this grid's tail leaves idle;
  // they wait for its end before they read a state
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int steps = nst * gi;
  // step i: tokens [64 (i & 1), 64 (i & 1) + 64) of chunk i / gi, head (i % gi) / 2
  auto phase = [](int i) -> uint32_t { return static_cast<uint32_t>(i / Z::kRing) & 1u; };

  if (warp == 0) {
    // ============================ TMA producer ============================
    if (lane == 0) {
      const CUtensorMap *mx = role ? &tmQ : &tmK, *my = role ? &tmDO32 : &tmV32;
      prefetch_tensormap(mx);
      prefetch_tensormap(my);
      int issued = 0;
      for (int i = 0, s = 0, ph = 1, m = 0, g = 0; i < steps; ++i) {
        if (!wt(bar(Z::kDone + s), ph)) break;
        const int h = role ? kv * p.z.G + g / 2 : kv, t0 = chunk(m) * kC + (g & 1) * kSub;
        const uint32_t st = sb + s * Z::kSlot, fb = bar(Z::kFull + s);
        mbar_arrive_expect_tx(fb, NH * 8192 + 4096);
        for (int x = 0; x < NH; ++x) tma_load_4d(st + x * 8192, mx, x * 64, h, t0, b, fb);
        tma_load_4d(st + 16384, my, part * kCW, h, t0, b, fb);
        issued = i + 1;
        if (++g == gi) g = 0, ++m;
        if (++s == Z::kRing) s = 0, ph ^= 1;
      }
      // The last load of every slot has landed before the block may end, whoever
      // gives up and when (otherwise this finds every phase complete).
      for (int i = (issued > Z::kRing ? issued - Z::kRing : 0); i < issued; ++i)
        mbar_wait_bounded(bar(Z::kFull + i % Z::kRing), phase(i), 2000000000ull);
    }
  } else if (warp == 1 || warp == kSMma2) {
    // ============================ MMA issuers =============================
    // Two warps take the steps in turn: a step's hundred instructions of one
    // warp among busy ones take about as long as the step.
    // X is the M-major A operand.  For D = 64 rows 64-127 of A come from the
    // unused second part of the X slot; they only reach TMEM lanes 64-127,
    // which nobody reads.
    constexpr uint32_t id_u = tc::idesc_bf16_f32(128, Z::kN, 1, 1);
    const int u = warp == 1 ? 0 : 1;
    const uint64_t dX = tc::sdesc_sw128(sb, 8192, 1024);
    const uint64_t dW = tc::sdesc_sw128(sb + Z::kOffW, 8192, 1024);
    const bool ok = u >= steps || lw.start(Z::kW + u);
    for (int i = u, s = u, w = u, wph = 0, uph = 1; ok && i < steps; i += 2, uph ^= 1) {
      // (weighted rows that are there were formed from a stage that is there)
      if (!wtw(bar(Z::kUEmpty + u), uph) || !wtw(bar(Z::kW + w), wph)) break;
      tc::fence_after_sync();
      const uint64_t so = static_cast<uint64_t>(s * Z::kSlot) >> 4, wo = static_cast<uint64_t>(w * Z::kWSlot) >> 4;
      // the terms side by side as N: X is read once for all of them
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        tc::mma_bf16_w(tmem + u * 256, dX + so + ((kk * 2048) >> 4), dW + wo + ((kk * 2048) >> 4), id_u, kk > 0);
      // one signal for all who wait for the step: the stage and the weighted
      // rows are free, U is there
      tc::commit_w(bar(Z::kDone + s));
      if ((s += 2) >= Z::kRing) s -= Z::kRing;
      if ((w += 2) >= Z::kWRing) w -= Z::kWRing, wph ^= 1;
    }
    tc::commit_w(bar(Z::kFinal + u));
    mbar_wait_bounded(bar(Z::kFinal + u), 0, 2000000000ull);   // every MMA has completed
  } else if (warp < 2 + 4 * kSGroups) {
    // ============================ weights =================================
    const int grp = (warp - 2) >> 2, wtid = (tid - 64) & 127;
    auto weight = [&](int row, int L) -> float {
      return role ? p.z.scale * lexp2(l2 * static_cast<float>(row + 1)) : lexp2(l2 * static_cast<float>(L - 1 - row));
    };
    float whole[2][kCW / 16];                                 // of this thread's rows in a whole chunk
#pragma unroll
    for (int c = 0; c < 2 * (kCW / 16); ++c)
      whole[c & 1][c >> 1] = weight(((wtid + 128 * (c >> 1)) >> 2) + (c & 1) * kSub, kC);
    for (int i = grp, s = grp, ph = 0, w = grp, m = 0, g = grp; i < steps; i += kSGroups) {
      while (g >= gi) g -= gi, ++m;
      const int u = g & 1;                                    // half of the chunk
      if (!wtw(bar(Z::kFull + s), ph)) break;
      // the buffer's last product, that of step i - kWRing, is done
      if (i >= Z::kWRing && !wtw(bar(Z::kDone + (i - Z::kWRing) % Z::kRing), ((i - Z::kWRing) / Z::kRing) & 1)) break;
      const int L = min(kC, len - chunk(m) * kC);
      unsigned char *st = smem + s * Z::kSlot, *wb = smem + Z::kOffW + w * Z::kWSlot;
#pragma unroll
      for (int c = 0; c < kCW / 16; ++c) {
        // 16-byte piece j of the row of token `row` of the chunk
        const int id = wtid + 128 * c, r = id >> 2, j = id & 3, row = r + u * kSub;
        uint4 out[NS];
        if (L == kC || row < L) {
          const float wgt = L < kC ? weight(row, L) : u ? whole[1][c] : whole[0][c];
          const uint4 y = *reinterpret_cast<const uint4 *>(st + 16384 + 16 * id);
          const uint32_t yi[4] = {y.x, y.y, y.z, y.w};
          uint32_t o[NS][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 f = __fmul2_rn(make_float2(bf16_lo(yi[e]), bf16_hi(yi[e])), make_float2(wgt, wgt));
#pragma unroll
            for (int t = 0; t < NS; ++t) {
              o[t][e] = lpack2(f.x, f.y);
              f = __ffma2_rn(make_float2(bf16_lo(o[t][e]), bf16_hi(o[t][e])), make_float2(-1.f, -1.f), f);
            }
          }
#pragma unroll
          for (int t = 0; t < NS; ++t) out[t] = make_uint4(o[t][0], o[t][1], o[t][2], o[t][3]);
        } else {
#pragma unroll
          for (int t = 0; t < NS; ++t) out[t] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < NS; ++t)
          *reinterpret_cast<uint4 *>(wb + (t >> 1) * 8192 + r * 128 + ((((t & 1) * 4 + j) ^ (r & 7)) << 4)) = out[t];
      }
      if (L < kC) {
        // rows behind the sequence may hold anything: 0 * NaN must not reach U
        for (int id = wtid; id < NH * 512; id += 128)
          if (((id >> 3) & 63) + u * kSub >= L) *reinterpret_cast<uint4 *>(st + 16 * id) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(Z::kW + w));
      if ((w += kSGroups) >= Z::kWRing) w -= Z::kWRing;
      if ((s += kSGroups) >= Z::kRing) s -= Z::kRing, ph ^= 1;
      g += kSGroups;
    }
  } else {
    // ============================ state ===================================
    const int qd = warp & 3, row = 32 * qd + lane;            // TMEM lane quarter, state row
    const uint32_t lanebase = static_cast<uint32_t>(32 * qd) << 16;
    const bool live = row < D;
    const size_t at = (static_cast<size_t>(bh) * D + row) * D + part * kCW;
    float2 S[kCW / 2];
#pragma unroll
    for (int c = 0; c < kCW / 2; ++c) S[c] = make_float2(0.f, 0.f);
    if (live && p.start[role]) {
      const float4 *src = reinterpret_cast<const float4 *>(p.start[role] + at);
#pragma unroll
      for (int c = 0; c < kCW / 4; ++c) {
        const float4 v = src[c];
        S[2 * c] = make_float2(v.x, v.y), S[2 * c + 1] = make_float2(v.z, v.w);
      }
    }
    const float2 whole = step_decay(p.z.log_decay[kv], kC, [&] { return lexp2(l2 * kC); });
    const float rest = lexp2(l2 * static_cast<float>(len - (ncb - 1) * kC));   // of the last chunk
    int owed = 0;
    auto settle = [&] {
      if (whole.y > 0.f) {                                    // (an infinity stays one)
        const float f = whole.y / whole.x * static_cast<float>(owed);
#pragma unroll
        for (int c = 0; c < kCW / 2; ++c) S[c] = __ffma2_rn(make_float2(f, f), S[c], S[c]);
      }
      owed = 0;
    };
    bool ok = true;
    int s = 0, ph = 0, u = 0;
    for (int m = 0; m < ncb; ++m) {
      const int n = chunk(m);
      if (owed == kOwed) settle();
      if (live && p.tiles[role] && (m > 0 || p.start[role])) {
        // the row's part, in the order of a 128-byte swizzled tile
        unsigned char *dst = reinterpret_cast<unsigned char *>(p.tiles[role]) +
                             (static_cast<size_t>(bh) * p.z.NC + n) * (D * D * 2) + part / 2 * (D * 128) + row * 128;
#pragma unroll
        for (int c = 0; c < kCW / 8; ++c)
          *reinterpret_cast<uint4 *>(dst + ((((part & 1) * 4 + c) ^ (row & 7)) << 4)) =
              make_uint4(lpack2(S[4 * c].x, S[4 * c].y), lpack2(S[4 * c + 1].x, S[4 * c + 1].y),
                         lpack2(S[4 * c + 2].x, S[4 * c + 2].y), lpack2(S[4 * c + 3].x, S[4 * c + 3].y));
      }
      if (m >= nst) break;
      for (int g = 0; g < gi; ++g) {
        if (!wtw(bar(Z::kDone + s), ph)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const float dec = g > 0 ? 1.f : n + 1 < ncb ? whole.x : rest;
#pragma unroll
        for (int x = 0; x < kCW / 16; ++x) {
          float2 t[8];
#pragma unroll
          for (int e = NS - 1; e >= 0; --e) {                 // the small terms first
            uint32_t v[16];
            tc::ld16_wait(tmem + lanebase + u * 256 + e * kCW + x * 16, v);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float2 w = make_float2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1]));
              t[c] = e == NS - 1 ? w : __fadd2_rn(t[c], w);
            }
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) S[x * 8 + c] = __ffma2_rn(make_float2(dec, dec), S[x * 8 + c], t[c]);
        }
        tc::fence_before_sync();
        mbar_arrive(bar(Z::kUEmpty + u));
        u ^= 1;
        if (++s == Z::kRing) s = 0, ph ^= 1;
      }
      if (!ok) break;
      if (n + 1 < ncb) ++owed;
    }
    if (owed) settle();
    if (ok && live && p.end[role]) {
      float4 *dst = reinterpret_cast<float4 *>(p.end[role] + at);
#pragma unroll
      for (int c = 0; c < kCW / 4; ++c) dst[c] = make_float4(S[2 * c].x, S[2 * c].y, S[2 * c + 1].x, S[2 * c + 1].y);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// lin_out: out = mask(A B^T) C + factor (A S), one item per (output, batch,
// head, chunk):
//   role 0  o  : A = Q,  B = K,  C = V,  S
//   role 1  dq : A = dO, B = V,  C = K,  S^T
//   role 2  dk : A = V,  B = dO, C = Q,  R^T    summed over the group's heads
//   role 3  dv : A = K,  B = Q,  C = dO, R      summed over the group's heads
// Persistent, one CTA per SM.  Tiles of 32 KB: A, which stays for the whole
// item, alternates between two slots; the others arrive through a ring of 5
// in the order B, [S], C, B, C, ...  Both run on across items, so the loads of
// the next item are in flight while this one computes.  The state
// tile serves S and S^T: the first as an N-major, the second as a K-major B
// operand.  Scores are rounded to bf16 as the next product's A operand (as in
// the softmax attention), the state tile is bf16; products accumulate in fp32
// and the two parts meet in fp32, each element rounded once on its way out.
// TMEM: [0,256) two score / P buffers, [256,384) mask(A B^T) C, [384,512) A S.
// Warps: 0 TMA loads, 1 MMA, 2-9 mask and output (thread = row and half of the
// columns: what an item waits for is the length of this chain, and the halves
// go side by side), 10 TMA stores.  The output tile is written over A, which
// no product needs by then, and leaves from there by TMA (16-byte stores by
// the rows' threads took 2,400 cycles of an item's 8,300).
// Over long sequences bound by memory: the forward of 8192 tokens of 32 heads
// takes 51-53 us behind the walk, its copies alone 50.  (Two sets of mask warps
// and scores formed an item ahead, as in lin_grad: no change here.)
// ---------------------------------------------------------------------------
constexpr int kOThr = 352;
constexpr int kOSlots = 5;            // of the ring; the two slots of A follow
constexpr int kOSlot = 32768;
constexpr int kOOffA = kOSlots * kOSlot;
constexpr int kOOffBar = kOOffA + 2 * kOSlot;
enum {
  kOBarFull = 0, kOBarEmpty = kOBarFull + kOSlots, kOBarAFull = kOBarEmpty + kOSlots, kOBarAEmpty = kOBarAFull + 2,
  kOBarS = kOBarAEmpty + 2, kOBarP = kOBarS + 2,
  kOBarStage = kOBarP + 2, kOBarO = kOBarStage + 2, kOBarOEmpty = kOBarO + 1, kOBarFinal = kOBarOEmpty + 1,
  kONumBars = kOBarFinal + 1
};
constexpr int kOOffTmem = kOOffBar + kONumBars * 8;
constexpr int kOOffAbort = kOOffTmem + 4;
constexpr int kOSmem = kOOffBar + 256 + 1024;        // + alignment slack
static_assert(kOOffAbort + 4 <= kOOffBar + 256 && kOSmem <= 232448, "output kernel shared memory");

struct LinOutParams {
  LinSizes z;
  int backward;
  int direct;                         // no state tiles: an item takes the other chunks itself
  int items;
  int start[2];                       // a state enters the first chunk / comes from behind the last
  const __nv_bfloat16 *tiles[2];
  __nv_bfloat16 *out[4];              // o, dq, dk, dv
  long long stride[4];                // elements between tokens of each output
  WaitCtl wait;
  CUtensorMap map[4];                 // of the outputs
};

struct LinItem {
  int role, b, kv, h, n, len, L, ns, gi;   // h: head of the output; ns: chunks of B and C; gi: (B, C) pairs
  bool st;                                 // has a state tile
};

// The item of a CTA's round r.  Where items differ in length rounds go back and
// forth: who had the longest of the first has the shortest of the second (2 x
// 512 tokens of 20/5 heads, backward: 21 us for 26).
__device__ __forceinline__ int item_at(const LinOutParams &p, int r) {
  const int g = gridDim.x, c = blockIdx.x;
  return r * g + (p.direct && (r & 1) ? g - 1 - c : c);
}

__device__ __noinline__ LinItem lin_item(const LinOutParams &p, int i) {
  LinItem it;
  const int NC = p.z.NC, G = p.z.G;
  int g = 0;
  if (!p.backward) {
    it.role = 0;
    g = i % G;
    i /= G;
  } else if (G == 1) {                // three outputs of one chunk next to each other: they share its tiles
    it.role = 1 + i % 3;
    i /= 3;
  } else {                            // the items that sum over the group first
    const int heavy = 2 * p.z.B * p.z.Hkv * NC;
    if (i < heavy) {
      it.role = 2 + (i & 1);
      i >>= 1;
    } else {
      i -= heavy;
      it.role = 1;
      g = i % G;
      i /= G;
    }
  }
  // heads before chunks: the CTAs of one moment read whole token rows
  it.kv = i % p.z.Hkv;
  i /= p.z.Hkv;
  it.n = i % NC;
  it.b = i / NC;
  if (p.direct) {                                             // the longer items first
    it.b = i % p.z.B;
    it.n = it.role < 2 ? NC - 1 - i / p.z.B : i / p.z.B;
  } else {
    it.n = NC - 1 - it.n, it.b = p.z.B - 1 - it.b;            // what lin_state has read last first: L2 still holds it
  }
  it.len = seq_len(p.z.lengths, it.b, p.z.T);
  it.L = min(kC, it.len - it.n * kC);
  if (it.role < 2) {
    it.h = it.kv * G + g;
    it.ns = p.direct ? it.n + 1 : 1;
    it.gi = it.ns;
    it.st = !p.direct && (it.n > 0 || p.start[0]);
  } else {
    it.h = it.kv;
    it.ns = p.direct ? max((it.len + kC - 1) / kC - it.n, 1) : 1;
    it.gi = G * it.ns;
    it.st = !p.direct && ((it.n + 1) * kC < it.len || p.start[1]);
  }
  return it;
}

// The output kernels start as programmatic dependents of lin_state: set up and
// with their first loads under way while it ends.  Nobody else starts before,
// so that no bounded wait runs while lin_state does.
__device__ __forceinline__ void wait_states() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The row and column powers of the weights scale a^(distance) of a score tile.
// Inside a block of 16 columns a weight is a power for the row times one for
// the column (pw).  Next to the diagonal the row's is above 1, up to a^-31;
// where that could overflow each weight is formed by itself.
struct MaskWeights {
  float l2, pw[16];
  bool mild;
  __device__ __forceinline__ MaskWeights(float l2_, bool rev) : l2(l2_), mild(l2_ > -3.8f) {
#pragma unroll
    for (int e = 0; e < 16; ++e) pw[e] = lexp2(l2 * static_cast<float>(rev ? e : 15 - e));
  }
};

// Scores to P in place, for one row and half of its columns: weights on and
// below the diagonal (rev: on and above it), 0 elsewhere, rounded to bf16.  far:
// chunks between the rows and the columns; L: columns that count.
__device__ __forceinline__ void mask_scores(uint32_t tS, const MaskWeights &w, float scale, int row, int qd, int hc,
                                            bool rev, int far, int L) {
  // A short loop over blocks of 16 columns: what all warps run over and
  // over stays in the instruction cache (unrolled, blocks on the
  // diagonal took 2,000 cycles).
#pragma unroll 1
  for (int c0 = 64 * hc; c0 < 64 * hc + 64; c0 += 16) {
    const bool inside = rev ? ((far || c0 >= 32 * qd + 31) && c0 + 16 <= L) : far || c0 + 15 <= 32 * qd;
    const bool outside = !far && (rev ? c0 + 15 < 32 * qd : c0 > 32 * qd + 31);
    uint32_t pk[8];
    if (outside) {
#pragma unroll
      for (int e = 0; e < 8; ++e) pk[e] = 0;
    } else {
      uint32_t sr[16];
      float v[16];
      tc::ld16_wait(tS + c0, sr);
      if (inside || w.mild || far) {
        const float base = scale * lexp2(w.l2 * static_cast<float>(far * kC + (rev ? c0 - row : row - c0 - 15)));
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(sr[e]) * (base * w.pw[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int gap = rev ? c0 + e - row : row - c0 - e;
          v[e] = __uint_as_float(sr[e]) * (scale * lexp2(w.l2 * static_cast<float>(gap)));
        }
      }
      if (!inside) {
        // columns of the block that count: from row on, or up to it
        const int lo = rev && !far ? row - c0 : 0, hi = min(rev || far ? 16 : row - c0 + 1, L - c0);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e < lo || e >= hi) v[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) pk[e] = lpack2(v[2 * e], v[2 * e + 1]);
    }
    // 16 columns c to the 8 columns 32 (c / 32) + 8 (c / 16 % 2)
    tc::st8_async(tS + (c0 & 96) + ((c0 >> 1) & 8), pk);
  }
}

// One row and half of its columns of P C + fac (A S) to the staged output tile,
// in the order of a 128-byte swizzled tile; rows behind the sequence are 0.
template <int D>
__device__ __forceinline__ void stage_rows(uint32_t tm, unsigned char *stage, int row, int hc, bool st, float fac,
                                           bool in) {
#pragma unroll 1
  for (int c = hc * (D / 2); c < (hc + 1) * (D / 2); c += 32) {
    float a[32], s[32];
    if (st) {
      tc::ld32x2_wait(tm + 256 + c, tm + 384 + c, a, s);
#pragma unroll
      for (int e = 0; e < 32; ++e) a[e] = fmaf(fac, s[e], a[e]);
    } else {
      tc::ld32_wait(tm + 256 + c, a);
    }
    // the row's 16-byte pieces, in the order of a 128-byte swizzled tile
#pragma unroll
    for (int e = 0; e < 32; e += 8)
      *reinterpret_cast<uint4 *>(stage + row * 128 + (c >> 6) * 16384 + ((((c & 63) + e) / 8 ^ (row & 7)) << 4)) =
          in ? make_uint4(lpack2(a[e], a[e + 1]), lpack2(a[e + 2], a[e + 3]), lpack2(a[e + 4], a[e + 5]),
                          lpack2(a[e + 6], a[e + 7]))
             : make_uint4(0, 0, 0, 0);
  }
}

template <int D>
__global__ void __launch_bounds__(kOThr, 1)
    lin_out_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                   const __grid_constant__ LinOutParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int NH = D / 64;

  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOOffAbort);
  const LinWait lw{sb + kOOffBar, abort_flag, kSiteLinOut, p.wait};
  auto bar = [&](int i) -> uint32_t { return lw.bar(i); };
  auto wt = [&](uint32_t br, uint32_t parity) -> bool { return lw.one(br, parity); };
  auto wtw = [&](uint32_t br, uint32_t parity) -> bool { return lw.warp(br, parity); };
  // load number q of the ring sits in slot q % kOSlots; its phase there
  auto phase = [](int q) -> uint32_t { return static_cast<uint32_t>(q / kOSlots) & 1u; };

  if (tid == 0) {
    for (int s = 0; s < kOSlots; ++s) {
      mbar_init(bar(kOBarFull + s), 1);
      mbar_init(bar(kOBarEmpty + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kOBarAFull + s), 1);
      mbar_init(bar(kOBarAEmpty + s), 1);
      mbar_init(bar(kOBarS + s), 1);
      mbar_init(bar(kOBarP + s), 256);
      mbar_init(bar(kOBarStage + s), 256);
    }
    mbar_init(bar(kOBarO), 1);
    mbar_init(bar(kOBarOEmpty), 256);
    mbar_init(bar(kOBarFinal), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(sb + kOOffTmem, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kOOffTmem);

  if (warp != 0) wait_states();
  if (warp == 0) {
    // ============================ TMA producer ============================
    if (lane == 0) {
      int q = 0, item = 0;
      bool ok = true, states = false;
      auto slot = [&](uint32_t bytes) -> bool {       // claims the next slot
        const int s = q % kOSlots;
        if (!wt(bar(kOBarEmpty + s), phase(q) ^ 1u)) return ok = false;
        mbar_arrive_expect_tx(bar(kOBarFull + s), bytes);
        ++q;
        return true;
      };
      auto tile = [&](const CUtensorMap *m, const LinItem &it, int h, int n) {
        if (!ok || !slot(NH * 16384)) return;
        const int s = (q - 1) % kOSlots;
        for (int x = 0; x < 2 * NH; ++x)
          tma_load_4d(sb + s * kOSlot + x * 8192, m, (x >> 1) * 64, h, n * kC + (x & 1) * kSub, it.b,
                      bar(kOBarFull + s));
      };
      for (int r = 0, i = item_at(p, 0); ok && i < p.items; i = item_at(p, ++r)) {
        const LinItem it = lin_item(p, i);
        if (it.L <= 0) continue;
        const CUtensorMap *ma = it.role == 0 ? &tmQ : it.role == 1 ? &tmDO : it.role == 2 ? &tmV : &tmK;
        const CUtensorMap *mb = it.role == 0 ? &tmK : it.role == 1 ? &tmV : it.role == 2 ? &tmDO : &tmQ;
        const CUtensorMap *mc = it.role == 0 ? &tmV : it.role == 1 ? &tmK : it.role == 2 ? &tmQ : &tmDO;
        const int as = item & 1;
        if (!wt(bar(kOBarAEmpty + as), ((item >> 1) & 1) ^ 1)) break;
        mbar_arrive_expect_tx(bar(kOBarAFull + as), NH * 16384);
        for (int x = 0; x < 2 * NH; ++x)
          tma_load_4d(sb + kOOffA + as * kOSlot + x * 8192, ma, (x >> 1) * 64, it.h, it.n * kC + (x & 1) * kSub, it.b,
                      bar(kOBarAFull + as));
        ++item;
        int hg = it.role < 2 ? it.kv : it.kv * p.z.G, far = 0;    // far: chunks away
        for (int g = 0; g < it.gi; ++g) {
          const int n = it.role < 2 ? it.n - far : it.n + far;
          tile(mb, it, hg, n);
          if (!states) wait_states();
          states = true;
          if (g == 0 && it.st && ok && slot(D * D * 2)) {
            const int s = (q - 1) % kOSlots;
            const __nv_bfloat16 *src = p.tiles[it.role >> 1] +
                                       (static_cast<size_t>(it.b * p.z.Hkv + it.kv) * p.z.NC + it.n) * (D * D);
            bulk_load(sb + s * kOSlot, src, D * D * 2, bar(kOBarFull + s));
          }
          tile(mc, it, hg, n);
          if (++far == it.ns) far = 0, ++hg;
        }
      }
      if (!states) wait_states();                             // nor does this grid end before it
      // the last load of every slot, before the block may end (as in lin_state)
      for (int x = (q > kOSlots ? q - kOSlots : 0); x < q; ++x)
        mbar_wait_bounded(bar(kOBarFull + x % kOSlots), phase(x), 2000000000ull);
      for (int x = (item > 2 ? item - 2 : 0); x < item; ++x)
        mbar_wait_bounded(bar(kOBarAFull + (x & 1)), (x >> 1) & 1, 2000000000ull);
    }
  } else if (warp == 1) {
    // ============================ MMA issuer ==============================
    constexpr uint32_t id_s = tc::idesc_bf16_f32(128, 128, 0, 0);   // A B^T
    constexpr uint32_t id_n = tc::idesc_bf16_f32(128, D, 0, 1);     // P C and A S: B operand N-major
    constexpr uint32_t id_k = tc::idesc_bf16_f32(128, D, 0, 0);     // A S^T: B operand K-major
    auto kmaj = [&](int q) { return tc::sdesc_sw128(sb + (q % kOSlots) * kOSlot, 16, 1024); };
    auto nmaj = [&](int q, uint32_t half) { return tc::sdesc_sw128(sb + (q % kOSlots) * kOSlot, half, 1024); };
    auto kstep = [](int kk, int half) -> uint32_t { return static_cast<uint32_t>((kk >> 2) * half + (kk & 3) * 32) >> 4; };
    int q = 0, ss = 0, item = 0;
    bool ok = true;
    auto full = [&](int x) -> bool { return wtw(bar(kOBarFull + x % kOSlots), phase(x)); };
    for (int r = 0, i = item_at(p, 0); ok && i < p.items; i = item_at(p, ++r)) {
      const LinItem it = lin_item(p, i);
      if (it.L <= 0) continue;
      const int q0 = q, st = it.st ? 1 : 0, as = item & 1;
      auto qb = [&](int g) { return q0 + (g ? st + 2 * g : 0); };
      const uint64_t dA = tc::sdesc_sw128(sb + kOOffA + as * kOSlot, 16, 1024);
      // A B^T into the score buffer that held P two steps ago (its product
      // was issued before: the tensor core works in order)
      auto scores = [&](int g) -> bool {
        if (!full(qb(g))) return false;
        tc::fence_after_sync();
        const uint64_t dB = kmaj(qb(g));
        const uint32_t tS = tmem + ((ss + g) & 1) * 128;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) tc::mma_bf16_w(tS, dA + kstep(kk, 16384), dB + kstep(kk, 16384), id_s, kk > 0);
        tc::commit_w(bar(kOBarS + ((ss + g) & 1)));
        tc::commit_w(bar(kOBarEmpty + qb(g) % kOSlots));
        return true;
      };
      ok = (item > 0 || lw.start(kOBarAFull)) && wtw(bar(kOBarAFull + as), (item >> 1) & 1) && scores(0);
      // the accumulators are free once the last item's rows have been read
      if (ok) ok = wtw(bar(kOBarOEmpty), (item & 1) ^ 1);
      if (ok && st) {
        ok = full(q0 + 1);
        if (ok) {
          tc::fence_after_sync();
          if (it.role == 0 || it.role == 3) {
            const uint64_t dS = nmaj(q0 + 1, D * 128);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_bf16_w(tmem + 384, dA + kstep(kk, 16384), dS + ((kk * 2048) >> 4), id_n, kk > 0);
          } else {
            const uint64_t dS = kmaj(q0 + 1);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_bf16_w(tmem + 384, dA + kstep(kk, 16384), dS + kstep(kk, D * 128), id_k, kk > 0);
          }
          tc::commit_w(bar(kOBarEmpty + (q0 + 1) % kOSlots));
        }
      }
      for (int g = 0; ok && g < it.gi; ++g) {
        if (g + 1 < it.gi && !scores(g + 1)) {
          ok = false;
          break;
        }
        const int qc = g ? qb(g) + 1 : q0 + 1 + st, sbuf = (ss + g) & 1;
        ok = full(qc) && wtw(bar(kOBarP + sbuf), ((ss + g) >> 1) & 1);
        if (!ok) break;
        tc::fence_after_sync();
        const uint64_t dC = nmaj(qc, 16384);
        // P chunk c (16 columns) sits in the 8 columns 32 (c / 2) + 8 (c % 2)
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc::mma_bf16_ts_w(tmem + 256, tmem + sbuf * 128 + (kk >> 1) * 32 + (kk & 1) * 8, dC + ((kk * 2048) >> 4), id_n,
                            g > 0 || kk > 0);
        tc::commit_w(bar(kOBarEmpty + qc % kOSlots));
      }
      if (ok) tc::commit_w(bar(kOBarO));
      q = q0 + st + 2 * it.gi;
      ss += it.gi;
      ++item;
    }
    tc::commit_w(bar(kOBarFinal));
    mbar_wait_bounded(bar(kOBarFinal), 0, 2000000000ull);   // every MMA has completed
  } else if (warp == 10) {
    // ============================ TMA stores ==============================
    if (lane == 0) {
      int item = 0;
      for (int r = 0, i = item_at(p, 0); i < p.items; i = item_at(p, ++r)) {
        const LinItem it = lin_item(p, i);
        if (it.L <= 0) continue;
        const int as = item & 1;
        if (!wt(bar(kOBarStage + as), (item >> 1) & 1)) break;
        for (int x = 0; x < 2 * NH; ++x) {
          const int t0 = it.n * kC + (x & 1) * kSub;
          if (t0 < p.z.T)
            tma_store_4d(&p.map[it.role], sb + kOOffA + as * kOSlot + x * 8192, (x >> 1) * 64, it.h, t0, it.b);
        }
        bulk_commit_group();
        bulk_wait_group_read0();
        mbar_arrive(bar(kOBarAEmpty + as));
        ++item;
      }
      bulk_wait_group0();
    }
  } else {
    // ============================ mask and output =========================
    const int qd = warp & 3, row = 32 * qd + lane, hc = (warp - 2) >> 2;   // hc: half of the columns
    const uint32_t lanebase = static_cast<uint32_t>(32 * qd) << 16;
    int q = 0, ss = 0, item = 0;
    bool ok = true;
    for (int r = 0, i = item_at(p, 0); ok && i < p.items; i = item_at(p, ++r)) {
      const LinItem it = lin_item(p, i);
      const int t = it.n * kC + row;
      if (it.L <= 0) {                                        // rows behind the sequence
        if (t < p.z.T) {
          __nv_bfloat16 *dst = p.out[it.role] + (static_cast<size_t>(it.b) * p.z.T + t) * p.stride[it.role] + it.h * D;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) reinterpret_cast<uint4 *>(dst)[hc * (D / 16) + c] = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      const bool rev = it.role >= 2;
      const float l2 = log2_decay(p.z.log_decay[it.kv]);
      const int st = it.st ? 1 : 0;
      const MaskWeights mw(l2, rev);
      int far = 0;                                            // chunks between A and this step's B and C
      for (int g = 0; ok && g < it.gi; ++g, far = far + 1 == it.ns ? 0 : far + 1) {
        const int sbuf = (ss + g) & 1;
        const int L = far ? min(kC, it.len - (it.role < 2 ? it.n - far : it.n + far) * kC) : it.L;   // columns that count
        if (!wtw(bar(kOBarS + sbuf), ((ss + g) >> 1) & 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint32_t tS = tmem + lanebase + sbuf * 128;
        mask_scores(tS, mw, p.z.scale, row, qd, hc, rev, far, L);
        if (L < kC) {
          // rows of C behind the sequence may hold anything: 0 * NaN must not reach the product
          const int qc = q + 1 + st + 2 * g;
          if (!wtw(bar(kOBarFull + qc % kOSlots), phase(qc))) {
            ok = false;
            break;
          }
          if (row >= L && hc < NH) {
            unsigned char *cr = smem + (qc % kOSlots) * kOSlot + hc * 16384 + row * 128;
#pragma unroll
            for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4 *>(cr + 16 * e) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(bar(kOBarP + sbuf));
      }
      if (!ok || !wtw(bar(kOBarO), item & 1)) break;
      tc::fence_after_sync();
      const float fac = rev ? lexp2(l2 * static_cast<float>(max(it.L - 1 - row, 0)))
                            : p.z.scale * lexp2(l2 * static_cast<float>(row + 1));
      stage_rows<D>(tmem + lanebase, smem + kOOffA + (item & 1) * kOSlot, row, hc, st, fac, row < it.L);
      tc::fence_before_sync();
      mbar_arrive(bar(kOBarOEmpty));
      fence_proxy_async_smem();
      mbar_arrive(bar(kOBarStage + (item & 1)));
      q += st + 2 * it.gi;
      ss += it.gi;
      ++item;
    }
    tc::wait_st();                                            // scores on their way when this warp gave up
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// lin_grad: dq, dk and dv of one (batch, head, chunk) as one item, where every
// query head has a KV head of its own: the three outputs (roles 1, 2, 3 of
// lin_out, in this order) share Q, K, V, dO, S and R, so 192 KB a chunk arrive
// in place of 384.  lin_out there is bound by those copies: without all else its
// loads took 46 us of its 81 (4 x 2048 tokens of 20 heads).  This one takes 67;
// its copies alone, 378 MB, 51.
// Every tile has a slot of its own, dO two.  An output is staged over a tile
// that no product needs any more (dq over S, dk over Q, dv over dO), chosen such
// that the next item's tiles can arrive in the order in which they are needed.
// Two sets of mask and output warps take the steps in turn; the scores of the
// next step are formed before the product of this one.
// TMEM as in lin_out.  Warps: 0 TMA loads, 1 MMA, 2-17 mask and output, 18 TMA
// stores.
// ---------------------------------------------------------------------------
constexpr int kGThr = 608;
constexpr int kGV = 0, kGS = 1, kGQ = 2, kGK = 3, kGR = 4, kGDO = 5;   // slots; dO: kGDO, kGDO + 1
enum {
  kGBarFull = 0, kGBarEmpty = kGBarFull + 7, kGBarS = kGBarEmpty + 7, kGBarP = kGBarS + 2, kGBarO = kGBarP + 2,
  kGBarStage = kGBarO + 2, kGBarOEmpty = kGBarStage + 3, kGBarFinal = kGBarOEmpty + 1, kGNumBars = kGBarFinal + 1
};
static_assert(kGNumBars * 8 + 8 <= 256, "barriers of the gradient kernel");

// Item i of lin_grad; false: behind the sequence.
__device__ __noinline__ LinItem grad_item(const LinOutParams &p, int i) {
  LinItem it;
  it.kv = it.h = i % p.z.Hkv;
  i /= p.z.Hkv;
  it.n = p.z.NC - 1 - i % p.z.NC;                             // what lin_state has read last first
  it.b = p.z.B - 1 - i / p.z.NC;
  it.len = seq_len(p.z.lengths, it.b, p.z.T);
  it.L = min(kC, it.len - it.n * kC);
  return it;
}

template <int D>
__global__ void __launch_bounds__(kGThr, 1)
    lin_grad_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                    const __grid_constant__ LinOutParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int NH = D / 64;

  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOOffBar + kGNumBars * 8 + 4);
  const LinWait lw{sb + kOOffBar, abort_flag, kSiteLinGrad, p.wait};
  auto bar = [&](int i) -> uint32_t { return lw.bar(i); };
  auto wt = [&](uint32_t br, uint32_t parity) -> bool { return lw.one(br, parity); };
  auto wtw = [&](uint32_t br, uint32_t parity) -> bool { return lw.warp(br, parity); };
  // the slot of a tile in item `item`, and the phase of its barriers there
  auto slot = [](int tile, int item) -> int { return tile == kGDO ? kGDO + (item & 1) : tile; };
  auto phase = [](int tile, int item) -> uint32_t { return (tile == kGDO ? item >> 1 : item) & 1; };
  // the slot that output r = 0, 1, 2 (dq, dk, dv) is staged in
  auto out_tile = [](int r) -> int { return r == 0 ? kGS : r == 1 ? kGQ : kGDO; };
  auto has_s = [&](const LinItem &it) -> bool { return it.n > 0 || p.start[0]; };
  auto has_r = [&](const LinItem &it) -> bool { return (it.n + 1) * kC < it.len || p.start[1]; };

  if (tid == 0) {
    for (int s = 0; s < 7; ++s) {
      mbar_init(bar(kGBarFull + s), 1);
      mbar_init(bar(kGBarEmpty + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kGBarS + s), 1);
      mbar_init(bar(kGBarP + s), 256);
      mbar_init(bar(kGBarO + s), 1);
    }
    for (int s = 0; s < 3; ++s) mbar_init(bar(kGBarStage + s), 256);
    mbar_init(bar(kGBarOEmpty), 256);
    mbar_init(bar(kGBarFinal), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(sb + kOOffBar + kGNumBars * 8, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kOOffBar + kGNumBars * 8);

  if (warp != 0) wait_states();
  if (warp == 0) {
    // ============================ TMA producer ============================
    if (lane == 0) {
      // in the order in which the last item's tiles are done with: dO, V, S, Q, K, R
      auto tile_at = [](int e) -> int { return e == 0 ? kGDO : e - 1; };
      int loads = 0, item = 0;
      bool ok = true, states = false;
      for (int i = blockIdx.x; ok && i < p.items; i += gridDim.x) {
        const LinItem it = grad_item(p, i);
        if (it.L <= 0) continue;
#pragma unroll 1
        for (int e = 0; e < 6; ++e) {
          const int tile = tile_at(e), s = slot(tile, item);
          if (tile == kGS && !states) {
            wait_states();
            states = true;
          }
          const uint32_t fb = bar(kGBarFull + s), dst = sb + s * kOSlot;
          if (!wt(bar(kGBarEmpty + s), phase(tile, item) ^ 1u)) {
            ok = false;
            break;
          }
          if (tile == kGS || tile == kGR) {
            if (tile == kGS ? has_s(it) : has_r(it)) {
              mbar_arrive_expect_tx(fb, D * D * 2);
              bulk_load(dst, p.tiles[tile == kGR] + (static_cast<size_t>(it.b * p.z.Hkv + it.kv) * p.z.NC + it.n) * (D * D),
                        D * D * 2, fb);
            } else {
              mbar_arrive(fb);
            }
          } else {
            const CUtensorMap *m = tile == kGDO ? &tmDO : tile == kGV ? &tmV : tile == kGQ ? &tmQ : &tmK;
            mbar_arrive_expect_tx(fb, NH * 16384);
            for (int x = 0; x < 2 * NH; ++x)
              tma_load_4d(dst + x * 8192, m, (x >> 1) * 64, it.h, it.n * kC + (x & 1) * kSub, it.b, fb);
          }
          ++loads;
        }
        if (ok) ++item;
      }
      if (!states) wait_states();
      // the last load of every slot, before the block may end (as in lin_state);
      // an older phase of a slot would pass for one that is still to come
#pragma unroll 1
      for (int e = 0; e < 6; ++e) {
        const int tile = tile_at(e), n = loads / 6 + (e < loads % 6 ? 1 : 0);   // loads of this tile
        for (int x = max(n - (tile == kGDO ? 2 : 1), 0); x < n; ++x)
          mbar_wait_bounded(bar(kGBarFull + slot(tile, x)), phase(tile, x), 2000000000ull);
      }
    }
  } else if (warp == 1) {
    // ============================ MMA issuer ==============================
    constexpr uint32_t id_s = tc::idesc_bf16_f32(128, 128, 0, 0);   // A B^T
    constexpr uint32_t id_n = tc::idesc_bf16_f32(128, D, 0, 1);     // P C and A S: B operand N-major
    constexpr uint32_t id_k = tc::idesc_bf16_f32(128, D, 0, 0);     // A S^T: B operand K-major
    auto kmaj = [&](int tile, int item) { return tc::sdesc_sw128(sb + slot(tile, item) * kOSlot, 16, 1024); };
    auto nmaj = [&](int tile, int item, uint32_t half) {
      return tc::sdesc_sw128(sb + slot(tile, item) * kOSlot, half, 1024);
    };
    auto kstep = [](int kk, int half) -> uint32_t { return static_cast<uint32_t>((kk >> 2) * half + (kk & 3) * 32) >> 4; };
    auto full = [&](int tile, int item) -> bool { return wtw(bar(kGBarFull + slot(tile, item)), phase(tile, item)); };
    auto next = [&](int &i, LinItem &it) -> bool {            // the next item that holds tokens
      for (; i < p.items; i += gridDim.x) {
        it = grad_item(p, i);
        if (it.L > 0) return true;
      }
      return false;
    };
    // A B^T of output r into the buffer of step k, which held P two steps ago
    // (its product was issued before: the tensor core works in order)
    auto scores = [&](int r, int item, int k) -> bool {
      const int ta = r == 0 ? kGDO : r == 1 ? kGV : kGK, tb = r == 0 ? kGV : r == 1 ? kGDO : kGQ;
      if (!full(ta, item) || !full(tb, item)) return false;
      tc::fence_after_sync();
      const uint64_t dA = kmaj(ta, item), dB = kmaj(tb, item);
      const uint32_t tS = tmem + (k & 1) * 128;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) tc::mma_bf16_w(tS, dA + kstep(kk, 16384), dB + kstep(kk, 16384), id_s, kk > 0);
      tc::commit_w(bar(kGBarS + (k & 1)));
      return true;
    };
    LinItem it, nx;
    int i = blockIdx.x, item = 0, k = 0;
    bool more = next(i, it), ok = !more || (lw.start(kGBarFull + kGDO) && scores(0, 0, 0));
    while (ok && more) {
      i += gridDim.x;
      more = next(i, nx);
      for (int r = 0; ok && r < 3; ++r, ++k) {
        const int ta = r == 0 ? kGDO : r == 1 ? kGV : kGK, ts = r == 0 ? kGS : kGR;
        const int tb = r == 0 ? kGK : r == 1 ? kGQ : kGDO;
        // the accumulators are free once the last output's rows have been read
        ok = wtw(bar(kGBarOEmpty), (k & 1) ^ 1) && full(ts, item);
        if (!ok) break;
        tc::fence_after_sync();
        if (r == 0 ? has_s(it) : has_r(it)) {
          const uint64_t dA = kmaj(ta, item);
          if (r == 2) {
            const uint64_t dS = nmaj(ts, item, D * 128);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_bf16_w(tmem + 384, dA + kstep(kk, 16384), dS + ((kk * 2048) >> 4), id_n, kk > 0);
          } else {
            const uint64_t dS = kmaj(ts, item);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_bf16_w(tmem + 384, dA + kstep(kk, 16384), dS + kstep(kk, D * 128), id_k, kk > 0);
          }
        }
        // the last products that read V, K and R
        if (r == 1) tc::commit_w(bar(kGBarEmpty + kGV));
        if (r == 2) {
          tc::commit_w(bar(kGBarEmpty + kGK));
          tc::commit_w(bar(kGBarEmpty + kGR));
        }
        ok = r < 2 ? scores(r + 1, item, k + 1) : !more || scores(0, item + 1, k + 1);
        ok = ok && full(tb, item) && wtw(bar(kGBarP + (k & 1)), (k >> 1) & 1);
        if (!ok) break;
        tc::fence_after_sync();
        const uint64_t dC = nmaj(tb, item, 16384);
        // P chunk c (16 columns) sits in the 8 columns 32 (c / 2) + 8 (c % 2)
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc::mma_bf16_ts_w(tmem + 256, tmem + (k & 1) * 128 + (kk >> 1) * 32 + (kk & 1) * 8, dC + ((kk * 2048) >> 4),
                            id_n, kk > 0);
        tc::commit_w(bar(kGBarO + (k & 1)));
      }
      ++item;
      it = nx;
    }
    tc::commit_w(bar(kGBarFinal));
    mbar_wait_bounded(bar(kGBarFinal), 0, 2000000000ull);   // every MMA has completed
  } else if (warp == 18) {
    // ============================ TMA stores ==============================
    if (lane == 0) {
      int item = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < p.items; i += gridDim.x) {
        const LinItem it = grad_item(p, i);
        if (it.L <= 0) continue;
        for (int r = 0; r < 3; ++r) {
          if (!wt(bar(kGBarStage + r), item & 1)) {
            ok = false;
            break;
          }
          const int s = slot(out_tile(r), item);
          for (int x = 0; x < 2 * NH; ++x) {
            const int t0 = it.n * kC + (x & 1) * kSub;
            if (t0 < p.z.T) tma_store_4d(&p.map[1 + r], sb + s * kOSlot + x * 8192, (x >> 1) * 64, it.h, t0, it.b);
          }
          bulk_commit_group();
          bulk_wait_group_read0();
          mbar_arrive(bar(kGBarEmpty + s));
        }
        ++item;
      }
      bulk_wait_group0();
    }
  } else {
    // ============================ mask and output =========================
    const int qd = warp & 3, row = 32 * qd + lane, hc = ((warp - 2) >> 2) & 1;   // hc: half of the columns
    const int set = (warp - 2) >> 3;                          // takes the steps of one parity
    const uint32_t lanebase = static_cast<uint32_t>(32 * qd) << 16;
    int item = 0, k = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < p.items; i += gridDim.x) {
      const LinItem it = grad_item(p, i);
      if (it.L <= 0) {                                        // rows behind the sequence
        const int t = it.n * kC + row;
        for (int r = 1; r < 4 && set == 0 && t < p.z.T; ++r) {
          __nv_bfloat16 *dst = p.out[r] + (static_cast<size_t>(it.b) * p.z.T + t) * p.stride[r] + it.h * D;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) reinterpret_cast<uint4 *>(dst)[hc * (D / 16) + c] = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      const float l2 = log2_decay(p.z.log_decay[it.kv]);
      for (int r = 0; ok && r < 3; ++r, ++k) {
        if ((k & 1) != set) continue;
        const bool rev = r > 0;
        const MaskWeights mw(l2, rev);
        if (!wtw(bar(kGBarS + set), (k >> 1) & 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        mask_scores(tmem + lanebase + set * 128, mw, p.z.scale, row, qd, hc, rev, 0, it.L);
        if (it.L < kC) {
          // rows of C behind the sequence may hold anything: 0 * NaN must not reach the product
          const int ct = r == 0 ? kGK : r == 1 ? kGQ : kGDO, s = slot(ct, item);
          if (!wtw(bar(kGBarFull + s), phase(ct, item))) {
            ok = false;
            break;
          }
          if (row >= it.L && hc < NH) {
            unsigned char *cr = smem + s * kOSlot + hc * 16384 + row * 128;
#pragma unroll
            for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4 *>(cr + 16 * e) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(bar(kGBarP + set));
        if (!wtw(bar(kGBarO + set), (k >> 1) & 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const float fac = rev ? lexp2(l2 * static_cast<float>(max(it.L - 1 - row, 0)))
                              : p.z.scale * lexp2(l2 * static_cast<float>(row + 1));
        stage_rows<D>(tmem + lanebase, smem + slot(out_tile(r), item) * kOSlot, row, hc, rev ? has_r(it) : has_s(it), fac,
                      row < it.L);
        tc::fence_before_sync();
        mbar_arrive(bar(kGBarOEmpty));
        fence_proxy_async_smem();
        mbar_arrive(bar(kGBarStage + r));
      }
      ++item;
    }
    tc::wait_st();                                            // scores on their way when this warp gave up
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// lin_decode: one token per sequence.  Bound by reading and writing the fp32
// states.  A block takes 32 columns of one (batch row, KV head) state: 8
// lanes of 4 columns span a row, 32 rows go at a time, every thread holds its
// rows' pieces at once; the group's query products are summed over the rows
// by shuffles and shared memory.
// ---------------------------------------------------------------------------
constexpr int kDThr = 256;
constexpr int kDCols = 32;

struct LinDecodeParams {
  const void *q, *k, *v;
  void *o;
  float *state;
  const float *log_decay;
  const int *slots;
  int Hq, Hkv, G, D, nstates;
  float scale;
};

template <typename T>
__device__ __forceinline__ float lin_ld(const void *p, size_t i) {
  return static_cast<float>(reinterpret_cast<const T *>(p)[i]);
}

// Blocks an SM: what is under way is what counts (64 rows of 20 heads of 128:
// 25.0 us with six, 25.7 with five).
constexpr int decode_blocks(int D, int G) { return D == 64 ? (G <= 4 ? 8 : 6) : G <= 2 ? 6 : G <= 4 ? 5 : 4; }

template <typename T, int D, int G>
__global__ void __launch_bounds__(kDThr, decode_blocks(D, G)) lin_decode_kernel(const LinDecodeParams p) {
  __shared__ float sk[D], sq[G][D];
  __shared__ float red[kDThr / 32][G][kDCols];
  constexpr int NSL = D / kDCols, R = D / 32;
  const int slice = blockIdx.x % NSL, bh = blockIdx.x / NSL;
  const int b = bh / p.Hkv, kv = bh % p.Hkv;
  const int tid = threadIdx.x, c4 = tid & 7, r0 = tid >> 3;
  const int slot = p.slots ? p.slots[b] : b;
  const size_t ob = (static_cast<size_t>(b) * p.Hq + kv * p.G) * D + slice * kDCols;
  if (slot < 0 || slot >= p.nstates) {                        // an empty row of the batch
    for (int i = tid; i < p.G * kDCols; i += kDThr)
      reinterpret_cast<T *>(p.o)[ob + static_cast<size_t>(i / kDCols) * D + i % kDCols] = static_cast<T>(0.f);
    return;
  }
  float4 *st = reinterpret_cast<float4 *>(p.state + (static_cast<size_t>(slot) * p.Hkv + kv) * (D * D) + slice * kDCols);
  float4 s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) s[r] = st[(r0 + 32 * r) * (D / 4) + c4];
  // a and what one float misses of it; where nothing is missing nothing is added
  // (an infinity stays one)
  const float ld = p.log_decay[kv];
  const float2 dec = step_decay(ld, 1, [&] { return expf(ld); });
  const float a = dec.x, low = dec.y;
  if (tid < D) sk[tid] = lin_ld<T>(p.k, static_cast<size_t>(bh) * D + tid);
  for (int i = tid; i < G * D; i += kDThr)
    sq[i / D][i % D] = i / D < p.G ? lin_ld<T>(p.q, (static_cast<size_t>(b) * p.Hq + kv * p.G) * D + i) : 0.f;
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = lin_ld<T>(p.v, static_cast<size_t>(bh) * D + slice * kDCols + 4 * c4 + e);
  __syncthreads();
  float4 acc[G];
#pragma unroll
  for (int g = 0; g < G; ++g) acc[g] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int d = r0 + 32 * r;
    const float k = sk[d];
    float4 t = make_float4(k * v[0], k * v[1], k * v[2], k * v[3]);
    if (low > 0.f)
      t = make_float4(fmaf(low, s[r].x, t.x), fmaf(low, s[r].y, t.y), fmaf(low, s[r].z, t.z), fmaf(low, s[r].w, t.w));
    s[r].x = fmaf(a, s[r].x, t.x);
    s[r].y = fmaf(a, s[r].y, t.y);
    s[r].z = fmaf(a, s[r].z, t.z);
    s[r].w = fmaf(a, s[r].w, t.w);
    st[d * (D / 4) + c4] = s[r];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float q = sq[g][d];
      acc[g].x = fmaf(q, s[r].x, acc[g].x);
      acc[g].y = fmaf(q, s[r].y, acc[g].y);
      acc[g].z = fmaf(q, s[r].z, acc[g].z);
      acc[g].w = fmaf(q, s[r].w, acc[g].w);
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      acc[g].x += __shfl_xor_sync(0xffffffffu, acc[g].x, o);
      acc[g].y += __shfl_xor_sync(0xffffffffu, acc[g].y, o);
      acc[g].z += __shfl_xor_sync(0xffffffffu, acc[g].z, o);
      acc[g].w += __shfl_xor_sync(0xffffffffu, acc[g].w, o);
    }
    if ((tid & 31) < 8) *reinterpret_cast<float4 *>(&red[tid >> 5][g][4 * c4]) = acc[g];
  }
  __syncthreads();
  for (int i = tid; i < p.G * kDCols; i += kDThr) {
    const int g = i / kDCols, c = i % kDCols;
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kDThr / 32; ++w) t += red[w][g][c];
    reinterpret_cast<T *>(p.o)[ob + static_cast<size_t>(g) * D + c] = static_cast<T>(p.scale * t);
  }
}

template <typename T, int D>
cudaError_t decode_groups(const LinDecodeParams &p, unsigned blocks, cudaStream_t st) {
  if (p.G <= 1)
    lin_decode_kernel<T, D, 1><<<blocks, kDThr, 0, st>>>(p);
  else if (p.G <= 2)
    lin_decode_kernel<T, D, 2><<<blocks, kDThr, 0, st>>>(p);
  else if (p.G <= 4)
    lin_decode_kernel<T, D, 4><<<blocks, kDThr, 0, st>>>(p);
  else
    lin_decode_kernel<T, D, 8><<<blocks, kDThr, 0, st>>>(p);
  return cudaGetLastError();
}

// Rows of D elements at `stride` elements from token to token, in boxes of 64
// tokens by 64 columns (128-byte swizzle, as the products read them) or 32
// (plain rows).  Encoding a map takes the host about a microsecond, and a
// backward call has nine: each thread keeps the layouts it met last and points
// a copy at the buffer.
bool lin_map(CUtensorMap *mp, const void *base, int D, int H, int T, int B, long long stride, const char **why,
             int cols = 64) {
  struct Entry {
    int D, H, T, B, cols;
    long long stride;
    CUtensorMap map;
  };
  constexpr int kKept = 16;
  thread_local Entry kept[kKept];
  thread_local int count = 0, oldest = 0;
  for (int i = 0; i < count; ++i) {
    const Entry &e = kept[i];
    if (e.D == D && e.H == H && e.T == T && e.B == B && e.cols == cols && e.stride == stride) {
      *mp = e.map;
      if (move_tiled(mp, base)) return true;
      break;
    }
  }
  const uint64_t ts = static_cast<uint64_t>(stride) * 2;
  const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(H), static_cast<uint64_t>(T),
                            static_cast<uint64_t>(B)};
  const uint64_t strides[3] = {static_cast<uint64_t>(D) * 2, ts, ts * T};
  const uint32_t box[4] = {static_cast<uint32_t>(cols), 1, kSub, 1};
  if (!encode_tiled(mp, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box,
                    cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, why))
    return false;
  const int at = count < kKept ? count++ : oldest++ % kKept;
  kept[at] = Entry{D, H, T, B, cols, stride, *mp};
  return true;
}

template <int D, int NS>
cudaError_t launch_state(const CUtensorMap (&tm)[6], const LinStateParams &p, cudaStream_t st) {
  const auto kern = lin_state_kernel<D, NS>;
  constexpr int smem = StateShape<NS>::kSmem;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(p.nroles) * p.z.B * p.z.Hkv * (D / kCW);
  kern<<<grid, kSThr, smem, st>>>(tm[1], tm[4], tm[0], tm[5], p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_lin(const CUtensorMap (&tm)[6], const LinStateParams &sp, const LinOutParams &op, bool exact,
                       int sms, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (sp.nroles) {
    e = exact ? launch_state<D, 3>(tm, sp, st) : launch_state<D, 2>(tm, sp, st);
    if (e != cudaSuccess) return e;
  }
  const bool grad = op.backward && op.z.G == 1 && !op.direct;
  const auto kern = grad ? lin_grad_kernel<D> : lin_out_kernel<D>;
  e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), kOSmem);
  if (e != cudaSuccess) return e;
  LinOutParams o = op;
  if (grad) o.items /= 3;               // the three outputs of a chunk together
  const int grid = o.items < sms ? o.items : sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(grad ? kGThr : kOThr);
  cfg.dynamicSmemBytes = kOSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = sp.nroles ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, tm[0], tm[1], tm[2], tm[3], o);
}

size_t tiles_bytes(int B, int T, int Hkv, int D) {
  const size_t nc = (static_cast<size_t>(T) + kC - 1) / kC;
  return static_cast<size_t>(B) * Hkv * nc * D * D * 2;
}

}  // namespace

size_t lin_attn_workspace_bytes(int B, int T, int Hkv, int D, int backward) {
  return tiles_bytes(B, T, Hkv, D) * (backward ? 2 : 1);
}

cudaError_t launch_lin_attn(const LinAttnArgs &a, const WaitCtl &w, cudaStream_t st, const char **why) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const bool bwd = a.dout != nullptr;
  LinOutParams op = {};
  op.z.B = a.B, op.z.T = a.T, op.z.Hq = a.Hq, op.z.Hkv = a.Hkv, op.z.G = a.Hq / a.Hkv;
  op.z.NC = (a.T + kC - 1) / kC;
  op.z.scale = a.scale;
  op.z.log_decay = a.log_decay;
  op.z.lengths = a.lengths;
  op.backward = bwd;
  const long long items = static_cast<long long>(a.B) * op.z.NC * (bwd ? a.Hq + 2LL * a.Hkv : a.Hq);
  if (items > 0x7ffffff0LL - 2 * sms || 8LL * a.B * a.Hkv > 0x7fffffffLL) {
    *why = "grid too large";
    return cudaErrorNotSupported;
  }
  op.items = static_cast<int>(items);
  LinStateParams sp = {};
  sp.z = op.z;
  sp.start[0] = a.initial_state;
  sp.start[1] = a.dfinal_state;
  sp.end[0] = a.final_state;
  sp.end[1] = a.dinitial_state;
  // which recurrences anything reads: the tiles of more than one chunk or of
  // a given start, and the states that leave
  op.direct = op.z.NC <= direct_chunks(bwd, op.z.G) && !a.initial_state && !a.final_state && !a.dfinal_state &&
              !a.dinitial_state;
  const bool far = op.z.NC > 1 && !op.direct;
  const bool tiles0 = far || a.initial_state, tiles1 = bwd && (far || a.dfinal_state);
  const bool f = tiles0 || a.final_state, r = tiles1 || a.dinitial_state;
  sp.first_role = f ? 0 : 1;
  sp.nroles = (f ? 1 : 0) + (r ? 1 : 0);
  sp.tiles[0] = tiles0 ? static_cast<__nv_bfloat16 *>(a.ws) : nullptr;
  sp.tiles[1] = tiles1 ? reinterpret_cast<__nv_bfloat16 *>(static_cast<unsigned char *>(a.ws) +
                                                           tiles_bytes(a.B, a.T, a.Hkv, a.D))
                       : nullptr;
  sp.wait = w;
  for (int i = 0; i < 2; ++i) {
    op.tiles[i] = sp.tiles[i];
    op.start[i] = sp.start[i] != nullptr;
  }
  void *const out[4] = {a.o, a.dq, a.dk, a.dv};
  const long long os[4] = {a.o_stride, a.dq_stride, a.dk_stride, a.dv_stride};
  for (int i = 0; i < 4; ++i) {
    op.out[i] = static_cast<__nv_bfloat16 *>(out[i]);
    op.stride[i] = os[i];
  }
  op.wait = w;
  CUtensorMap tm[6];                    // q, k, v, dout; v and dout in narrow boxes
  if (!lin_map(&tm[0], a.q, a.D, a.Hq, a.T, a.B, a.q_stride, why) ||
      !lin_map(&tm[1], a.k, a.D, a.Hkv, a.T, a.B, a.k_stride, why) ||
      !lin_map(&tm[2], a.v, a.D, a.Hkv, a.T, a.B, a.v_stride, why) ||
      (bwd && !lin_map(&tm[3], a.dout, a.D, a.Hq, a.T, a.B, static_cast<long long>(a.Hq) * a.D, why)))
    return cudaErrorInvalidValue;
  if ((f && !lin_map(&tm[4], a.v, a.D, a.Hkv, a.T, a.B, a.v_stride, why, kCW)) ||
      (r && !lin_map(&tm[5], a.dout, a.D, a.Hq, a.T, a.B, static_cast<long long>(a.Hq) * a.D, why, kCW)))
    return cudaErrorInvalidValue;
  if (!bwd) tm[3] = tm[0];              // these are not read
  if (!f) tm[4] = tm[0];
  if (!r) tm[5] = tm[0];
  for (int i = 0; i < 4; ++i)
    if (out[i] && !lin_map(&op.map[i], out[i], a.D, i < 2 ? a.Hq : a.Hkv, a.T, a.B, os[i], why))
      return cudaErrorInvalidValue;
  const bool exact = a.final_state || a.dinitial_state;   // a state leaves in fp32
  return a.D == 128 ? launch_lin<128>(tm, sp, op, exact, sms, st) : launch_lin<64>(tm, sp, op, exact, sms, st);
}

cudaError_t launch_lin_attn_decode(const void *q, const void *k, const void *v, float *state, const float *log_decay,
                                   const int *slots, void *o, int bf16, int B, int Hq, int Hkv, int D, int nstates,
                                   float scale, cudaStream_t st) {
  LinDecodeParams p;
  p.q = q, p.k = k, p.v = v, p.o = o;
  p.state = state;
  p.log_decay = log_decay;
  p.slots = slots;
  p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv, p.D = D, p.nstates = nstates;
  p.scale = scale;
  const long long blocks = static_cast<long long>(B) * Hkv * (D / kDCols);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned n = static_cast<unsigned>(blocks);
  if (bf16) return D == 128 ? decode_groups<__nv_bfloat16, 128>(p, n, st) : decode_groups<__nv_bfloat16, 64>(p, n, st);
  return D == 128 ? decode_groups<float, 128>(p, n, st) : decode_groups<float, 64>(p, n, st);
}

}  // namespace abw
