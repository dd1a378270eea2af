// RMS norm of every query and key head with the position rotation in the same
// pass, forward and backward.  Per head row x[D]:
//   rms = sqrt(mean x^2 + eps),  n = x gamma / rms,  y = R(theta) n
// R turns the pairs of the first rotary_dim components, theta_i = pos base^(-2i
// / rotary_dim), pos the token's position on the axis that pair i belongs to.
// Backward, with dn = R(-theta) dy and c = sum dn gamma x:
//   dx = (dn gamma - x c / (D rms^2)) / rms,   dgamma = sum over rows dn x / rms
//
// Bound by memory: x is read once and y written once (backward: x and dy read,
// dx written); the norm's sum is taken in registers.
//
// Angles without double precision on the device: the host forms the turns per
// position, base^(-2i / rotary_dim) / (2 pi) mod 1, in double and hands them on as
// a 64-bit binary fraction; an integer product with the position, modulo 2^64, is
// the angle modulo one turn for every 32-bit position, negative ones included.
// The product adds no more than 2^-31 turns; the table's own error (below 2^-54
// turns where base >= 1: pow, the division and 2 pi, each to a double's rounding of
// at most 0.16) grows with the position, to 2^-23 turns at 2^31.
#include <math.h>

#include "abw_host.h"

namespace abw {
namespace {

constexpr int kQThr = 256;
constexpr int kQMaxPairs = 256;       // D <= 512

struct QkParams {
  const void *x[2];                   // queries, keys
  const void *dy[2];
  void *out[2];                       // y, or dx
  const float *gamma[2];              // null: no norm
  float *part;                        // backward: [gridDim.x][D] partial dgamma
  float *dgamma[2];                   // null: not wanted
  long long xs[2], os[2];             // elements from token to token
  int H[2];
  int D, rot;                         // components per head, pairs that turn
  int T, pos0;
  int slots[2];                       // lane groups that share a token's heads
  int first_k;                        // first block that works on keys
  long long ntok;
  float eps, inv_n;
  const int *pos;                     // [axes][ntok] or null: pos0 + t
  int sec_end[3];                     // first pair behind each axis' pairs, but for the last axis
};

// A launch's parameters are written out with it: heads of up to 128 components
// carry a table of 64 turns, longer ones of 256 (0.5 us less per launch).
template <int NP>
struct QkTable : QkParams {
  unsigned long long freq[NP];
};

// Arithmetic on V values at a time: two float2 (packed fp32 instructions) for
// V = 4, one float for V = 1.
template <int V>
struct Num;
template <>
struct Num<4> {
  using F = float2;
  static constexpr int kC = 2;
};
template <>
struct Num<1> {
  using F = float;
  static constexpr int kC = 1;
};
__device__ __forceinline__ float2 f_mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 f_fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float f_sum(float2 a) { return a.x + a.y; }
__device__ __forceinline__ float f_mul(float a, float b) { return a * b; }
__device__ __forceinline__ float f_fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float f_sum(float a) { return a; }
template <typename F>
__device__ __forceinline__ F f_all(float a);
template <>
__device__ __forceinline__ float2 f_all<float2>(float a) { return make_float2(a, a); }
template <>
__device__ __forceinline__ float f_all<float>(float a) { return a; }

__device__ __forceinline__ uint32_t q_pack(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

// Where the V pairs of the pair slots s .. s + V - 1 of a row are: two runs of V
// elements, at x and y.  Interleaved pairs are neighbours; split pairs are rot
// apart.  Components behind the rotated ones are paired with their neighbours
// (their angle is 0).
template <int V, bool INTER>
struct Place {
  int x, y;
  __device__ __forceinline__ Place(int s, int rot) {
    const bool near = INTER || s >= rot;
    x = near ? 2 * s : s;
    y = near ? 2 * s + V : s + rot;
  }
};

// V pairs of a row as they are in memory, so that loads of the next rows can
// be under way while these are at work.  get / set: members a, b of the pairs.
template <typename T, int V, bool INTER>
struct Pairs;
template <bool INTER>
struct Pairs<__nv_bfloat16, 4, INTER> {
  uint2 x, y;
  __device__ __forceinline__ void clear() { x = y = make_uint2(0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *row, const Place<4, INTER> &at) {
    if constexpr (INTER) {
      const uint4 u = __ldg(reinterpret_cast<const uint4 *>(row + at.x));
      x = make_uint2(u.x, u.y), y = make_uint2(u.z, u.w);
    } else {
      x = __ldg(reinterpret_cast<const uint2 *>(row + at.x));
      y = __ldg(reinterpret_cast<const uint2 *>(row + at.y));
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *row, const Place<4, INTER> &at) const {
    if constexpr (INTER) {
      *reinterpret_cast<uint4 *>(row + at.x) = make_uint4(x.x, x.y, y.x, y.y);
    } else {
      *reinterpret_cast<uint2 *>(row + at.x) = x;
      *reinterpret_cast<uint2 *>(row + at.y) = y;
    }
  }
  __device__ __forceinline__ void get(float2 (&a)[2], float2 (&b)[2]) const {
    if constexpr (INTER) {
      a[0] = make_float2(bf16_lo(x.x), bf16_lo(x.y)), a[1] = make_float2(bf16_lo(y.x), bf16_lo(y.y));
      b[0] = make_float2(bf16_hi(x.x), bf16_hi(x.y)), b[1] = make_float2(bf16_hi(y.x), bf16_hi(y.y));
    } else {
      a[0] = make_float2(bf16_lo(x.x), bf16_hi(x.x)), a[1] = make_float2(bf16_lo(x.y), bf16_hi(x.y));
      b[0] = make_float2(bf16_lo(y.x), bf16_hi(y.x)), b[1] = make_float2(bf16_lo(y.y), bf16_hi(y.y));
    }
  }
  __device__ __forceinline__ void set(const float2 (&a)[2], const float2 (&b)[2]) {
    if constexpr (INTER) {
      x = make_uint2(q_pack(a[0].x, b[0].x), q_pack(a[0].y, b[0].y));
      y = make_uint2(q_pack(a[1].x, b[1].x), q_pack(a[1].y, b[1].y));
    } else {
      x = make_uint2(q_pack(a[0].x, a[0].y), q_pack(a[1].x, a[1].y));
      y = make_uint2(q_pack(b[0].x, b[0].y), q_pack(b[1].x, b[1].y));
    }
  }
};
template <bool INTER>
struct Pairs<float, 4, INTER> {
  float4 x, y;
  __device__ __forceinline__ void clear() { x = y = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float *row, const Place<4, INTER> &at) {
    x = __ldg(reinterpret_cast<const float4 *>(row + at.x));
    y = __ldg(reinterpret_cast<const float4 *>(row + at.y));
  }
  __device__ __forceinline__ void store(float *row, const Place<4, INTER> &at) const {
    *reinterpret_cast<float4 *>(row + at.x) = x;
    *reinterpret_cast<float4 *>(row + at.y) = y;
  }
  __device__ __forceinline__ void get(float2 (&a)[2], float2 (&b)[2]) const {
    if constexpr (INTER) {
      a[0] = make_float2(x.x, x.z), a[1] = make_float2(y.x, y.z);
      b[0] = make_float2(x.y, x.w), b[1] = make_float2(y.y, y.w);
    } else {
      a[0] = make_float2(x.x, x.y), a[1] = make_float2(x.z, x.w);
      b[0] = make_float2(y.x, y.y), b[1] = make_float2(y.z, y.w);
    }
  }
  __device__ __forceinline__ void set(const float2 (&a)[2], const float2 (&b)[2]) {
    if constexpr (INTER) {
      x = make_float4(a[0].x, b[0].x, a[0].y, b[0].y);
      y = make_float4(a[1].x, b[1].x, a[1].y, b[1].y);
    } else {
      x = make_float4(a[0].x, a[0].y, a[1].x, a[1].y);
      y = make_float4(b[0].x, b[0].y, b[1].x, b[1].y);
    }
  }
};
template <typename T, bool INTER>
struct Pairs<T, 1, INTER> {
  T x, y;
  __device__ __forceinline__ void clear() { x = y = static_cast<T>(0.f); }
  __device__ __forceinline__ void load(const T *row, const Place<1, INTER> &at) { x = row[at.x], y = row[at.y]; }
  __device__ __forceinline__ void store(T *row, const Place<1, INTER> &at) const { row[at.x] = x, row[at.y] = y; }
  __device__ __forceinline__ void get(float (&a)[1], float (&b)[1]) const {
    a[0] = static_cast<float>(x), b[0] = static_cast<float>(y);
  }
  __device__ __forceinline__ void set(const float (&a)[1], const float (&b)[1]) {
    x = static_cast<T>(a[0]), y = static_cast<T>(b[0]);
  }
};

// Rows on their way: each lane copies its own pieces of the next rows into slots
// of its own in shared memory and takes them from there, so that what is under
// way costs no registers, and no thread waits for another.  (What bounds these
// kernels otherwise is bytes under way: one row a lane in registers gave 4.5
// TB/s.)  A piece that is not there is copied as zeros.
template <int BYTES>
__device__ __forceinline__ void copy_piece(uint32_t dst, const void *src, bool live) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(live ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

template <typename T>
constexpr int kPieces = 2 * sizeof(T) * 4;                    // bytes of a lane's four pairs
// dst: this thread's slot; a float row's second piece is kQThr slots on.
template <bool INTER>
__device__ __forceinline__ void copy_pairs(uint32_t dst, const __nv_bfloat16 *row, const Place<4, INTER> &at, bool live) {
  if constexpr (INTER) {
    copy_piece<16>(dst, row + at.x, live);
  } else {
    copy_piece<8>(dst, row + at.x, live);
    copy_piece<8>(dst + 8, row + at.y, live);
  }
}
template <bool INTER>
__device__ __forceinline__ void copy_pairs(uint32_t dst, const float *row, const Place<4, INTER> &at, bool live) {
  copy_piece<16>(dst, row + at.x, live);
  copy_piece<16>(dst + 16 * kQThr, row + at.y, live);
}
template <bool INTER>
__device__ __forceinline__ void take_pairs(Pairs<__nv_bfloat16, 4, INTER> &p, const unsigned char *slot) {
  const uint4 u = *reinterpret_cast<const uint4 *>(slot);
  p.x = make_uint2(u.x, u.y), p.y = make_uint2(u.z, u.w);
}
template <bool INTER>
__device__ __forceinline__ void take_pairs(Pairs<float, 4, INTER> &p, const unsigned char *slot) {
  p.x = *reinterpret_cast<const float4 *>(slot);
  p.y = *reinterpret_cast<const float4 *>(slot + 16 * kQThr);
}
// Stages of such a ring.  4 x 2048 tokens, 20 + 20 heads of 128 bf16, us: forward
// with rows in registers 32.6, with rings of 2, 3, 4 stages 33.1, 28.4, 29.3;
// backward 56.5 with registers and 3 blocks an SM, 50.7 with 3 stages and 3
// blocks, 51.1, 48.2, 48.2 with 3, 4, 6 stages and 2 blocks.
constexpr int kFwdStages = 3, kBwdStages = 4;
// Rows that a group of lanes has to have for the ring to pay: with five it costs
// a microsecond (2050 tokens, 20 + 5 heads of 80 fp32: 8.8 us, with it 10.0).
constexpr int kRingRows = 8;

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 1 / sqrt(m): the approximation (2 ulp) and one Newton step.  Finite for m = 0:
// where eps is 0, a group of lanes without a row (zeros) would otherwise carry
// 0 * NaN into dgamma.
__device__ __forceinline__ float inv_root(float m) {
  const float r = fminf(rsqrtf(m), 8.5e37f);                  // (1.5 of it still fits)
  return r * fmaf(-0.5f * m * r, r, 1.5f);
}

template <int V, int L>
constexpr int table_size() { return V == 4 && L <= 16 ? 64 : kQMaxPairs; }

// sin and cos of t 2^-32 turns: the nearest quarter turn, and the Taylor series
// for what is left, at most pi / 4 (cut off at 2e-9 and 2e-10), in some 20
// instructions.  The angle is an integer until its one rounding to float.
__device__ __forceinline__ void turn_sincos(unsigned t, float &sn, float &cs) {
  const unsigned q = (t + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int>(t - (q << 30))) * 1.4629180792671596e-9f;   // 2 pi 2^-32
  const float y = x * x;
  const float a = fmaf(fmaf(fmaf(fmaf(1.f / 362880, y, -1.f / 5040), y, 1.f / 120), y, -1.f / 6), y * x, x);
  const float b =
      fmaf(fmaf(fmaf(fmaf(fmaf(-1.f / 3628800, y, 1.f / 40320), y, -1.f / 720), y, 1.f / 24), y, -0.5f), y, 1.f);
  const float s = q & 1 ? b : a, c = q & 1 ? a : b;
  sn = __uint_as_float(__float_as_uint(s) ^ ((q & 2) << 30));
  cs = __uint_as_float(__float_as_uint(c) ^ (((q + 1) & 2) << 30));
}

// The launch's turns in shared memory: lanes read them by an index of their
// own, which the constant bank serves one at a time.
template <int NP>
__device__ __forceinline__ void load_turns(const QkTable<NP> &p, unsigned long long *turns) {
  for (int i = threadIdx.x; i < p.rot; i += kQThr) turns[i] = p.freq[i];
  __syncthreads();
}

// cos and sin of token tok's angles for this lane's pair slots; 1 and 0 behind
// the rotated pairs.
template <int V, int N, int L, typename F = typename Num<V>::F, int C = Num<V>::kC>
__device__ __forceinline__ void lane_angles(const QkParams &p, const unsigned long long *turns, long long tok, int lane,
                                            F (&c)[N][C], F (&z)[N][C]) {
  long long step = 0;
  if (!p.pos)
    step = p.pos0 + (p.ntok <= 0x7fffffffLL
                         ? static_cast<long long>(static_cast<unsigned>(tok) % static_cast<unsigned>(p.T))
                         : tok % p.T);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float cv[V], zv[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int s = (lane + L * k) * V + e;
      cv[e] = 1.f, zv[e] = 0.f;
      if (s < p.rot) {
        const int axis = (s >= p.sec_end[0]) + (s >= p.sec_end[1]) + (s >= p.sec_end[2]);
        const long long pos = p.pos ? p.pos[axis * p.ntok + tok] : step;
        // the upper half of the product, modulo one turn
        const unsigned lo = static_cast<unsigned>(turns[s]), hi = static_cast<unsigned>(turns[s] >> 32);
        const unsigned plo = static_cast<unsigned>(pos);
        const unsigned phi = static_cast<unsigned>(static_cast<unsigned long long>(pos) >> 32);
        turn_sincos(__umulhi(plo, lo) + plo * hi + phi * lo, zv[e], cv[e]);
      }
    }
    if constexpr (V == 4) {
      c[k][0] = make_float2(cv[0], cv[1]), c[k][1] = make_float2(cv[2], cv[3]);
      z[k][0] = make_float2(zv[0], zv[1]), z[k][1] = make_float2(zv[2], zv[3]);
    } else {
      c[k][0] = cv[0], z[k][0] = zv[0];
    }
  }
}

// gamma of this lane's components, 1 where there is no norm.
template <int V, int N, int L, bool INTER, typename F = typename Num<V>::F, int C = Num<V>::kC>
__device__ __forceinline__ void lane_gamma(const float *gamma, int lane, int rot, int h2, F (&ga)[N][C],
                                           F (&gb)[N][C]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int s = (lane + L * k) * V;
#pragma unroll
    for (int e = 0; e < C; ++e) ga[k][e] = gb[k][e] = f_all<F>(1.f);
    if (gamma && s < h2) {
      Pairs<float, V, INTER> g;
      g.load(gamma, Place<V, INTER>(s, rot));
      g.get(ga[k], gb[k]);
    }
  }
}

// What a block works on: queries or keys (blocks from p.first_k on).
struct Side {
  int w, block, nblocks, H, slots;
  long long xs, os;
  const float *gamma;
  __device__ __forceinline__ explicit Side(const QkParams &p) {
    w = static_cast<int>(blockIdx.x) >= p.first_k;
    block = static_cast<int>(blockIdx.x) - (w ? p.first_k : 0);
    nblocks = w ? static_cast<int>(gridDim.x) - p.first_k : p.first_k;
    H = w ? p.H[1] : p.H[0];
    slots = w ? p.slots[1] : p.slots[0];
    xs = w ? p.xs[1] : p.xs[0];
    os = w ? p.os[1] : p.os[0];
    gamma = w ? p.gamma[1] : p.gamma[0];
  }
};

// Forward.  A row belongs to L lanes, V pair slots each (N times); a group of
// L lanes takes every slots-th head of one token, so that the token's angles
// stay in its registers, multiplied by gamma once for all its heads.  U rows at
// a time; the next ones are loaded while these are at work.
// 4 x 2048 tokens, 40 heads of 128 bf16 (167 MB): 28 us, 5.9 TB/s; it is bound by
// instruction issue nearly as much as by memory, so what counts is instructions per
// row (with rows dealt out one by one 196 a lane, 38 us).
template <typename XT, bool INTER, int V, int N, int L, int U, bool RING>
__global__ void __launch_bounds__(kQThr, V == 4 && N == 1 ? 3 : 1)
    qk_fwd_kernel(const __grid_constant__ QkTable<table_size<V, L>()> p) {
  __shared__ unsigned long long turns[table_size<V, L>()];
  using F = typename Num<V>::F;
  constexpr int kGroups = kQThr / L, C = Num<V>::kC;
  const Side sd(p);
  const int h2 = p.D >> 1, slots = sd.slots;
  const int lane = threadIdx.x % L, grp = threadIdx.x / L, slot = grp % slots;
  const long long tok = static_cast<long long>(sd.block) * (kGroups / slots) + grp / slots;
  const bool norm = sd.gamma != nullptr;
  const int H = tok < p.ntok ? sd.H : 0;                      // heads of this group's token
  const XT *x0 = static_cast<const XT *>(sd.w ? p.x[1] : p.x[0]), *x = x0 + tok * sd.xs;
  XT *o = static_cast<XT *>(sd.w ? p.out[1] : p.out[0]) + tok * sd.os;
  const int hop = slots * p.D;
    extern __shared__ __align__(16) unsigned char ring[];
  Pairs<XT, V, INTER> raw[U][N];
  auto fetch = [&](int h, int off, int stage) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int s = (lane + L * k) * V;
        const bool live = h + u * slots < H && s < h2;
        const Place<V, INTER> at(s, p.rot);
        if constexpr (RING)
          copy_pairs(smem_u32(ring) + (stage * U * N + u * N + k) * (kPieces<XT> * kQThr) + threadIdx.x * 16,
                     live ? x + (off + u * hop) : x0, at, live);
        else if (live)
          raw[u][k].load(x + (off + u * hop), at);
      }
    if constexpr (RING) copies_commit();
  };
  int fh = slot, foff = slot * p.D;
  if constexpr (RING) {
#pragma unroll
    for (int d = 0; d < kFwdStages - 1; ++d, fh += U * slots, foff += U * hop) fetch(fh, foff, d);
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k) raw[u][k].clear();          // what is not loaded adds nothing to a row's sum
    fetch(fh, foff, 0);
  }
  load_turns(p, turns);
  // y_a = (a gamma_a cos - b gamma_b sin) / rms, y_b = (a gamma_a sin + b gamma_b cos) / rms
  F ac[N][C], bs[N][C], as[N][C], bc[N][C];
  {
    F c[N][C], z[N][C];
    lane_gamma<V, N, L, INTER>(sd.gamma, lane, p.rot, h2, ac, bc);
    if (H) lane_angles<V, N, L>(p, turns, tok, lane, c, z);
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int e = 0; e < C; ++e) {
        as[k][e] = f_mul(ac[k][e], z[k][e]);
        bs[k][e] = f_mul(f_mul(bc[k][e], f_all<F>(-1.f)), z[k][e]);
        ac[k][e] = f_mul(ac[k][e], c[k][e]);
        bc[k][e] = f_mul(bc[k][e], c[k][e]);
      }
  }
  // every lane of a warp makes the same number of steps: the row sums exchange
  // values across it
  const int steps = (sd.H + slots - 1) / slots;
  int h = slot, off = slot * p.D, stage = 0;
  for (int i = 0; i < steps; i += U, h += U * slots, off += U * hop) {
    F a[U][N][C], b[U][N][C];
    if constexpr (RING) {
      copies_wait<kFwdStages - 2>();
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < N; ++k)
          take_pairs(raw[u][k], ring + (stage * U * N + u * N + k) * (kPieces<XT> * kQThr) + threadIdx.x * 16);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k) raw[u][k].get(a[u][k], b[u][k]);
    if constexpr (RING) {
      // into the stage that the last step took its rows from
      fetch(fh, foff, stage == 0 ? kFwdStages - 1 : stage - 1);
      fh += U * slots, foff += U * hop;
      if (++stage == kFwdStages) stage = 0;
    } else {
      fetch(h + U * slots, off + U * hop, 0);
    }
    float inv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      F ss = f_all<F>(0.f);
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int e = 0; e < C; ++e) ss = f_fma(a[u][k][e], a[u][k][e], f_fma(b[u][k][e], b[u][k][e], ss));
      inv[u] = f_sum(ss);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) inv[u] = norm ? inv_root(fmaf(lanes_sum<L>(inv[u]), p.inv_n, p.eps)) : 1.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const F v = f_all<F>(inv[u]);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int s = (lane + L * k) * V;
        if (h + u * slots < H && s < h2) {
          F ya[C], yb[C];
#pragma unroll
          for (int e = 0; e < C; ++e) {
            ya[e] = f_mul(f_fma(b[u][k][e], bs[k][e], f_mul(a[u][k][e], ac[k][e])), v);
            yb[e] = f_mul(f_fma(b[u][k][e], bc[k][e], f_mul(a[u][k][e], as[k][e])), v);
          }
          Pairs<XT, V, INTER> out;
          out.set(ya, yb);
          out.store(o + (off + u * hop), Place<V, INTER>(s, p.rot));
        }
      }
    }
  }
  if constexpr (RING) copies_wait<0>();
}

// Backward, laid out as the forward; the groups of a block go on to further
// tokens and keep their lanes' dgamma in registers.  Registers are held to what
// lets bwd_blocks blocks be resident.  4 x 2048 tokens, 20 + 20 heads of 128
// bf16, dy bf16 (252 MB): 48 us with dgamma, 5.2 TB/s.
constexpr int bwd_blocks(bool ring) { return ring ? 2 : 3; }

template <typename XT, typename DT, bool INTER, int V, int N, int L, bool RING>
__global__ void __launch_bounds__(kQThr, V == 4 && N == 1 ? bwd_blocks(RING) : 1)
    qk_bwd_kernel(const __grid_constant__ QkTable<table_size<V, L>()> p) {
  extern __shared__ __align__(16) unsigned char ring[];
  float *sums = reinterpret_cast<float *>(ring);              // [kGroups][D], at the end
  __shared__ unsigned long long turns[table_size<V, L>()];
  using F = typename Num<V>::F;
  constexpr int kGroups = kQThr / L, C = Num<V>::kC;
  const Side sd(p);
  const int h2 = p.D >> 1, slots = sd.slots, per = kGroups / slots, hop = slots * p.D;
  const int lane = threadIdx.x % L, grp = threadIdx.x / L, slot = grp % slots;
  const int steps = (sd.H + slots - 1) / slots;
  const bool norm = sd.gamma != nullptr;
  // qk_dgamma may start; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  load_turns(p, turns);
  F ga[N][C], gb[N][C], dga[N][C], dgb[N][C];                 // of this lane's components
  lane_gamma<V, N, L, INTER>(sd.gamma, lane, p.rot, h2, ga, gb);
  constexpr int kRow = kPieces<XT> + kPieces<DT>;
  Pairs<XT, V, INTER> rx[N];
  Pairs<DT, V, INTER> rd[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
#pragma unroll
    for (int e = 0; e < C; ++e) dga[k][e] = dgb[k][e] = f_all<F>(0.f);
  }
  // the row to fetch next: the groups' rows of one token after the other
  const XT *x0 = static_cast<const XT *>(sd.w ? p.x[1] : p.x[0]);
  const DT *d0 = static_cast<const DT *>(sd.w ? p.dy[1] : p.dy[0]);
  const long long stride = static_cast<long long>(sd.nblocks) * per;
  long long ftok = static_cast<long long>(sd.block) * per + grp / slots;
  const XT *fx = x0 + ftok * sd.xs;
  const DT *fd = d0 + ftok * sd.H * p.D;
  int fi = 0, fh = slot, foff = slot * p.D;
  auto fetch = [&](int stage) {
    const bool in = ftok < p.ntok && fh < sd.H;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int s = (lane + L * k) * V;
      const bool live = in && s < h2;
      const Place<V, INTER> at(s, p.rot);
      if constexpr (RING) {
        const uint32_t dst = smem_u32(ring) + (stage * N + k) * (kRow * kQThr) + threadIdx.x * 16;
        copy_pairs(dst, live ? fx + foff : x0, at, live);
        copy_pairs(dst + kPieces<XT> * kQThr, live ? fd + foff : d0, at, live);
      } else if (live) {
        rx[k].load(fx + foff, at);
        rd[k].load(fd + foff, at);
      } else {                                                // (adds nothing to sums and dgamma)
        rx[k].clear();
        rd[k].clear();
      }
    }
    if constexpr (RING) copies_commit();
    fh += slots, foff += hop;
    if (++fi == steps) {
      fi = 0, fh = slot, foff = slot * p.D;
      ftok += stride;
      fx += stride * sd.xs;
      fd += stride * sd.H * p.D;
    }
  };
  int stage = 0;
  if constexpr (RING) {
#pragma unroll
    for (int d = 0; d < kBwdStages - 1; ++d) fetch(d);
  } else {
    fetch(0);
  }
  for (long long tok0 = static_cast<long long>(sd.block) * per; tok0 < p.ntok; tok0 += stride) {
    const long long tok = tok0 + grp / slots;
    const int H = tok < p.ntok ? sd.H : 0;                    // heads of this group's token
    XT *o = static_cast<XT *>(sd.w ? p.out[1] : p.out[0]) + tok * sd.os;
    int h = slot, off = slot * p.D;
    F c[N][C], z[N][C];
    if (H) {
      lane_angles<V, N, L>(p, turns, tok, lane, c, z);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int e = 0; e < C; ++e) c[k][e] = z[k][e] = f_all<F>(0.f);
    }
    // every lane of a warp makes the same number of steps: the row sums
    // exchange values across it
    for (int i = 0; i < steps; ++i, h += slots, off += hop) {
      F a[N][C], b[N][C], u[N][C], v[N][C];
      F ss = f_all<F>(0.f), cc = f_all<F>(0.f);
      if constexpr (RING) {
        copies_wait<kBwdStages - 2>();
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const unsigned char *src = ring + (stage * N + k) * (kRow * kQThr) + threadIdx.x * 16;
          take_pairs(rx[k], src);
          take_pairs(rd[k], src + kPieces<XT> * kQThr);
        }
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        F da[C], db[C];
        rx[k].get(a[k], b[k]);
        rd[k].get(da, db);
        // dn = R(-theta) dy; with the norm, c = sum dn gamma x
#pragma unroll
        for (int e = 0; e < C; ++e) {
          u[k][e] = f_fma(db[e], z[k][e], f_mul(da[e], c[k][e]));
          v[k][e] = f_fma(db[e], c[k][e], f_mul(f_mul(da[e], f_all<F>(-1.f)), z[k][e]));
        }
      }
      if constexpr (RING) {
        // into the stage that the last step took its row from
        fetch(stage == 0 ? kBwdStages - 1 : stage - 1);
        if (++stage == kBwdStages) stage = 0;
      } else {
        fetch(0);
      }
      float inv = 1.f, coef = 0.f;
      if (norm) {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int e = 0; e < C; ++e) {
            ss = f_fma(a[k][e], a[k][e], f_fma(b[k][e], b[k][e], ss));
            cc = f_fma(f_mul(u[k][e], ga[k][e]), a[k][e], f_fma(f_mul(v[k][e], gb[k][e]), b[k][e], cc));
          }
        const float s2 = lanes_sum<L>(f_sum(ss)), c2 = lanes_sum<L>(f_sum(cc));
        inv = inv_root(fmaf(s2, p.inv_n, p.eps));
        coef = -c2 * p.inv_n * (inv * inv);                   // -c / (D rms^2)
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int e = 0; e < C; ++e) {
            const F r = f_all<F>(inv), xa = f_mul(a[k][e], r), xb = f_mul(b[k][e], r);
            const F ua = f_mul(f_mul(u[k][e], ga[k][e]), r), vb = f_mul(f_mul(v[k][e], gb[k][e]), r);
            dga[k][e] = f_fma(u[k][e], xa, dga[k][e]);
            dgb[k][e] = f_fma(v[k][e], xb, dgb[k][e]);
            u[k][e] = f_fma(xa, f_all<F>(coef), ua);
            v[k][e] = f_fma(xb, f_all<F>(coef), vb);
          }
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int s = (lane + L * k) * V;
        if (h < H && s < h2) {
          Pairs<XT, V, INTER> out;
          out.set(u[k], v[k]);
          out.store(o + off, Place<V, INTER>(s, p.rot));
        }
      }
    }
  }
  // one partial dgamma per block, its row groups added in a fixed order
  if constexpr (RING) copies_wait<0>();
  if (p.part == nullptr) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int s = (lane + L * k) * V;
    if (s < h2) {
      Pairs<float, V, INTER> out;
      out.set(dga[k], dgb[k]);
      out.store(sums + grp * p.D, Place<V, INTER>(s, p.rot));
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.D; i += kQThr) {
    float t = 0.f;
    for (int g = 0; g < kGroups; ++g) t += sums[g * p.D + i];
    p.part[static_cast<size_t>(blockIdx.x) * p.D + i] = t;
  }
}

// dgamma = sum of the blocks' partials, in a fixed order: a block takes 32
// components of queries or keys, its 32 warps every 32nd partial (8 warps: 3 us
// more for 600 partials, all of it waiting for loads).
constexpr int kGammaWarps = 32;
__global__ void __launch_bounds__(32 * kGammaWarps)
    qk_dgamma_kernel(const float *part, float *__restrict__ dgq, float *__restrict__ dgk, int first_k, int nparts, int D) {
  __shared__ float red[kGammaWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float *dst = blockIdx.y ? dgk : dgq;
  const int lo = blockIdx.y ? first_k : 0, hi = blockIdx.y ? nparts : first_k;
  float t = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (col < D) {
#pragma unroll 8
    for (int i = lo + warp; i < hi; i += kGammaWarps) t += __ldcg(part + static_cast<size_t>(i) * D + col);
  }
  red[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && col < D) {
    for (int i = 1; i < kGammaWarps; ++i) t += red[i][lane];
    if (dst) dst[col] = t;
  }
}

template <typename XT, typename DT, bool BWD, bool INTER, int V, int N, int L>
cudaError_t qk_launch(QkParams &p, const unsigned long long *freq, int sms, cudaStream_t st) {
  // Lane groups per token: one forms the token's angles once for all its heads,
  // more of them keep the SMs busy when tokens are few.  Up to kFill groups an
  // SM as long as each has four rows (2050 tokens, 20 + 5 heads of 80 fp32:
  // 12 us, with fewer rows each 16), up to a block an SM in any case.
  constexpr int kGroups = kQThr / L, kFill = 4 * kGroups;
  long long blocks[2];
  for (int w = 0; w < 2; ++w) {
    int slots = 1;
    while (slots < kGroups && 8 * slots <= p.H[w] && p.ntok * slots < static_cast<long long>(kFill) * sms) slots *= 2;
    while (slots < kGroups && slots < p.H[w] && p.ntok * slots < static_cast<long long>(kGroups) * sms) slots *= 2;
    p.slots[w] = slots;
    const int per = kGroups / slots;
    blocks[w] = p.H[w] ? (p.ntok + per - 1) / per : 0;
  }
  // rows of a group of lanes: its token's heads, and in the backward those of
  // the tokens that it goes on to
  const int w0 = p.H[0] ? 0 : 1;
  long long rows = (p.H[w0] + p.slots[w0] - 1) / p.slots[w0];
  if (BWD) {
    const long long most = bwd_blocks(false) * static_cast<long long>(sms);
    if (blocks[0] + blocks[1] > most) rows *= (blocks[0] + blocks[1]) / most;
  }
  const bool ring = V == 4 && rows >= kRingRows;
  if (BWD) {
    // resident blocks, shared out by the number of heads
    const long long all = (V == 4 && N == 1 ? bwd_blocks(ring) : 2) * static_cast<long long>(sms);
    const long long most = all < kQkParts ? all : kQkParts;
    long long q = most * p.H[0] / (p.H[0] + p.H[1]);
    if (p.H[0] && q < 1) q = 1;
    if (p.H[1] && q > most - 1) q = most - 1;
    if (blocks[0] > q) blocks[0] = q;
    if (blocks[1] > most - q) blocks[1] = most - q;
  }
  if (blocks[0] + blocks[1] > 0x7fffffffLL) return cudaErrorInvalidValue;
  p.first_k = static_cast<int>(blocks[0]);
  QkTable<table_size<V, L>()> t;
  static_cast<QkParams &>(t) = p;
  for (int i = 0; i < p.rot; ++i) t.freq[i] = freq[i];
  const unsigned grid = static_cast<unsigned>(blocks[0] + blocks[1]);
  if constexpr (BWD) {
    const auto kern = ring ? qk_bwd_kernel<XT, DT, INTER, V, N, L, V == 4> : qk_bwd_kernel<XT, DT, INTER, V, N, L, false>;
    const int need = p.part ? kGroups * p.D * 4 : 0, rb = ring ? kBwdStages * N * (kPieces<XT> + kPieces<DT>) * kQThr : 0;
    const int smem = need > rb ? need : rb;
    if (smem > 40960) {
      const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), smem);
      if (e != cudaSuccess) return e;
    }
    kern<<<grid, kQThr, smem, st>>>(t);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.part) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.D + 31) / 32, 2);
    cfg.blockDim = dim3(32 * kGammaWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qk_dgamma_kernel, static_cast<const float *>(p.part), p.dgamma[0], p.dgamma[1],
                              p.first_k, static_cast<int>(grid), p.D);
  } else {
    constexpr int U = V == 1 || N > 1 ? 1 : 2;
    const auto kern = ring ? qk_fwd_kernel<XT, INTER, V, N, L, U, V == 4> : qk_fwd_kernel<XT, INTER, V, N, L, U, false>;
    const int smem = ring ? kFwdStages * U * N * kPieces<XT> * kQThr : 0;
    if (smem > 40960) {
      const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), smem);
      if (e != cudaSuccess) return e;
    }
    kern<<<grid, kQThr, smem, st>>>(t);
  }
  return cudaGetLastError();
}

template <typename XT, typename DT, bool BWD, bool INTER>
cudaError_t qk_dispatch(QkParams &p, const unsigned long long *freq, bool vec, int sms, cudaStream_t st) {
  if (!vec) return qk_launch<XT, DT, BWD, INTER, 1, 8, 32>(p, freq, sms, st);
  if (p.D <= 64) return qk_launch<XT, DT, BWD, INTER, 4, 1, 8>(p, freq, sms, st);
  if (p.D <= 128) return qk_launch<XT, DT, BWD, INTER, 4, 1, 16>(p, freq, sms, st);
  if (p.D <= 256) return qk_launch<XT, DT, BWD, INTER, 4, 1, 32>(p, freq, sms, st);
  return qk_launch<XT, DT, BWD, INTER, 4, 2, 32>(p, freq, sms, st);
}

// Turns per position of each pair, mod 1, as 64-bit binary fractions.  A model
// calls with one base and size, so each thread keeps the last table it formed.
const unsigned long long *turn_table(double base, int rotary_dim) {
  thread_local double last_base = 0.0;
  thread_local int last_dim = 0;
  thread_local unsigned long long turns[kQMaxPairs];
  if (base != last_base || rotary_dim != last_dim) {
    for (int i = 0; i < rotary_dim / 2; ++i)
      turns[i] = static_cast<unsigned long long>(
          ldexp(fmod(pow(base, -2.0 * i / rotary_dim) / 6.283185307179586476925286766559, 1.0), 64));
    last_base = base;
    last_dim = rotary_dim;
  }
  return turns;
}

bool at16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

size_t qk_norm_rope_bwd_workspace_bytes(int D) { return static_cast<size_t>(kQkParts) * D * 4; }

cudaError_t launch_qk_norm_rope(const QkNormRopeArgs &a, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const bool bwd = a.backward;
  QkParams p;
  const int rot = a.rotary_dim / 2;
  // 16-byte accesses: pairs come in groups of 4, so D is a multiple of 8, a
  // group of split pairs does not straddle the end of the rotation, and every
  // row starts on a 16-byte boundary
  bool vec = a.D % 8 == 0 && (a.interleaved || rot % 4 == 0);
  const long long unit = a.bf16 ? 8 : 4;
  for (int w = 0; w < 2; ++w) {
    p.x[w] = a.x[w], p.dy[w] = a.dy[w], p.out[w] = a.out[w], p.gamma[w] = a.gamma[w], p.dgamma[w] = a.dgamma[w];
    p.xs[w] = a.x_stride[w], p.os[w] = a.out_stride[w];
    p.H[w] = a.H[w];
    if (a.H[w] == 0) continue;
    vec = vec && at16(a.x[w]) && at16(a.out[w]) && a.x_stride[w] % unit == 0 && a.out_stride[w] % unit == 0;
  }
  p.part = bwd && (a.gamma[0] || a.gamma[1]) ? static_cast<float *>(a.ws) : nullptr;
  p.D = a.D, p.rot = rot, p.T = a.T, p.pos0 = a.pos0;
  p.ntok = static_cast<long long>(a.B) * a.T;
  p.eps = a.eps;
  p.inv_n = 1.f / static_cast<float>(a.D);
  p.pos = a.positions;
  for (int i = 0, end = 0; i < 3; ++i) {
    end += a.sections[i];
    p.sec_end[i] = i + 1 < a.n_axes ? end : 0x7fffffff;
  }
  const unsigned long long *freq = turn_table(a.base, a.rotary_dim);
  if (p.ntok > 0 && a.H[0] + a.H[1] > 0) {
    if (!bwd) {
      if (a.bf16)
        e = a.interleaved ? qk_dispatch<__nv_bfloat16, float, false, true>(p, freq, vec, sms, st)
                          : qk_dispatch<__nv_bfloat16, float, false, false>(p, freq, vec, sms, st);
      else
        e = a.interleaved ? qk_dispatch<float, float, false, true>(p, freq, vec, sms, st)
                          : qk_dispatch<float, float, false, false>(p, freq, vec, sms, st);
      return e;
    }
    const int how = (a.bf16 ? 4 : 0) | (a.dy_bf16 ? 2 : 0) | (a.interleaved ? 1 : 0);
    using bf = __nv_bfloat16;
    switch (how) {
      case 0: e = qk_dispatch<float, float, true, false>(p, freq, vec, sms, st); break;
      case 1: e = qk_dispatch<float, float, true, true>(p, freq, vec, sms, st); break;
      case 2: e = qk_dispatch<float, bf, true, false>(p, freq, vec, sms, st); break;
      case 3: e = qk_dispatch<float, bf, true, true>(p, freq, vec, sms, st); break;
      case 4: e = qk_dispatch<bf, float, true, false>(p, freq, vec, sms, st); break;
      case 5: e = qk_dispatch<bf, float, true, true>(p, freq, vec, sms, st); break;
      case 6: e = qk_dispatch<bf, bf, true, false>(p, freq, vec, sms, st); break;
      default: e = qk_dispatch<bf, bf, true, true>(p, freq, vec, sms, st); break;
    }
    return e;
  }
  for (int w = 0; w < 2 && bwd && e == cudaSuccess; ++w)
    if (a.dgamma[w]) e = cudaMemsetAsync(a.dgamma[w], 0, static_cast<size_t>(a.D) * 4, st);
  return e;
}

}  // namespace abw
