// RMS norm of every query and key head with the position rotation in the same
// pass, forward and backward.  Per head row x[D]:
//   rms = sqrt(mean x^2 + eps),  n = x gamma / rms,  y = R(theta) n
// R turns the pairs of the first rotary_dim components, theta_i = pos base^(-2i
// / rotary_dim), pos the token's position on the axis that pair i belongs to.
// Backward, with dn = R(-theta) dy and c = sum dn gamma x:
//   dx = (dn gamma - x c / (D rms^2)) / rms,   dgamma = sum over rows dn x / rms
//
// Bound by memory: x is read once and y written once (backward: x and dy read,
// dx written); the norm's sum is taken in registers.  A row belongs to 8-32
// lanes, each with V pairs; a block takes the rows of a few tokens, so the
// angles of a token are formed once for all its heads.
//
// Angles without double precision: the host forms the turns per position,
// base^(-2i / rotary_dim) / (2 pi) mod 1, as a 64-bit binary fraction; an
// integer product with the position, modulo 2^64, is the angle modulo one turn,
// exact to 2^-32 turns for every 32-bit position, negative ones included.
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
  float *part;                        // backward: [gridDim.x][2][D] partial dgamma
  long long xs[2], os[2];             // elements from token to token
  int H[2];
  int D, rot;                         // components per head, pairs that turn
  int T, pos0, tt;                    // tokens per block and step
  long long ntok;
  float eps, inv_n;
  const int *pos;                     // [axes][ntok] or null: pos0 + t
  int axes, sec_end[4];               // first pair behind each axis' pairs
};

// A launch's parameters are written out with it: heads of up to 128 components
// carry a table of 64 turns, longer ones of 256 (0.5 us less per launch).
template <int NP>
struct QkTable : QkParams {
  unsigned long long freq[NP];
};

template <typename T, int V>
__device__ __forceinline__ void qload(const T *p, float (&v)[V]) {
  if constexpr (V == 4 && sizeof(T) == 2) {
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
    v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
  } else if constexpr (V == 4) {
    const float4 u = __ldg(reinterpret_cast<const float4 *>(p));
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  } else {
    v[0] = static_cast<float>(p[0]);
  }
}

template <typename T, int V>
__device__ __forceinline__ void qstore(T *p, const float (&v)[V]) {
  if constexpr (V == 4 && sizeof(T) == 2) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
  } else if constexpr (V == 4) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    p[0] = static_cast<T>(v[0]);
  }
}

// The V pairs (a[i], b[i]) of pair slots s .. s + V - 1.  Interleaved pairs are
// neighbours; split pairs are rot apart.  Components behind the rotated ones
// are paired with their neighbours (their angle is 0).
template <typename T, int V, bool INTER>
__device__ __forceinline__ void qload_pairs(const T *row, int s, int rot, float (&a)[V], float (&b)[V]) {
  if constexpr (INTER || V == 1) {
    if constexpr (V == 1) {
      const bool near = INTER || s >= rot;
      qload<T, 1>(row + (near ? 2 * s : s), a);
      qload<T, 1>(row + (near ? 2 * s + 1 : s + rot), b);
    } else {
      float lo[4], hi[4];
      if constexpr (sizeof(T) == 2) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(row + 2 * s));
        lo[0] = bf16_lo(u.x), lo[1] = bf16_hi(u.x), lo[2] = bf16_lo(u.y), lo[3] = bf16_hi(u.y);
        hi[0] = bf16_lo(u.z), hi[1] = bf16_hi(u.z), hi[2] = bf16_lo(u.w), hi[3] = bf16_hi(u.w);
      } else {
        qload<T, 4>(row + 2 * s, lo);
        qload<T, 4>(row + 2 * s + 4, hi);
      }
      a[0] = lo[0], b[0] = lo[1], a[1] = lo[2], b[1] = lo[3];
      a[2] = hi[0], b[2] = hi[1], a[3] = hi[2], b[3] = hi[3];
    }
  } else {
    const bool near = s >= rot;
    qload<T, V>(row + (near ? 2 * s : s), a);
    qload<T, V>(row + (near ? 2 * s + V : s + rot), b);
  }
}

template <typename T, int V, bool INTER>
__device__ __forceinline__ void qstore_pairs(T *row, int s, int rot, const float (&a)[V], const float (&b)[V]) {
  if constexpr (INTER && V == 4) {
    const float lo[4] = {a[0], b[0], a[1], b[1]}, hi[4] = {a[2], b[2], a[3], b[3]};
    if constexpr (sizeof(T) == 2) {
      __nv_bfloat162 u[4] = {__floats2bfloat162_rn(lo[0], lo[1]), __floats2bfloat162_rn(lo[2], lo[3]),
                             __floats2bfloat162_rn(hi[0], hi[1]), __floats2bfloat162_rn(hi[2], hi[3])};
      *reinterpret_cast<uint4 *>(row + 2 * s) =
          make_uint4(*reinterpret_cast<uint32_t *>(&u[0]), *reinterpret_cast<uint32_t *>(&u[1]),
                     *reinterpret_cast<uint32_t *>(&u[2]), *reinterpret_cast<uint32_t *>(&u[3]));
    } else {
      qstore<T, 4>(row + 2 * s, lo);
      qstore<T, 4>(row + 2 * s + 4, hi);
    }
  } else {
    const bool near = INTER || s >= rot;
    qstore<T, V>(row + (near ? 2 * s : s), a);
    qstore<T, V>(row + (near ? 2 * s + V : s + rot), b);
  }
}

// cos and sin of nt tokens' angles, [nt][D / 2] each; 1 and 0 behind the
// rotated pairs.
template <int NP>
__device__ __forceinline__ void fill_angles(const QkTable<NP> &p, long long tok0, int nt, float *cs, float *sn) {
  const int h2 = p.D >> 1;
  for (int i = threadIdx.x; i < nt * h2; i += kQThr) {
    const int n = i / h2, s = i % h2;
    float c = 1.f, z = 0.f;
    if (s < p.rot) {
      int axis = 0;
      while (axis + 1 < p.axes && s >= p.sec_end[axis]) ++axis;
      const long long tok = tok0 + n;
      const long long pos = p.pos ? p.pos[axis * p.ntok + tok] : static_cast<long long>(p.pos0) + tok % p.T;
      const unsigned long long turns = static_cast<unsigned long long>(pos) * p.freq[s];
      const float half_turns = static_cast<float>(static_cast<int>(turns >> 32)) * 4.656612873077393e-10f;   // 2^-31
      sincospif(half_turns, &z, &c);
    }
    cs[i] = c;
    sn[i] = z;
  }
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int V, int L>
constexpr int table_size() { return V == 4 && L <= 16 ? 64 : kQMaxPairs; }

// N: groups of V pair slots per lane; L: lanes per row.
template <typename XT, typename DT, bool BWD, bool INTER, int V, int N, int L>
__global__ void __launch_bounds__(kQThr) qk_kernel(const __grid_constant__ QkTable<table_size<V, L>()> p) {
  extern __shared__ __align__(16) float ang[];
  const int h2 = p.D >> 1;
  float *cs = ang, *sn = ang + p.tt * h2;
  constexpr int kGroups = kQThr / L;
  const int lane = threadIdx.x % L, grp = threadIdx.x / L;
  float dga[2][N][V], dgb[2][N][V];     // dgamma of this lane's components
  if constexpr (BWD) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) dga[w][k][e] = dgb[w][k][e] = 0.f;
  }
  for (long long tok0 = static_cast<long long>(blockIdx.x) * p.tt; tok0 < p.ntok;
       tok0 += static_cast<long long>(gridDim.x) * p.tt) {
    const int nt = static_cast<int>(min(static_cast<long long>(p.tt), p.ntok - tok0));
    __syncthreads();
    fill_angles(p, tok0, nt, cs, sn);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int H = p.H[w], rows = nt * H;
      if (rows == 0) continue;
      const bool norm = p.gamma[w] != nullptr;
      float ga[N][V], gb[N][V];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int s = (lane + L * k) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) ga[k][e] = gb[k][e] = 1.f;
        if (norm && s < h2) qload_pairs<float, V, INTER>(p.gamma[w], s, p.rot, ga[k], gb[k]);
      }
      // every lane of a warp makes the same number of steps: the row sums
      // exchange values across it
      for (int r0 = 0; r0 < rows; r0 += kGroups) {
        const int r = r0 + grp;
        const bool on = r < rows;
        const int n = on ? r / H : 0, h = on ? r - n * H : 0;
        const XT *x = static_cast<const XT *>(p.x[w]) + (tok0 + n) * p.xs[w] + static_cast<long long>(h) * p.D;
        XT *o = static_cast<XT *>(p.out[w]) + (tok0 + n) * p.os[w] + static_cast<long long>(h) * p.D;
        float a[N][V], b[N][V], da[N][V], db[N][V];
        float ss = 0.f, cc = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int s = (lane + L * k) * V;
#pragma unroll
          for (int e = 0; e < V; ++e) a[k][e] = b[k][e] = 0.f;
          if constexpr (BWD) {
#pragma unroll
            for (int e = 0; e < V; ++e) da[k][e] = db[k][e] = 0.f;
          }
          if (on && s < h2) {
            qload_pairs<XT, V, INTER>(x, s, p.rot, a[k], b[k]);
            if constexpr (BWD)
              qload_pairs<DT, V, INTER>(static_cast<const DT *>(p.dy[w]) + ((tok0 + n) * H + h) * p.D, s, p.rot, da[k],
                                        db[k]);
          }
#pragma unroll
          for (int e = 0; e < V; ++e) ss = fmaf(a[k][e], a[k][e], fmaf(b[k][e], b[k][e], ss));
        }
        if constexpr (BWD) {
          // dn = R(-theta) dy; with the norm, c = sum dn gamma x
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const int s = (lane + L * k) * V;
            if (on && s < h2) {
#pragma unroll
              for (int e = 0; e < V; ++e) {
                const float c = cs[n * h2 + s + e], z = sn[n * h2 + s + e];
                const float u = da[k][e] * c + db[k][e] * z;
                db[k][e] = db[k][e] * c - da[k][e] * z;
                da[k][e] = u;
                cc = fmaf(da[k][e] * ga[k][e], a[k][e], fmaf(db[k][e] * gb[k][e], b[k][e], cc));
              }
            }
          }
        }
        float inv = 1.f, coef = 0.f;
        if (norm) {
          ss = lanes_sum<L>(ss);
          const float ms = fmaf(ss, p.inv_n, p.eps);          // rms^2
          inv = 1.f / sqrtf(ms);
          if constexpr (BWD) {
            cc = lanes_sum<L>(cc);
            coef = cc * p.inv_n / ms;
          }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int s = (lane + L * k) * V;
          if (on && s < h2) {
            float ya[V], yb[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
              if constexpr (BWD) {
                if (norm) {
                  dga[w][k][e] = fmaf(da[k][e] * a[k][e], inv, dga[w][k][e]);
                  dgb[w][k][e] = fmaf(db[k][e] * b[k][e], inv, dgb[w][k][e]);
                  ya[e] = (da[k][e] * ga[k][e] - a[k][e] * coef) * inv;
                  yb[e] = (db[k][e] * gb[k][e] - b[k][e] * coef) * inv;
                } else {
                  ya[e] = da[k][e];
                  yb[e] = db[k][e];
                }
              } else {
                const float c = cs[n * h2 + s + e], z = sn[n * h2 + s + e];
                const float u = a[k][e] * inv * ga[k][e], v = b[k][e] * inv * gb[k][e];
                ya[e] = u * c - v * z;
                yb[e] = u * z + v * c;
              }
            }
            qstore_pairs<XT, V, INTER>(o, s, p.rot, ya, yb);
          }
        }
      }
    }
  }
  if constexpr (BWD) {
    // one partial dgamma per block, its row groups added in a fixed order
    if (p.part == nullptr) return;
    float *sums = ang;                  // [kGroups][D]
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int s = (lane + L * k) * V;
        if (s < h2) qstore_pairs<float, V, INTER>(sums + grp * p.D, s, p.rot, dga[w][k], dgb[w][k]);
      }
      __syncthreads();
      for (int i = threadIdx.x; i < p.D; i += kQThr) {
        float t = 0.f;
        for (int g = 0; g < kGroups; ++g) t += sums[g * p.D + i];
        p.part[(static_cast<size_t>(blockIdx.x) * 2 + w) * p.D + i] = t;
      }
    }
  }
}

// dgamma = sum of the blocks' partials, in a fixed order: a block takes 32
// columns, its 8 warps every 8th partial.
__global__ void __launch_bounds__(256) qk_dgamma_kernel(const float *__restrict__ part, float *__restrict__ dgq,
                                                        float *__restrict__ dgk, int nparts, int D) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;               // of [2][D]
  float t = 0.f;
  if (col < 2 * D)
    for (int i = w; i < nparts; i += 8) t += part[static_cast<size_t>(i) * 2 * D + col];
  red[w][lane] = t;
  __syncthreads();
  if (w == 0 && col < 2 * D) {
    for (int i = 1; i < 8; ++i) t += red[i][lane];
    float *dst = col < D ? dgq : dgk;
    if (dst) dst[col < D ? col : col - D] = t;
  }
}

template <typename XT, typename DT, bool BWD, bool INTER, int V, int N, int L>
cudaError_t qk_launch(QkParams &p, const unsigned long long *freq, int max_blocks, int sms, cudaStream_t st) {
  // Tokens per block and step: enough rows for every row group, four times
  // over when there are tokens for all SMs.
  constexpr int kGroups = kQThr / L;
  const int H = p.H[0] + p.H[1];
  int tt = (4 * kGroups + H - 1) / H;
  if (tt > 16) tt = 16;
  while (tt > 1 && (p.ntok + tt - 1) / tt < 4 * sms) tt >>= 1;
  p.tt = tt;
  long long blocks = (p.ntok + tt - 1) / tt;
  if (BWD && blocks > max_blocks) blocks = max_blocks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  size_t smem = static_cast<size_t>(tt) * p.D * 4;
  if (BWD && smem < static_cast<size_t>(kGroups) * p.D * 4) smem = static_cast<size_t>(kGroups) * p.D * 4;
  QkTable<table_size<V, L>()> t;
  static_cast<QkParams &>(t) = p;
  for (int i = 0; i < p.rot; ++i) t.freq[i] = freq[i];
  qk_kernel<XT, DT, BWD, INTER, V, N, L><<<static_cast<unsigned>(blocks), kQThr, smem, st>>>(t);
  p.tt = static_cast<int>(blocks);                      // for the caller: partials written
  return cudaGetLastError();
}

template <typename XT, typename DT, bool BWD, bool INTER>
cudaError_t qk_dispatch(QkParams &p, const unsigned long long *freq, bool vec, int max_blocks, int sms, cudaStream_t st) {
  if (!vec) return qk_launch<XT, DT, BWD, INTER, 1, 8, 32>(p, freq, max_blocks, sms, st);
  if (p.D <= 64) return qk_launch<XT, DT, BWD, INTER, 4, 1, 8>(p, freq, max_blocks, sms, st);
  if (p.D <= 128) return qk_launch<XT, DT, BWD, INTER, 4, 1, 16>(p, freq, max_blocks, sms, st);
  if (p.D <= 256) return qk_launch<XT, DT, BWD, INTER, 4, 1, 32>(p, freq, max_blocks, sms, st);
  return qk_launch<XT, DT, BWD, INTER, 4, 2, 32>(p, freq, max_blocks, sms, st);
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

size_t qk_norm_rope_bwd_workspace_bytes(int D) { return static_cast<size_t>(kQkParts) * 2 * D * 4; }

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
    p.x[w] = a.x[w], p.dy[w] = a.dy[w], p.out[w] = a.out[w], p.gamma[w] = a.gamma[w];
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
  p.axes = a.n_axes;
  for (int i = 0, end = 0; i < 4; ++i) {
    end += i < a.n_axes ? a.sections[i] : 0;
    p.sec_end[i] = end;
  }
  const unsigned long long *freq = turn_table(a.base, a.rotary_dim);
  if (p.ntok > 0) {
    if (!bwd) {
      if (a.bf16)
        e = a.interleaved ? qk_dispatch<__nv_bfloat16, float, false, true>(p, freq, vec, 0, sms, st)
                          : qk_dispatch<__nv_bfloat16, float, false, false>(p, freq, vec, 0, sms, st);
      else
        e = a.interleaved ? qk_dispatch<float, float, false, true>(p, freq, vec, 0, sms, st)
                          : qk_dispatch<float, float, false, false>(p, freq, vec, 0, sms, st);
      return e;
    }
    const int most = kQkParts < 4 * sms ? kQkParts : 4 * sms;
    const int how = (a.bf16 ? 4 : 0) | (a.dy_bf16 ? 2 : 0) | (a.interleaved ? 1 : 0);
    using bf = __nv_bfloat16;
    switch (how) {
      case 0: e = qk_dispatch<float, float, true, false>(p, freq, vec, most, sms, st); break;
      case 1: e = qk_dispatch<float, float, true, true>(p, freq, vec, most, sms, st); break;
      case 2: e = qk_dispatch<float, bf, true, false>(p, freq, vec, most, sms, st); break;
      case 3: e = qk_dispatch<float, bf, true, true>(p, freq, vec, most, sms, st); break;
      case 4: e = qk_dispatch<bf, float, true, false>(p, freq, vec, most, sms, st); break;
      case 5: e = qk_dispatch<bf, float, true, true>(p, freq, vec, most, sms, st); break;
      case 6: e = qk_dispatch<bf, bf, true, false>(p, freq, vec, most, sms, st); break;
      default: e = qk_dispatch<bf, bf, true, true>(p, freq, vec, most, sms, st); break;
    }
    if (e != cudaSuccess || !p.part) return e;
    qk_dgamma_kernel<<<(2 * a.D + 31) / 32, 256, 0, st>>>(p.part, a.dgamma[0], a.dgamma[1], p.tt, a.D);
    return cudaGetLastError();
  }
  for (int w = 0; w < 2 && bwd && e == cudaSuccess; ++w)
    if (a.dgamma[w]) e = cudaMemsetAsync(a.dgamma[w], 0, static_cast<size_t>(a.D) * 4, st);
  return e;
}

}  // namespace abw
