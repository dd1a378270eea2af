// Softmax attention over a sliding window with first tokens that stay visible:
// query i sees key j where j <= i and (j > i - window or j < sinks).
//
// Plain kernels, one warp per row: the forward and dq walk the keys a query
// sees, dk and dv the queries that see a key.
#include <math.h>

#include "abw_host.h"

namespace abw {
namespace {

constexpr int kThr = 256;
constexpr float kLog2e = 1.4426950408889634f;

struct WinParams {
  const __nv_bfloat16 *q, *k, *v, *dout;
  const int *lengths;
  __nv_bfloat16 *o, *dq, *dk, *dv;
  float *lse, *delta;
  int B, T, Hq, Hkv, G;
  long long q_stride, k_stride, v_stride, o_stride, dq_stride, dk_stride, dv_stride;
  int window, sinks;
  float scale;
};

template <int kD>
struct Row {
  float x[kD / 32];
  __device__ void load(const __nv_bfloat16 *p, int lane) {
#pragma unroll
    for (int i = 0; i < kD / 32; ++i) x[i] = __bfloat162float(p[lane + 32 * i]);
  }
  __device__ void store(__nv_bfloat16 *p, int lane, float f) const {
#pragma unroll
    for (int i = 0; i < kD / 32; ++i) p[lane + 32 * i] = __float2bfloat16_rn(x[i] * f);
  }
  __device__ float dot(const Row &o) const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kD / 32; ++i) s = fmaf(x[i], o.x[i], s);
    return warp_sum(s);
  }
  __device__ void add(float f, const Row &o) {
#pragma unroll
    for (int i = 0; i < kD / 32; ++i) x[i] = fmaf(f, o.x[i], x[i]);
  }
  __device__ void zero() {
#pragma unroll
    for (int i = 0; i < kD / 32; ++i) x[i] = 0.f;
  }
};

__device__ __forceinline__ int tokens_of(const WinParams &p, int b) {
  return p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
}

template <int kD, bool kBackward>
__global__ void __launch_bounds__(kThr) window_query_kernel(const __grid_constant__ WinParams p) {
  const long long r = static_cast<long long>(blockIdx.x) * (kThr / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= static_cast<long long>(p.B) * p.T * p.Hq) return;
  const int h = static_cast<int>(r % p.Hq);
  const long long tok = r / p.Hq;
  const int i = static_cast<int>(tok % p.T), b = static_cast<int>(tok / p.T), kvh = h / p.G;
  const size_t stat = (static_cast<size_t>(b) * p.Hq + h) * p.T + i;
  const int n = tokens_of(p, b);
  Row<kD> acc, q, d, x;
  acc.zero();
  float m = -INFINITY, l = 0.f, delta = 0.f, lse = 0.f;
  if (i < n) {
    q.load(p.q + tok * p.q_stride + static_cast<size_t>(h) * kD, lane);
    if (kBackward) {
      d.load(p.dout + (tok * p.Hq + h) * kD, lane);
      x.load(p.o + tok * p.o_stride + static_cast<size_t>(h) * kD, lane);
      delta = d.dot(x);
      lse = p.lse[stat];
    }
    const long long t0 = static_cast<long long>(b) * p.T;
    for (int j = 0; j <= i; ++j) {
      if (j >= p.sinks && j <= i - p.window) {
        j = i - p.window;   // on to the window
        continue;
      }
      x.load(p.k + (t0 + j) * p.k_stride + static_cast<size_t>(kvh) * kD, lane);
      const float s = q.dot(x) * p.scale;
      Row<kD> y;
      y.load(p.v + (t0 + j) * p.v_stride + static_cast<size_t>(kvh) * kD, lane);
      if (kBackward) {
        acc.add(exp2f((s - lse) * kLog2e) * (d.dot(y) - delta), x);
      } else {
        const float mn = fmaxf(m, s), f = exp2f((m - mn) * kLog2e), e = exp2f((s - mn) * kLog2e);
#pragma unroll
        for (int c = 0; c < kD / 32; ++c) acc.x[c] *= f;
        acc.add(e, y);
        l = l * f + e;
        m = mn;
      }
    }
  }
  if (kBackward) {
    acc.store(p.dq + tok * p.dq_stride + static_cast<size_t>(h) * kD, lane, p.scale);
    if (lane == 0) p.delta[stat] = delta;
  } else {
    acc.store(p.o + tok * p.o_stride + static_cast<size_t>(h) * kD, lane, i < n ? 1.f / l : 0.f);
    if (lane == 0) p.lse[stat] = i < n ? m + logf(l) : -INFINITY;
  }
}

template <int kD>
__global__ void __launch_bounds__(kThr) window_key_kernel(const __grid_constant__ WinParams p) {
  const long long r = static_cast<long long>(blockIdx.x) * (kThr / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= static_cast<long long>(p.B) * p.T * p.Hkv) return;
  const int kvh = static_cast<int>(r % p.Hkv);
  const long long tok = r / p.Hkv;
  const int j = static_cast<int>(tok % p.T), b = static_cast<int>(tok / p.T);
  const int n = tokens_of(p, b);
  Row<kD> dk, dv;
  dk.zero();
  dv.zero();
  if (j < n) {
    Row<kD> k, v, q, d;
    k.load(p.k + tok * p.k_stride + static_cast<size_t>(kvh) * kD, lane);
    v.load(p.v + tok * p.v_stride + static_cast<size_t>(kvh) * kD, lane);
    const int last = j < p.sinks || p.window >= n - j ? n - 1 : j + p.window - 1;
    for (int h = kvh * p.G; h < (kvh + 1) * p.G; ++h)
      for (int i = j; i <= last; ++i) {
        const long long ti = static_cast<long long>(b) * p.T + i;
        const size_t stat = (static_cast<size_t>(b) * p.Hq + h) * p.T + i;
        q.load(p.q + ti * p.q_stride + static_cast<size_t>(h) * kD, lane);
        d.load(p.dout + (ti * p.Hq + h) * kD, lane);
        const float w = exp2f((q.dot(k) * p.scale - p.lse[stat]) * kLog2e);
        dv.add(w, d);
        dk.add(w * (d.dot(v) - p.delta[stat]), q);
      }
  }
  dk.store(p.dk + tok * p.dk_stride + static_cast<size_t>(kvh) * kD, lane, p.scale);
  dv.store(p.dv + tok * p.dv_stride + static_cast<size_t>(kvh) * kD, lane, 1.f);
}

WinParams params(const WindowArgs &a) {
  WinParams p;
  p.q = static_cast<const __nv_bfloat16 *>(a.q), p.k = static_cast<const __nv_bfloat16 *>(a.k);
  p.v = static_cast<const __nv_bfloat16 *>(a.v), p.dout = static_cast<const __nv_bfloat16 *>(a.dout);
  p.lengths = a.lengths;
  p.o = static_cast<__nv_bfloat16 *>(a.o), p.dq = static_cast<__nv_bfloat16 *>(a.dq);
  p.dk = static_cast<__nv_bfloat16 *>(a.dk), p.dv = static_cast<__nv_bfloat16 *>(a.dv);
  p.lse = a.lse, p.delta = static_cast<float *>(a.ws);
  p.B = a.B, p.T = a.T, p.Hq = a.Hq, p.Hkv = a.Hkv, p.G = a.Hq / a.Hkv;
  p.q_stride = a.q_stride, p.k_stride = a.k_stride, p.v_stride = a.v_stride, p.o_stride = a.o_stride;
  p.dq_stride = a.dq_stride, p.dk_stride = a.dk_stride, p.dv_stride = a.dv_stride;
  p.window = a.window, p.sinks = a.sinks;
  p.scale = a.scale;
  return p;
}

unsigned blocks_of(long long rows) { return static_cast<unsigned>((rows + kThr / 32 - 1) / (kThr / 32)); }

}  // namespace

size_t window_bwd_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int window, int sinks) {
  (void)Hkv, (void)D, (void)window, (void)sinks;
  return static_cast<size_t>(B) * T * Hq * 4;
}

cudaError_t launch_window_bwd(const WindowArgs &a, const WaitCtl &w, cudaStream_t st, const char **why) {
  (void)w, (void)why;
  const WinParams p = params(a);
  const unsigned gq = blocks_of(static_cast<long long>(a.B) * a.T * a.Hq);
  const unsigned gk = blocks_of(static_cast<long long>(a.B) * a.T * a.Hkv);
  if (a.D == 64) window_query_kernel<64, true><<<gq, kThr, 0, st>>>(p);
  else window_query_kernel<128, true><<<gq, kThr, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.D == 64) window_key_kernel<64><<<gk, kThr, 0, st>>>(p);
  else window_key_kernel<128><<<gk, kThr, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace abw
