// What the windowed attention's kernels share: which blocks of 128 keys a block
// of 128 queries meets, and small pieces of arithmetic.
#pragma once

#include <math.h>

#include "abw_host.h"
#include "tcgen05.cuh"

namespace abw {
namespace win {

constexpr int kBlk = 128;   // queries and keys per block
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

// Tokens of sequence b.
__device__ __forceinline__ int tokens_of(const int *lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}
// The same where a whole warp asks for one b: a value that the compiler knows to
// be uniform, so what follows from it stays in uniform registers, which the
// tensor core's instructions take their operands from.
__device__ __forceinline__ int tokens_warp(const int *lengths, int b, int T) {
  return lengths ? __shfl_sync(0xffffffffu, tokens_of(lengths, b, T), 0) : T;
}

// n / d for 0 <= n < 2^31 by a product: m = ceil(2^(31 + k) / d) with 2^k >= d > 2^(k - 1)
// is off by e < d 2^-(31 + k) <= 2^-31 from 2^(31 + k) / d, relative to it below 1 / n.
struct Div {
  unsigned d, mul, shift;
  static Div by(int x) {
    Div r;
    r.d = x;
    unsigned k = 0;
    while ((1ull << k) < r.d) ++k;
    r.mul = static_cast<unsigned>(((1ull << (31 + k)) + r.d - 1) / r.d);
    r.shift = k;
    return r;
  }
  // quotient; n becomes the remainder
  __device__ __forceinline__ int operator()(int &n) const {
    const unsigned q = static_cast<unsigned>((static_cast<unsigned long long>(mul) * static_cast<unsigned>(n)) >> 31) >> shift;
    n -= q * d;
    return q;
  }
};

// Item of a CTA's r-th round, in rounds that go through the CTAs back and forth: items
// become shorter towards the list's end, so the CTAs' sums come out alike.
__device__ __forceinline__ int nth_item(int r) {
  const int c = blockIdx.x, n = gridDim.x;
  return r * n + ((r & 1) ? n - 1 - c : c);
}

// The lowest x of 32 bits.
__device__ __forceinline__ uint32_t below(int x) {
  const int n = min(max(x, 0), 32);
  return n == 32 ? 0xffffffffu : (1u << n) - 1u;
}

// 2^x on the MUFU unit, to some 2^-22; 2^-inf = 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two fp32 operations at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long &>(d))
      : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)),
        "l"(reinterpret_cast<unsigned long long &>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long &>(d))
      : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
  return d;
}

// Waits of a kernel's roles.  All of them stop once one has run out: the first
// to give up reports it, the others find the flag.  The polling is out of line, as
// is whatever else runs seldom: the roles of a block run different code at one
// time, and it has to fit the instruction cache (with it in line, and an election for
// every instruction of a product, the forward of 8192 tokens of 32 heads, window 1024,
// took 174 us in place of 159; other changes brought it to 136).
struct Waits {
  uint32_t bars;                  // shared address of barrier 0
  volatile int *abort_flag;
  const WaitCtl *ctl;
  unsigned site;
};
static __device__ __noinline__ bool wait_slowly(uint32_t bar, uint32_t parity, const Waits &w) {
  WaitClock wc(w.ctl->limit_ns);
  while (!*w.abort_flag) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (wc.expired()) {
      *w.abort_flag = 1;
      report_timeout(w.ctl->err, w.site, (bar - w.bars) / 8);
    }
  }
  return false;
}
__device__ __forceinline__ bool wait_one(const Waits &w, int slot, uint32_t parity) {
  const uint32_t bar = w.bars + slot * 8;
  return mbar_try_wait(bar, parity) || wait_slowly(bar, parity, w);
}
// In line and without a call, for the warp that issues products: a call would
// empty its uniform registers.  `gave_up` is 1 + the slot of a wait that ran out,
// which the warp reports behind its loop.
__device__ __forceinline__ bool wait_issuer(const Waits &w, int slot, uint32_t parity, int &gave_up) {
  const uint32_t bar = w.bars + slot * 8;
  bool done = mbar_try_wait(bar, parity);
  if (!done) {
    WaitClock wc(w.ctl->limit_ns);
    while (!*w.abort_flag) {
#pragma unroll 1
      for (int i = 0; i < 32 && !done; ++i) done = mbar_try_wait(bar, parity);
      if (done) break;
      if (wc.expired()) {
        gave_up = slot + 1;
        *w.abort_flag = 1;
      }
    }
  }
  return __shfl_sync(0xffffffffu, done, 0);
}
__device__ __forceinline__ void report_issuer(const Waits &w, int gave_up) {
  if (gave_up != 0) report_timeout(w.ctl->err, w.site, gave_up - 1);
}
// Whole-warp form: lane 0's outcome for every lane, so that a warp never splits
// in front of a warp-collective instruction.
__device__ __forceinline__ bool wait_warp(const Waits &w, int slot, uint32_t parity) {
  return __shfl_sync(0xffffffffu, wait_one(w, slot, parity), 0);
}
// The end of a copy that is under way, which has to come before its shared memory is
// let go of, whoever gave up and when.
static __device__ __noinline__ void wait_landed(uint32_t bar, uint32_t parity) {
  mbar_wait_bounded(bar, parity, 2000000000ull);
}

// Clears rows live .. 127 of a block of [halves][128 rows][128 B] whose copy is
// under way behind barrier `raw`, then hands it on behind barrier `full`; by a
// whole warp.
template <int kHalves>
static __device__ __noinline__ void clear_tail(const Waits &w, unsigned char *at, int live, int raw, uint32_t parity,
                                               uint32_t full) {
  if (!wait_one(w, raw, parity)) wait_landed(w.bars + raw * 8, parity);
  __syncwarp();
  for (int i = max(live, 0) * 8 + (threadIdx.x & 31); i < kBlk * 8; i += 32)
#pragma unroll
    for (int hx = 0; hx < kHalves; ++hx) *reinterpret_cast<uint4 *>(at + hx * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(full);
}

// bf16 [B][T][H][kD] rows with a token stride (elements), in boxes of 64
// components x `rows` tokens, 128B-swizzled.
inline bool token_map(CUtensorMap *m, const void *base, int H, int T, int B, int D, long long stride, int rows,
                      const char **why) {
  const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(H), static_cast<uint64_t>(T),
                            static_cast<uint64_t>(B)};
  const uint64_t st = static_cast<uint64_t>(stride) * 2;
  const uint64_t strides[3] = {static_cast<uint64_t>(D) * 2, st, st * T};
  const uint32_t box[4] = {64, 1, static_cast<uint32_t>(rows), 1};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                      why);
}

}  // namespace win
}  // namespace abw
