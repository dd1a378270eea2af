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

// Registers per thread of a warpgroup, from what the block was launched with.
template <int kN>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kN));
}
template <int kN>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kN));
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
