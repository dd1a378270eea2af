// Internal host-side interface between the C ABI (api.cu) and the kernel
// translation units.  Not installed; not part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "abw_device.cuh"

namespace abw {

// Unique id of the calling thread's current CUDA context (0 if none).
// Per-device caches (symbol addresses, raised attribute limits) are keyed on
// it as well as on the ordinal, so that they are resolved again in a context
// created after cudaDeviceReset.
unsigned long long context_id();

// Error word + wait limit for the current device (resolved once per device
// and context).  `err` is null if the symbol address could not be obtained.
WaitCtl wait_ctl();

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// against libcuda).  Returns false and fills `why` on failure.
bool encode_tiled(CUtensorMap *map, CUtensorMapDataType dt, uint32_t rank, const void *base,
                  const uint64_t *dims, const uint64_t *strides_bytes, const uint32_t *box,
                  CUtensorMapSwizzle swizzle, const char **why);

// Points an encoded map at another buffer of the same layout
// (cuTensorMapReplaceAddress).  Returns false where that is not available.
bool move_tiled(CUtensorMap *map, const void *base);

// Raises a kernel's dynamic shared-memory limit on the current device to at
// least `bytes`, calling the runtime only when the limit has to grow: calls
// after the first make no runtime call for it (which keeps them free of
// anything but launches, e.g. under stream capture).
cudaError_t ensure_dynamic_smem(const void *func, int bytes);

// Launchers: validate nothing (api.cu has done it), enqueue, and return the
// launch error.
cudaError_t launch_softmax_bwd(const float *s, const float *dy, float *dx, int rows, int n,
                               cudaStream_t st);
cudaError_t launch_rope_bwd(const float *dy, float *dx, int B, int T, int H, int D, const float *theta,
                            int pos0, double base, int interleaved, cudaStream_t st);
cudaError_t launch_rmsnorm_bwd(const void *x, int x_bf16, const float *gamma, const float *dy, void *dx,
                               int dx_bf16, int rows, int n, float eps, cudaStream_t st);

// Zeroes dgamma, then adds every row's dy x / rms into it; dx may be null.
cudaError_t launch_rmsnorm_bwd_dgamma(const void *x, int x_bf16, const float *gamma, const float *dy, void *dx,
                                      int dx_bf16, float *dgamma, int rows, int n, float eps, cudaStream_t st);
cudaError_t launch_relu2_mul_bwd(const void *gate, const void *up, int bf16, const float *dh, float *dgate,
                                 float *dup, long long n, cudaStream_t st);
size_t lora_workspace_bytes(int rows, int r);
cudaError_t launch_lora_bwd(const void *x, int x_bf16, const float *dy, const float *A, const float *B, float *dA,
                            float *dB, int rows, int n_in, int n_out, int r, float scale, void *ws,
                            cudaStream_t st);

// Returns cudaErrorNotSupported (and sets *why) when a shape has no kernel.
cudaError_t launch_attn_bwd_decode(const float *q, const void *k, const void *v, const float *dout,
                                   float *dq, float *dk, float *dv, int B, int Hq, int Hkv, int S, int D,
                                   int kv_bf16, float scale, double rope_base, int q_pos,
                                   const WaitCtl &w, cudaStream_t st, const char **why);

cudaError_t launch_attn_fwd_causal(const void *q, const void *k, const void *v, void *o, float *lse, int B, int T,
                                   int Hq, int Hkv, int D, float scale, const WaitCtl &w, cudaStream_t st,
                                   const char **why);

size_t causal_workspace_bytes(int B, int T, int Hq, int D);
// pattn: saved probabilities [B][Hq][T][T] bf16 (then lse may be null), or
// null to recompute them from lse.
cudaError_t launch_attn_bwd_causal(const void *q, const void *k, const void *v, const void *pattn, const void *o,
                                   const void *dout, const float *lse, float *dq, float *dk, float *dv,
                                   int B, int T, int Hq, int Hkv, int D, float scale, double rope_base,
                                   int pos0, void *ws, size_t ws_bytes, const WaitCtl &w,
                                   cudaStream_t st, const char **why);

// Per-head norm of queries (index 0) and keys (1) with the rotation.  H 0:
// absent.  Strides are elements from token to token.
struct QkNormRopeArgs {
  const void *x[2], *dy[2];
  void *out[2];
  const float *gamma[2];
  float *dgamma[2];
  int backward, bf16, dy_bf16;
  int B, T, H[2], D;
  long long x_stride[2], out_stride[2];
  float eps;
  double base;
  int rotary_dim, interleaved;        // rotary_dim 0: no rotation
  const int *positions;               // device, [n_axes][B][T], or null
  int n_axes, sections[4], pos0;
  void *ws;
};
constexpr int kQkParts = 1216;        // most partial dgamma rows a backward call writes
size_t qk_norm_rope_bwd_workspace_bytes(int D);
cudaError_t launch_qk_norm_rope(const QkNormRopeArgs &a, cudaStream_t st);

// Linear attention with a decay per KV head; dout null: forward.
struct LinAttnArgs {
  const void *q, *k, *v, *dout;
  const float *log_decay, *initial_state, *dfinal_state;
  const int *lengths;
  void *o, *dq, *dk, *dv;
  float *final_state, *dinitial_state;
  int B, T, Hq, Hkv, D;
  long long q_stride, k_stride, v_stride, o_stride, dq_stride, dk_stride, dv_stride;
  float scale;
  void *ws;
};
size_t lin_attn_workspace_bytes(int B, int T, int Hkv, int D, int backward);
cudaError_t launch_lin_attn(const LinAttnArgs &a, const WaitCtl &w, cudaStream_t st, const char **why);
cudaError_t launch_lin_attn_decode(const void *q, const void *k, const void *v, float *state, const float *log_decay,
                                   const int *slots, void *o, int bf16, int B, int Hq, int Hkv, int D, int nstates,
                                   float scale, cudaStream_t st);

// Attention over a sliding window with first tokens that stay visible; dout
// null: forward.  Strides are elements from token to token.
struct WindowArgs {
  const void *q, *k, *v, *dout;
  const int *lengths;
  void *o, *dq, *dk, *dv;             // o: written forward, read backward
  float *lse;
  int B, T, Hq, Hkv, D;
  long long q_stride, k_stride, v_stride, o_stride, dout_stride, dq_stride, dk_stride, dv_stride;
  int window, sinks;
  float scale;
  void *ws;
};
size_t window_bwd_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int window, int sinks);
cudaError_t launch_window_fwd(const WindowArgs &a, const WaitCtl &w, cudaStream_t st, const char **why);
cudaError_t launch_window_bwd(const WindowArgs &a, const WaitCtl &w, cudaStream_t st, const char **why);

// A paged cache and the rows that a call works on.
struct PagesArgs {
  void *k_pages, *v_pages;
  const int *table, *lengths;
  int B, Hkv, D, n_pages, page_size, max_pages;
};
cudaError_t launch_kv_pages_write(const PagesArgs &a, const void *k, const void *v, const int *starts, int T,
                                  long long k_stride, long long v_stride, cudaStream_t st);
size_t decode_paged_workspace_bytes(int B, int Hq, int Hkv, int D, long long tokens, bool weights);
cudaError_t launch_attn_decode_paged(const PagesArgs &a, const void *q, int bf16, float *weight_sums, void *o, int Hq,
                                     int window, int sinks, float scale, void *ws, cudaStream_t st);
cudaError_t launch_kv_pages_evict(const PagesArgs &a, const float *weight_sums, const int *new_table, int *kept,
                                  int *new_lengths, float *new_weight_sums, int new_max_pages, int budget, int sinks,
                                  int recent, cudaStream_t st);

cudaError_t launch_selftest_wait(const WaitCtl &w, cudaStream_t st);

// Size of the fixed device scratch behind attn_bwd_causal_noalloc.
constexpr size_t kNoAllocScratchBytes = 32ull << 20;   // 32 MiB

// Device address of that scratch on the current device (resolved once per
// device).  Never allocates.
cudaError_t noalloc_scratch(void **ptr, const char **why);

}  // namespace abw
