/*
 * attn_bwd.h -- C ABI of the attention backward chain for NVIDIA GB300 (sm_103a).
 *
 * The backward (vector-Jacobian product) of each step of a transformer
 * attention layer, as specified by the CPU specs of the
 * "Hesper.Training.VerifiedBackward" API page and the backward chain of
 * Hesper pull request #1 ("Attention backward GPU kernels"), plus the steps
 * around it that the chain runs (the norm's scale gradient, the FFN's gated
 * activation, the LoRA adapter gradients):
 *
 *   softmax_bwd      dx = s * (dy - sum(s * dy))                     (section Softmax)
 *   rope_bwd         dx = R(-theta) dy per rotary pair               (section RoPE)
 *   rmsnorm_bwd      dx = (dy g - x sum(dy g x) / (n rms^2)) / rms   (section RMSNorm)
 *   attn_bwd_decode  one query per sequence over a KV cache, GQA     (section Attention
 *                    (full single-head): attentionBackwardQ/V; Scaled Dot-Product:
 *                    scaledDotBackwardK), with RoPE backward fused on dq
 *   attn_bwd_causal  T queries over T keys under a causal mask, recomputing the
 *                    probabilities from the saved log-sum-exp; RoPE backward fused on
 *                    dq and dk (DaisyChain-Train transformer.js, backward(): dV = A^T dctx,
 *                    dA = dctx V^T, dS = A (dA - sum A dA), dQ = dS K, dK = dS^T Q)
 *   attn_bwd_causal_saved_p  the same from the saved attention weights (PR #1 softmax fix)
 *   attn_fwd_causal  the forward whose O and log-sum-exp attn_bwd_causal consumes
 *   rmsnorm_bwd_dgamma  rmsnorm_bwd plus dgamma = sum_rows dy x / rms
 *   relu2_mul_bwd    dgate = dh up 2 ReLU(gate), dup = dh ReLU(gate)^2  (PR #1, FFN backward)
 *   lora_bwd         dA, dB of y = s B A x                             (PR #1, LoRA backward)
 *
 * and, next to the softmax attention, the step before it and a second
 * attention of linear cost (neither has a counterpart on those pages):
 *
 *   qk_norm_rope_fwd, qk_norm_rope_bwd  RMS norm of every query and key head with
 *                    the position rotation in the same pass (one or several position axes)
 *   lin_attn_fwd, lin_attn_bwd, lin_attn_decode  linear attention with a decay for each
 *                    KV head: chunked over sequences, recurrent for single tokens
 *   attn_fwd_window, attn_bwd_window  softmax attention over a sliding window with a few
 *                    first tokens that stay visible
 *   kv_pages_write, attn_decode_paged, kv_pages_evict  its serving side: a paged cache,
 *                    one new token over it, and eviction by accumulated attention weight
 *
 * Conventions shared by every entry point
 *   - All pointers are DEVICE pointers (cudaMalloc'd or equivalent), owned by
 *     the caller.  The library never allocates device memory.  Scratch memory,
 *     where an operation needs it, is a caller-provided workspace.
 *   - Work is enqueued on `stream` (NULL = the legacy default stream) and the
 *     call returns without synchronizing.  Outputs are overwritten, never
 *     accumulated into (but weight_sums of attn_decode_paged, and pages, of
 *     which a call writes the rows that it names).
 *   - Inputs and outputs must not overlap, except where stated (rope_bwd allows
 *     dx == dy).
 *   - Every tensor is dense and row-major in the layout given, with its base
 *     address 16-byte aligned, except where a token stride is stated: such a
 *     tensor [B][T][H][D] has dense rows of H * D elements whose starts are
 *     `stride` elements apart from token to token, over all B * T tokens (so
 *     it may be a part of a packed projection); stride 0 means H * D.
 *   - A non-OK status leaves the outputs unspecified; abw_last_error() returns
 *     a message for the last non-OK status of the calling thread.
 *   - Nothing crosses the ABI as a C++ exception, and nothing aborts.
 *   - Calls neither synchronise nor allocate: the work they enqueue on
 *     `stream` is kernel launches (and a memset or a copy of an output for
 *     rmsnorm_bwd_dgamma, and where no tokens are left to work on for
 *     qk_norm_rope_bwd and lin_attn_fwd / _bwd).  The first call of an operation on a device also resolves
 *     per-device state and raises the kernels' shared-memory limits.  So the
 *     calls can be captured into CUDA graphs; make one call of each operation
 *     on the device before capturing.
 *
 * Notation: B batch, Hq query heads, Hkv KV heads (Hq % Hkv == 0; query head
 * h reads KV head h / (Hq / Hkv)), D head dim, S KV length (decode), T
 * sequence length (causal), n row length.  bf16 tensors are IEEE bfloat16
 * (passed as `const void*`).
 */
#ifndef ATTN_BWD_H
#define ATTN_BWD_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ABW_OK = 0,
    ABW_EINVAL = 1,      /* a null pointer, a negative size, a misaligned pointer, overlap */
    ABW_ENOTSUP = 2,     /* valid but unsupported shape (e.g. head dim) */
    ABW_ECUDA = 3,       /* a CUDA launch or runtime error; message has the CUDA string */
    ABW_ETIMEOUT = 4,    /* a device-side bounded wait ran out (see abw_device_check) */
    ABW_EWORKSPACE = 5   /* workspace null or smaller than *_workspace_bytes() */
} abw_status;

typedef enum { ABW_F32 = 0, ABW_BF16 = 1 } abw_dtype;

/* Same type as cudaStream_t. */
typedef struct CUstream_st *abw_stream;

/* Message for the last non-OK status returned to this thread ("" if none). */
const char *abw_last_error(void);

/* ABI version (major * 100 + minor). */
int abw_version(void);

/* Synchronizes `stream`, then reads and clears the library's device error
 * word.  Returns ABW_ETIMEOUT if any kernel since the last check gave up on a
 * bounded wait (it then drained its own copies and returned instead of
 * hanging), ABW_ECUDA on a CUDA error, else ABW_OK. */
abw_status abw_device_check(abw_stream stream);

/* Sets the time limit, in nanoseconds, of every device-side wait of the
 * library's kernels (default 2e9, i.e. 2 s).  For tests.  With 0 the
 * tensor-core kernels of both attentions give up at their first product. */
void abw_set_wait_limit_ns(unsigned long long ns);

/* Launches one block that waits, with the library's bounded wait, on a
 * shared-memory barrier nothing ever arrives at.  The wait runs out after
 * `limit_ns`, the kernel records the timeout in the device error word and
 * returns, so abw_device_check() then reports ABW_ETIMEOUT.  Exercises the
 * failure path of the bounded waits without faulting or hanging the GPU. */
abw_status abw_selftest_wait_timeout(unsigned long long limit_ns, abw_stream stream);

/*
 * softmax_bwd -- softmaxBackward ("Hesper.Training.VerifiedBackward", section
 * Softmax): dx_i = s_i (dy_i - sum_j s_j dy_j), row by row.
 *   s   [rows][n] f32  probabilities (the softmax output saved by the forward)
 *   dy  [rows][n] f32  upstream gradient
 *   dx  [rows][n] f32  output
 * rows >= 0, n >= 1.
 */
abw_status softmax_bwd(const float *s, const float *dy, float *dx, int rows, int n,
                       abw_stream stream);

/*
 * rope_bwd -- ropeBackward (section RoPE): every rotary pair (y0, y1) of dy is
 * rotated by -theta: (y0 cos t + y1 sin t, -y0 sin t + y1 cos t).
 *   dy, dx [B][T][H][D] f32 (dx == dy allowed: in place)
 *   theta  [B*T][D/2] f32 explicit angles, or NULL: theta(b, t, i) =
 *          (pos0 + t) * base^(-2i/D) with the angle formed in double precision
 *   interleaved  1: pairs (2i, 2i+1);  0: pairs (i, i + D/2)
 * D even, 2 <= D <= 512; base > 0 when theta is NULL.
 */
abw_status rope_bwd(const float *dy, float *dx, int B, int T, int H, int D,
                    const float *theta, int pos0, float base, int interleaved,
                    abw_stream stream);

/*
 * rmsnorm_bwd -- rmsNormBackward (section RMSNorm), per row of length n:
 *   rms = sqrt(sum_j x_j^2 / n + eps),  c = sum_j dy_j g_j x_j,
 *   dx_i = (dy_i g_i - x_i c / (n rms^2)) / rms.
 *   x     [rows][n] f32 or bf16 (x_dtype)   the saved forward input
 *   gamma [n] f32
 *   dy    [rows][n] f32
 *   dx    [rows][n] f32 or bf16 (dx_dtype)
 * Both row sums are taken in one pass with fp32 accumulation.
 */
abw_status rmsnorm_bwd(const void *x, abw_dtype x_dtype, const float *gamma,
                       const float *dy, void *dx, abw_dtype dx_dtype, int rows, int n,
                       float eps, abw_stream stream);

/*
 * rmsnorm_bwd_dgamma -- rmsNormBackward (section RMSNorm) together with the
 * gradient of the norm's scale.  The page states dx only; the forward
 * y_i = gamma_i x_i / rms is linear in gamma, so its scale gradient is
 *   dgamma_i = sum over rows of dy_i x_i / rms.
 *   x, gamma, dy, dx as rmsnorm_bwd; dx may be NULL (then gamma may be NULL
 *   too, and only dgamma is produced)
 *   dgamma [n] f32, overwritten (the call zeroes it, then adds every row)
 * The row sums are fp32; the order in which the rows' terms are added into
 * dgamma varies from call to call (reductions in L2), so results agree to
 * fp32 rounding, not bit for bit.
 */
abw_status rmsnorm_bwd_dgamma(const void *x, abw_dtype x_dtype, const float *gamma, const float *dy,
                              void *dx, abw_dtype dx_dtype, float *dgamma, int rows, int n, float eps,
                              abw_stream stream);

/*
 * relu2_mul_bwd -- backward of the FFN's gated activation
 * hidden = ReLU(gate)^2 * up (Hesper pull request #1, the FFN-backward
 * commit's "ReLU^2 x Mul backward"), element by element:
 *   dgate = dh * up * 2 ReLU(gate),   dup = dh * ReLU(gate)^2.
 *   gate, up  [n] act_dtype (f32 or bf16)  saved forward activations
 *   dh        [n] f32                      upstream gradient of hidden
 *   dgate, dup [n] f32                     outputs
 * n >= 0 (any layout: the operation is element-wise).
 */
abw_status relu2_mul_bwd(const void *gate, const void *up, abw_dtype act_dtype, const float *dh,
                         float *dgate, float *dup, long long n, abw_stream stream);

/*
 * lora_bwd -- parameter gradients of a rank-r LoRA adapter on a projection
 * (Hesper pull request #1: the backward chain ends "RoPE backward -> dQ ->
 * LoRA backward", the adapter's input being the layer's saved normed
 * activations, and its input gradient feeds only dA and dB).  The adapter
 * adds y = scale * B (A x) per row; with h = x A^T:
 *   dB = scale dy^T h,   dA = (scale dy B)^T x      (sums over the rows)
 *   x   [rows][n_in] f32 or bf16 (x_dtype)   saved adapter input
 *   dy  [rows][n_out] f32                    gradient of the projection's output
 *                                            (e.g. dq as [tokens][Hq*D])
 *   A   [r][n_in] f32;   B [n_out][r] f32
 *   dA  [r][n_in] f32;   dB [n_out][r] f32   overwritten
 *   workspace  device memory of at least lora_bwd_workspace_bytes(rows, r)
 * Supported: 1 <= r <= 16; n_in and n_out multiples of 4.  Sums over rows are
 * fp32, added in an order that varies from call to call.
 */
size_t lora_bwd_workspace_bytes(int rows, int r);
abw_status lora_bwd(const void *x, abw_dtype x_dtype, const float *dy, const float *A, const float *B,
                    float *dA, float *dB, int rows, int n_in, int n_out, int r, float scale,
                    void *workspace, size_t workspace_bytes, abw_stream stream);

/*
 * attn_bwd_decode -- one query per sequence against a KV cache (attentionBackwardQ,
 * attentionBackwardV, scaledDotBackwardK of section Attention / Scaled Dot-Product),
 * with grouped KV heads:
 *   s_hj = scale q_h . K_j,  P_h = softmax_j(s_h),  dP_hj = dout_h . V_j,
 *   delta_h = sum_j P_hj dP_hj,  dS_hj = P_hj (dP_hj - delta_h),
 *   dq_h = scale sum_j dS_hj K_j        (then R(-theta(q_pos)) when RoPE is on)
 *   dK_j = scale sum_{h in group} dS_hj q_h,   dV_j = sum_{h in group} P_hj dout_h
 *   q, dout, dq [B][Hq][D] f32
 *   k, v        [B][S][Hkv][D] kv_dtype (f32 or bf16); dk, dv the same shape, f32
 *   rope_base > 0 and q_pos >= 0: RoPE backward at position q_pos on dq
 *   (pairs (2i, 2i+1), theta_i = q_pos base^(-2i/D)); otherwise none.
 * Supported: S >= 1; Hq % Hkv == 0 with Hq / Hkv <= 8; D even with
 * D * sizeof(kv) a multiple of 16 bytes and at most 512 bytes.
 */
abw_status attn_bwd_decode(const float *q, const void *k, const void *v, const float *dout,
                           float *dq, float *dk, float *dv,
                           int B, int Hq, int Hkv, int S, int D, abw_dtype kv_dtype,
                           float scale, float rope_base, int q_pos, abw_stream stream);

/*
 * attn_fwd_causal -- the causal attention forward that produces the
 * activations attn_bwd_causal consumes: online-softmax attention (Hesper
 * pull request #1, FlashAttention commits: flashAttentionSpec, equal to the
 * three-step standardAttention) under the causal mask (keys j <= query i):
 *   s_ij = scale q_i . k_j,  lse_i = log sum_{j<=i} exp(s_ij),
 *   o_i = sum_{j<=i} exp(s_ij - lse_i) v_j
 *   q [B][T][Hq][D] bf16;  k, v [B][T][Hkv][D] bf16 (query head h reads KV
 *   head h / (Hq / Hkv))
 *   o [B][T][Hq][D] bf16 (rounded from fp32);  lse [B][Hq][T] f32, natural log
 * The probabilities enter the o product rounded to bf16; sums are fp32.
 * Supported: D == 128; T >= 1; Hq % Hkv == 0.
 */
abw_status attn_fwd_causal(const void *q, const void *k, const void *v, void *o, float *lse,
                           int B, int T, int Hq, int Hkv, int D, float scale, abw_stream stream);

/*
 * attn_bwd_causal_workspace_bytes -- workspace size attn_bwd_causal needs for
 * these sizes, with Tp = T rounded up to 128 and nb = Tp / 128: delta and
 * lse * log2(e), each f32 [B][Hq][Tp]; the RoPE table [T][D/2] of
 * scale * (cos, sin); the bf16 dS tiles of the causal half, 16 KB per
 * (128-key block, 64-query block) pair, B * Hq * (nb^2 + nb) of them; and
 * 256-byte alignment slack.  About B * Hq * Tp * (Tp + 136) bytes.
 */
size_t attn_bwd_causal_workspace_bytes(int B, int T, int Hq, int D);

/*
 * attn_bwd_causal -- causal multi-query attention backward (keys j <= query i).
 * The probabilities are recomputed from the saved log-sum-exp:
 *   P_ij = exp(scale q_i . k_j - lse_i) for j <= i, else 0,
 *   dP = dout V^T,  delta_i = dout_i . o_i (= sum_j P_ij dP_ij),
 *   dS = P (dP - delta),  dq = scale dS K,  dk = scale dS^T Q,  dv = P^T dout,
 * dk and dv summed over the query heads that share a KV head.  With
 * rope_base > 0, RoPE backward R(-theta(pos0 + t)) (pairs (2i, 2i+1),
 * theta_i = (pos0 + t) base^(-2i/D)) is applied to dq and dk.
 *   q, o, dout [B][T][Hq][D] bf16;   k, v [B][T][Hkv][D] bf16
 *   lse        [B][Hq][T] f32 natural-log log-sum-exp of the scaled scores
 *   dq [B][T][Hq][D] f32;  dk, dv [B][T][Hkv][D] f32
 *   workspace  device memory of at least attn_bwd_causal_workspace_bytes()
 * Supported: D == 128; T >= 1; Hq % Hkv == 0.
 */
abw_status attn_bwd_causal(const void *q, const void *k, const void *v, const void *o,
                           const void *dout, const float *lse,
                           float *dq, float *dk, float *dv,
                           int B, int T, int Hq, int Hkv, int D, float scale,
                           float rope_base, int pos0,
                           void *workspace, size_t workspace_bytes, abw_stream stream);

/*
 * attn_bwd_causal_saved_p -- attn_bwd_causal reading the attention weights
 * the forward saved instead of recomputing them from the log-sum-exp: the
 * form of Hesper pull request #1's softmax-backward fix ("save per-layer
 * attention weights ... use saved attnBuf": dScores = attn (dAttn -
 * sum attn dAttn)) and of transformer.js backward(), which reads the cached
 * attention A.
 *   p_attn [B][Hq][T][T] bf16  the softmax output, row = query i, column =
 *          key j; entries with j > i are not read (the causal mask makes
 *          them 0)
 *   o      [B][T][Hq][D] bf16  the forward's output, for
 *          delta_i = sum_j P_ij dP_ij = dout_i . o_i (the identity holds
 *          because o = P v)
 *   everything else as attn_bwd_causal (no lse), with the same workspace
 *   size (attn_bwd_causal_workspace_bytes).
 */
abw_status attn_bwd_causal_saved_p(const void *q, const void *k, const void *v, const void *p_attn,
                                   const void *o, const void *dout, float *dq, float *dk, float *dv,
                                   int B, int T, int Hq, int Hkv, int D, float scale,
                                   float rope_base, int pos0, void *workspace, size_t workspace_bytes,
                                   abw_stream stream);

/*
 * attn_bwd_causal_noalloc -- attn_bwd_causal for callers that cannot allocate
 * device memory: no workspace argument, and the call allocates nothing.  (The
 * pages have no counterpart; this is an interface convenience.)
 *
 * Who needs it: code that runs where cudaMalloc is off limits -- inside a
 * CUDA stream capture or a custom allocator's callback, in a process whose
 * device memory is owned by another framework's pool, or in a plugin given
 * only the tensors it works on.  Such a caller passes the inputs and outputs
 * as for attn_bwd_causal; the scratch comes from a 32 MiB array in the
 * library's device image (a file-scope __device__ variable), which every GPU
 * that loads the library keeps until the process exits.
 *
 *   Arguments, layouts and results: as attn_bwd_causal.
 *   Limit: the sizes must need at most 32 MiB of scratch
 *   (attn_bwd_causal_workspace_bytes(B, T, Hq, D) <= 33554432, roughly
 *   B * Hq * T^2 < 32 MiB, e.g. B=2, T=512, Hq=20 needs about 13 MB); larger
 *   sizes return ABW_EWORKSPACE without launching anything.
 *   First call on a device: looks up the array's device address on that
 *   device (cudaGetSymbolAddress) and caches it; make that first call before
 *   any stream capture that should contain it.
 *   Sharing: every call on a device uses the same array.  Each call writes
 *   every part of it that it later reads, so consecutive calls are
 *   independent -- but calls that overlap on the GPU (different streams, no
 *   ordering between them) race on the array.
 */
abw_status attn_bwd_causal_noalloc(const void *q, const void *k, const void *v, const void *o,
                                   const void *dout, const float *lse,
                                   float *dq, float *dk, float *dv,
                                   int B, int T, int Hq, int Hkv, int D, float scale,
                                   float rope_base, int pos0, abw_stream stream);

/*
 * qk_norm_rope_fwd -- what stands between the projections and an attention:
 * per head row x of D components, of queries and keys,
 *   rms = sqrt(sum_j x_j^2 / D + eps),  n_i = x_i gamma_i / rms,  y = R(theta) n,
 * where R turns the pairs of the first rotary_dim components,
 * (n0 cos t - n1 sin t, n0 sin t + n1 cos t), and leaves the others.
 *   q [B][T][Hq][D], k [B][T][Hkv][D] dtype (f32 or bf16), token strides
 *         q_stride, k_stride; Hkv == 0 (or Hq == 0): no keys (no queries)
 *   gamma_q, gamma_k [D] f32, or NULL: no norm (the rotation alone)
 *   q_out, k_out  dense, same dtype; computed in fp32 and rounded once
 *   rope_base > 0: theta_i = pos rope_base^(-2i / rotary_dim); rope_base 0:
 *         no rotation (rotary_dim, positions and sections are not looked at)
 *   rotary_dim    even, 2 .. D
 *   interleaved   1: pairs (2i, 2i+1);  0: pairs (i, i + rotary_dim / 2)
 *   positions     [n_axes][B][T] int32 (any value, negative ones included), or
 *         NULL: pos = pos0 + t on every axis
 *   n_axes, sections   1 <= n_axes <= 4; sections is a HOST array of n_axes
 *         counts >= 0 that add up to rotary_dim / 2: the first sections[0]
 *         pairs turn by the position on axis 0, the next sections[1] by that on
 *         axis 1, and so on (time, height and width of image and video
 *         tokens).  NULL with n_axes == 1.
 * The angle of a pair is off by at most |pos| 2^-54 + 2^-31 turns where rope_base
 * >= 1 (2^-23 turns at the farthest position), and by (4 + |ln rope_base|) 2^-53
 * of itself + 2^-31 turns below.  rope_base is the fp32 number given; the
 * exponents run through the pairs of all axes.  eps >= 0.  The sum of squares is
 * taken in fp32: a row that holds values above 1e18, or with eps 0 one of zeros or
 * of nothing above 1e-19, may come out as NaN or infinite.
 * Supported: D even, 2 <= D <= 512; below 2^31 elements a token.
 */
abw_status qk_norm_rope_fwd(const void *q, const void *k, abw_dtype dtype, const float *gamma_q,
                            const float *gamma_k, void *q_out, void *k_out, int B, int T, int Hq, int Hkv, int D,
                            long long q_stride, long long k_stride, float eps, float rope_base, int rotary_dim,
                            int interleaved, const int *positions, int n_axes, const int *sections, int pos0,
                            abw_stream stream);

/*
 * qk_norm_rope_bwd -- gradients of qk_norm_rope_fwd: with dn = R(-theta) dy and
 * c = sum_j dn_j gamma_j x_j,
 *   dx_i = (dn_i gamma_i - x_i c / (D rms^2)) / rms,
 *   dgamma_i = sum over tokens and heads of dn_i x_i / rms   (without a norm dx = dn).
 *   q, k (and strides), gamma_q, gamma_k, the rotation: as in the forward
 *   dq_out, dk_out  dense [B][T][Hq][D], [B][T][Hkv][D] dy_dtype (f32 as the
 *         softmax attention's gradients, or bf16 as the linear attention's)
 *   dq, dk        dtype, token strides dq_stride, dk_stride (so they may be parts
 *         of a packed gradient); must not overlap q, k
 *   dgamma_q, dgamma_k [D] f32, overwritten; each NULL where it is not wanted
 *         or its gamma is NULL
 *   workspace     at least qk_norm_rope_bwd_workspace_bytes(D) where a gamma is
 *         given, else it may be NULL
 * Sums are fp32 in a fixed order: equal calls on a device give equal bits.
 */
size_t qk_norm_rope_bwd_workspace_bytes(int D);
abw_status qk_norm_rope_bwd(const void *q, const void *k, abw_dtype dtype, const void *dq_out, const void *dk_out,
                            abw_dtype dy_dtype, const float *gamma_q, const float *gamma_k, void *dq, void *dk,
                            float *dgamma_q, float *dgamma_k, int B, int T, int Hq, int Hkv, int D,
                            long long q_stride, long long k_stride, long long dq_stride, long long dk_stride,
                            float eps, float rope_base, int rotary_dim, int interleaved, const int *positions,
                            int n_axes, const int *sections, int pos0, void *workspace, size_t workspace_bytes,
                            abw_stream stream);

/*
 * lin_attn_fwd -- causal linear attention with a decay for each KV head: with
 * a = exp(log_decay) of the head and its state S [D][D] (key component, value
 * component),
 *   S_t = a S_(t-1) + k_t v_t^T,   o_t = scale S_t^T q_t,
 * evaluated over chunks of 128 tokens on the tensor core.
 *   q [B][T][Hq][D], k, v [B][T][Hkv][D] bf16, token strides q_stride, k_stride,
 *         v_stride; query head h reads KV head h / (Hq / Hkv)
 *   log_decay     [Hkv] f32, <= 0 (0: no decay; -inf: only the token itself).  A
 *         constant of the model: it has no gradient
 *   initial_state [B][Hkv][D][D] f32 or NULL (zero)
 *   lengths       [B] int32 or NULL: sequence b has min(max(lengths[b], 0), T)
 *         tokens; what q, k, v hold behind them is not looked at (NaN included)
 *         and o there is written as 0.  Inside a sequence values are finite: an
 *         infinity or NaN of a token reaches all outputs of its 128-token chunk,
 *         those of earlier tokens too (a weight of 0 does not hold it back)
 *   o             [B][T][Hq][D] bf16, token stride o_stride
 *   final_state   [B][Hkv][D][D] f32 or NULL: the state behind each sequence's last
 *         token (may be the same buffer as initial_state)
 *   workspace     at least lin_attn_fwd_workspace_bytes() (also for short
 *         sequences without states, which leave it alone); unspecified contents
 * Scores and the chunk states that enter a product are rounded to bf16; sums
 * and the states themselves are fp32.  final_state is good to some 40 2^-23 of
 * its 2-norm, also where a head hardly decays (measured: 2e-7 after some hundred
 * tokens, 8e-7 after 100,000).  Equal calls give equal bits.
 * Supported: D == 64 or 128; T >= 0; Hq >= 1, Hq % Hkv == 0; strides multiples
 * of 8.
 */
size_t lin_attn_fwd_workspace_bytes(int B, int T, int Hkv, int D);
abw_status lin_attn_fwd(const void *q, const void *k, const void *v, const float *log_decay,
                        const float *initial_state, const int *lengths, void *o, float *final_state, int B, int T,
                        int Hq, int Hkv, int D, long long q_stride, long long k_stride, long long v_stride,
                        long long o_stride, float scale, void *workspace, size_t workspace_bytes,
                        abw_stream stream);

/*
 * lin_attn_bwd -- gradients of lin_attn_fwd.  With R_t the gradient of S_t,
 *   R_t = a R_(t+1) + scale q_t do_t^T (summed over the query heads of the group),
 *   dq_t = scale S_t do_t,   dk_t = R_t v_t,   dv_t = R_t^T k_t,
 *   dinitial_state = a R_1,   R behind the last token = dfinal_state.
 * The forward's states are formed again; nothing is saved by the forward.
 *   q, k, v, log_decay, initial_state, lengths: as in the forward
 *   dout          dense [B][T][Hq][D] bf16
 *   dfinal_state  [B][Hkv][D][D] f32 or NULL (zero)
 *   dq, dk, dv    bf16, token strides dq_stride, dk_stride, dv_stride; 0 behind
 *         each sequence's last token
 *   dinitial_state [B][Hkv][D][D] f32 or NULL (may be the same buffer as
 *         dfinal_state)
 *   workspace     at least lin_attn_bwd_workspace_bytes()
 * Supported sizes and precision: as in the forward.
 */
size_t lin_attn_bwd_workspace_bytes(int B, int T, int Hkv, int D);
abw_status lin_attn_bwd(const void *q, const void *k, const void *v, const void *dout, const float *log_decay,
                        const float *initial_state, const float *dfinal_state, const int *lengths, void *dq, void *dk,
                        void *dv, float *dinitial_state, int B, int T, int Hq, int Hkv, int D, long long q_stride,
                        long long k_stride, long long v_stride, long long dq_stride, long long dk_stride,
                        long long dv_stride, float scale, void *workspace, size_t workspace_bytes,
                        abw_stream stream);

/*
 * lin_attn_decode -- one token per sequence: the recurrence of lin_attn_fwd,
 *   S = a S + k v^T (in place),   o = scale S^T q.
 *   q [B][Hq][D], k, v [B][Hkv][D], o [B][Hq][D] dtype (f32 or bf16)
 *   state         [n_states][Hkv][D][D] f32, read and written
 *   log_decay     [Hkv] f32, <= 0; 1 - a is good to fp32, so heads that hardly decay
 *         keep their pace over many tokens
 *   slots         [B] int32 or NULL (then n_states >= B and row b works on state
 *         b): row b works on state slots[b].  A row whose slot is not in
 *         0 .. n_states - 1 is empty: o is 0 there and no state is touched.  Two rows
 *         of a call must not name the same state
 * Supported: D == 64 or 128; Hq % Hkv == 0 with Hq / Hkv <= 8.
 */
abw_status lin_attn_decode(const void *q, const void *k, const void *v, abw_dtype dtype, float *state,
                           const float *log_decay, const int *slots, void *o, int B, int Hq, int Hkv, int D,
                           int n_states, float scale, abw_stream stream);

/*
 * attn_fwd_window -- causal softmax attention over a sliding window with first
 * tokens that stay visible (sinks): query i sees key j where
 *   j <= i  and  (j > i - window  or  j < sinks),
 *   s_ij = scale q_i . k_j,  lse_i = log sum_j exp(s_ij),  o_i = sum_j exp(s_ij - lse_i) v_j.
 *   q [B][T][Hq][D], k, v [B][T][Hkv][D] bf16, token strides q_stride, k_stride,
 *         v_stride; query head h reads KV head h / (Hq / Hkv)
 *   lengths       [B] int32 or NULL: sequence b has min(max(lengths[b], 0), T)
 *         tokens; what q, k, v hold behind them is not looked at (NaN included), o
 *         there is written as 0 and lse as -infinity.  Inside a sequence values are
 *         finite: an infinity or NaN of a token may reach every query whose
 *         128-token block meets the token's (a weight of 0 does not hold it back)
 *   o             [B][T][Hq][D] bf16, token stride o_stride (rounded from fp32)
 *   lse           [B][Hq][T] f32, natural log
 *   window        >= 1 (1: the token itself; T and more: plain causal attention)
 *   sinks         >= 0
 * The probabilities enter the o product rounded to bf16; sums are fp32.  Equal
 * calls give equal bits.
 * Supported: D == 64 or 128; T >= 0; Hq >= 1, Hq % Hkv == 0; strides multiples
 * of 8.
 */
abw_status attn_fwd_window(const void *q, const void *k, const void *v, const int *lengths, void *o, float *lse,
                           int B, int T, int Hq, int Hkv, int D, long long q_stride, long long k_stride,
                           long long v_stride, long long o_stride, int window, int sinks, float scale,
                           abw_stream stream);

/*
 * attn_bwd_window -- gradients of attn_fwd_window from its o and lse:
 *   P_ij = exp(s_ij - lse_i) where key j is visible to query i, else 0,
 *   delta_i = dout_i . o_i,  dS = P (dout V^T - delta),
 *   dq = scale dS K,  dk = scale dS^T Q,  dv = P^T dout,
 * dk and dv summed over the query heads that share a KV head.
 *   q, k, v, lengths, window, sinks, scale: as in the forward
 *   o             as the forward wrote it, token stride o_stride
 *   dout          dense [B][T][Hq][D] bf16
 *   lse           [B][Hq][T] f32
 *   dq, dk, dv    bf16, token strides dq_stride, dk_stride, dv_stride (so they may
 *         be parts of a packed gradient); 0 behind each sequence's last token
 *   workspace     at least attn_bwd_window_workspace_bytes(): 32 KB for each query head
 *         and pair of 128-token blocks that meet (T (min(window, T) + 256) / 16384 pairs
 *         and less, and T / 128 for each 128 of the first tokens), of as many (sequence,
 *         KV head)s as fit 2 GiB, one at least, which the call goes through in turn; with
 *         8 bytes a query head and token, and sums of up to some 100 MB
 * P and dS enter their products rounded to bf16; sums are fp32 in a fixed order:
 * equal calls on a device give equal bits.
 * Supported sizes: as in the forward.
 */
size_t attn_bwd_window_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int window, int sinks);
abw_status attn_bwd_window(const void *q, const void *k, const void *v, const void *o, const void *dout,
                           const float *lse, const int *lengths, void *dq, void *dk, void *dv, int B, int T, int Hq,
                           int Hkv, int D, long long q_stride, long long k_stride, long long v_stride,
                           long long o_stride, long long dq_stride, long long dk_stride, long long dv_stride,
                           int window, int sinks, float scale, void *workspace, size_t workspace_bytes,
                           abw_stream stream);

/*
 * The paged cache of the three calls below: k_pages, v_pages
 * [n_pages][page_size][Hkv][D] bf16, and a block_table [B][max_pages] int32 that
 * gives position p of sequence b row p % page_size of page
 * block_table[b][p / page_size].  An entry outside 0 .. n_pages - 1 is an absent
 * page: its tokens are neither read nor written.  (A dense cache [B][S][Hkv][D]
 * is one of B pages of S rows.)  Any page_size >= 1 with page_size * max_pages
 * at most 2^31 - 2^16.
 */

/*
 * kv_pages_write -- puts the keys and values of new tokens into their pages:
 * token t of sequence b, t < min(max(lengths[b], 0), T), goes to position
 * starts[b] + t.  Positions below 0, at page_size * max_pages or above, and those
 * of absent pages are left out.
 *   k, v          [B][T][Hkv][D] bf16, token strides k_stride, v_stride
 *   starts        [B] int32;  lengths [B] int32 or NULL (T tokens each)
 * Two tokens of a call must not name the same row of a page.
 * Supported: D a multiple of 8; strides multiples of 8.
 */
abw_status kv_pages_write(const void *k, const void *v, void *k_pages, void *v_pages, const int *block_table,
                          const int *starts, const int *lengths, int B, int T, int Hkv, int D, int n_pages,
                          int page_size, int max_pages, long long k_stride, long long v_stride, abw_stream stream);

/*
 * attn_decode_paged -- one new token per sequence over the paged cache, which
 * holds its key and value already: with n = min(max(lengths[b], 0), page_size *
 * max_pages) the query of row b stands at position n - 1 and sees the positions
 *   j < n  with  (window == 0  or  j >= n - window  or  j < sinks)
 * of present pages:
 *   s_j = scale q . k_j,  p_j = exp(s_j) / sum exp(s),  o = sum_j p_j v_j.
 * A row that sees nothing (length 0, no page) gives o = 0.
 *   q, o          [B][Hq][D] dtype (f32 or bf16); query head h reads KV head
 *         h / (Hq / Hkv)
 *   lengths       [B] int32
 *   weight_sums   [B][Hkv][page_size * max_pages] f32 or NULL: every visible
 *         position's entry has the sum of its p_j over the query heads of the KV
 *         head added; the others are left as they are
 *   window        >= 0 (0: none);  sinks >= 0 (not looked at without a window)
 *   workspace     at least attn_decode_paged_workspace_bytes(); unspecified
 *         contents.  Some MB (the pieces of 304 CTAs), with weight_sums and 4 bytes for each
 *         row, query head and position that the table has room for (with a window:
 *         at most window + sinks), whatever the lengths
 * The cache is read once, in pieces of equal length over all sequences whatever
 * their lengths, and the pieces are joined.  q and p enter the products as sums of
 * bf16 terms that keep 16 bits of them and more, sums are fp32.  Values of visible
 * positions are finite; what others hold is not looked at.  Equal calls on a
 * device give equal bits.
 * Supported: D == 64 or 128; Hq % Hkv == 0.
 */
size_t attn_decode_paged_workspace_bytes(int B, int Hq, int Hkv, int D, int page_size, int max_pages, int window,
                                         int sinks, int with_weight_sums);
abw_status attn_decode_paged(const void *q, abw_dtype dtype, const void *k_pages, const void *v_pages,
                             const int *block_table, const int *lengths, float *weight_sums, void *o, int B, int Hq,
                             int Hkv, int D, int n_pages, int page_size, int max_pages, int window, int sinks,
                             float scale, void *workspace, size_t workspace_bytes, abw_stream stream);

/*
 * kv_pages_evict -- keeps, for each sequence and KV head, at most `budget` tokens
 * of the cache: those at positions below `sinks`, the last `recent` positions,
 * and of the others those of the largest weight_sums (ties: the lower position; a
 * NaN counts as -infinity).  Tokens of absent pages are not kept.  Only
 * attn_decode_paged adds to the sums: right behind a prompt they are what the
 * caller put there, and of equal ones (all 0) the lowest positions stay.  The kept
 * ones go, in their order, to positions 0, 1, .. of the pages that new_table names
 * (the old pages stay as they are: they may be shared with other sequences).
 *   k_pages, v_pages  read in the pages of block_table, written in those of
 *         new_table [B][new_max_pages] int32; no page may be named by both, nor
 *         twice by new_table.  A row of an absent new page is not written
 *   lengths       [B] int32, as for attn_decode_paged
 *   weight_sums   [B][Hkv][page_size * max_pages] f32
 *   kept          [B][Hkv][budget] int32: the positions kept, ascending, -1 behind
 *         the last one
 *   new_lengths   [B] int32: the tokens kept, min(budget, present ones)
 *   new_weight_sums [B][Hkv][page_size * new_max_pages] f32: the kept tokens'
 *         sums, 0 behind the last one
 *   budget >= 1, sinks >= 0, recent >= 0, sinks + recent <= budget <= page_size *
 *         new_max_pages
 * Supported: D a multiple of 8.
 */
abw_status kv_pages_evict(void *k_pages, void *v_pages, const int *block_table, const int *lengths,
                          const float *weight_sums, const int *new_table, int *kept, int *new_lengths,
                          float *new_weight_sums, int B, int Hkv, int D, int n_pages, int page_size, int max_pages,
                          int new_max_pages, int budget, int sinks, int recent, abw_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_BWD_H */
