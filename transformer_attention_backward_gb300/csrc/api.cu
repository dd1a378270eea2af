// The C ABI: argument validation, status codes, the per-thread error message,
// the device error word, and the TMA descriptor encoder.  Every compute step
// runs in the kernels of the other translation units.
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "../../include/attn_bwd.h"
#include "abw_host.h"

namespace {

thread_local std::string g_last_error;
std::atomic<unsigned long long> g_wait_limit_ns{2000000000ull};

// The device error word.  Kernels receive its device address (resolved per
// device with cudaGetSymbolAddress) and atomically OR failure bits into it.
__device__ unsigned int g_abw_err_word[2];   // bits, first timeout site

constexpr int kMaxDevices = 64;
std::mutex g_dev_mu;
unsigned int *g_err_addr[kMaxDevices] = {};
unsigned long long g_err_ctx[kMaxDevices] = {};   // context the cached address belongs to

abw_status fail(abw_status st, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

abw_status from_cuda(cudaError_t e, const char *what, const char *why = nullptr) {
  if (e == cudaSuccess) return ABW_OK;
  if (e == cudaErrorNotSupported) return fail(ABW_ENOTSUP, "%s: %s", what, why ? why : "unsupported shape");
  return fail(ABW_ECUDA, "%s: %s (%s)%s%s", what, cudaGetErrorString(e), cudaGetErrorName(e),
              why ? ": " : "", why ? why : "");
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
  const char *name;
  const void *p;
  size_t bytes;
};

bool overlaps(const Range &a, const Range &b) {
  if (a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Null / alignment checks for every buffer, and no output overlapping any
// other buffer.
abw_status check_buffers(const char *op, const Range *in, int nin, const Range *out, int nout) {
  for (int i = 0; i < nin + nout; ++i) {
    const Range &r = i < nin ? in[i] : out[i - nin];
    if (r.bytes == 0) continue;
    if (r.p == nullptr) return fail(ABW_EINVAL, "%s: %s is NULL", op, r.name);
    if (!aligned16(r.p)) return fail(ABW_EINVAL, "%s: %s is not 16-byte aligned", op, r.name);
  }
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlaps(out[i], in[j]))
        return fail(ABW_EINVAL, "%s: output %s overlaps input %s", op, out[i].name, in[j].name);
    for (int j = i + 1; j < nout; ++j)
      if (overlaps(out[i], out[j]))
        return fail(ABW_EINVAL, "%s: outputs %s and %s overlap", op, out[i].name, out[j].name);
  }
  return ABW_OK;
}

// A buffer with a token stride: `n` rows of `row` bytes, `stride` bytes apart.
struct Rows {
  const char *name;
  const void *p;
  size_t n, row, stride, align;
  size_t bytes() const { return n == 0 || row == 0 ? 0 : (n - 1) * stride + row; }
};

// Rows of one packed buffer interleave: with a common stride two of them
// overlap only if their rows do.
bool overlaps(const Rows &a, const Rows &b) {
  if (!overlaps(Range{a.name, a.p, a.bytes()}, Range{b.name, b.p, b.bytes()})) return false;
  if (a.stride != b.stride || a.row > a.stride || b.row > b.stride) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const size_t d = x >= y ? (x - y) % a.stride : (a.stride - (y - x) % a.stride) % a.stride;   // a behind b's row start
  return d < b.row || a.stride - d < a.row;
}

abw_status check_rows(const char *op, const Rows *in, int nin, const Rows *out, int nout) {
  for (int i = 0; i < nin + nout; ++i) {
    const Rows &r = i < nin ? in[i] : out[i - nin];
    if (r.bytes() == 0) continue;
    if (r.p == nullptr) return fail(ABW_EINVAL, "%s: %s is NULL", op, r.name);
    if (reinterpret_cast<uintptr_t>(r.p) % r.align != 0)
      return fail(ABW_EINVAL, "%s: %s is not %zu-byte aligned", op, r.name, r.align);
    if (r.n > 1 && r.stride < r.row) return fail(ABW_EINVAL, "%s: %s has a token stride below its row", op, r.name);
    if (r.n > 1 && r.stride % r.align != 0)
      return fail(ABW_ENOTSUP, "%s: %s has a token stride of %zu bytes, not a multiple of %zu", op, r.name, r.stride,
                  r.align);
  }
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlaps(out[i], in[j]))
        return fail(ABW_EINVAL, "%s: output %s overlaps input %s", op, out[i].name, in[j].name);
    for (int j = i + 1; j < nout; ++j)
      if (overlaps(out[i], out[j]))
        return fail(ABW_EINVAL, "%s: outputs %s and %s overlap", op, out[i].name, out[j].name);
  }
  return ABW_OK;
}

Rows dense(const char *name, const void *p, size_t bytes, size_t align = 16) {
  return Rows{name, p, bytes ? 1u : 0u, bytes, bytes, align};
}

// Argument checks that the linear attention's entry points share.
abw_status check_lin(const char *op, int B, int T, int Hq, int Hkv, int D, float scale) {
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0) return fail(ABW_EINVAL, "%s: negative size", op);
  if (Hkv == 0 || Hq % Hkv != 0) return fail(ABW_EINVAL, "%s: Hq=%d not a multiple of Hkv=%d", op, Hq, Hkv);
  if (Hq == 0) return fail(ABW_EINVAL, "%s: Hq=0 with Hkv=%d", op, Hkv);
  if (D != 64 && D != 128) return fail(ABW_ENOTSUP, "%s: D=%d unsupported (D == 64 or 128)", op, D);
  if (!(scale == scale)) return fail(ABW_EINVAL, "%s: scale is NaN", op);
  return ABW_OK;
}

Rows lin_rows(const char *name, const void *p, int B, int T, int H, int D, long long stride) {
  const size_t row = static_cast<size_t>(H) * D * 2;
  return Rows{name, p, static_cast<size_t>(B) * T, row, stride == 0 ? row : static_cast<size_t>(stride) * 2, 16};
}

// Elements from token to token; a single token has no next one.
long long token_stride(long long stride, int B, int T, long long row) {
  return stride == 0 || static_cast<long long>(B) * T <= 1 ? row : stride;
}

// The rotation's arguments as both directions of qk_norm_rope take them.
abw_status check_rotation(const char *op, abw::QkNormRopeArgs &a, float rope_base, int rotary_dim, int interleaved,
                          const int *positions, int n_axes, const int *sections, int pos0) {
  a.base = 1.0;
  a.rotary_dim = 0;
  a.interleaved = interleaved ? 1 : 0;
  a.positions = nullptr;
  a.n_axes = 1;
  a.pos0 = pos0;
  if (!(rope_base >= 0.0f)) return fail(ABW_EINVAL, "%s: rope_base must be >= 0 (0: no rotation)", op);
  if (rope_base == 0.0f) return ABW_OK;
  if (rope_base > 3.0e38f) return fail(ABW_EINVAL, "%s: rope_base is not finite", op);
  if (rotary_dim < 2 || (rotary_dim & 1) || rotary_dim > a.D)
    return fail(ABW_EINVAL, "%s: rotary_dim=%d must be even, 2 .. D=%d", op, rotary_dim, a.D);
  if (n_axes < 1 || n_axes > 4) return fail(ABW_EINVAL, "%s: n_axes=%d (1 .. 4)", op, n_axes);
  if (sections == nullptr && n_axes > 1) return fail(ABW_EINVAL, "%s: sections is NULL with n_axes=%d", op, n_axes);
  long long sum = 0;
  for (int i = 0; i < n_axes; ++i) {
    a.sections[i] = sections ? sections[i] : rotary_dim / 2;
    if (a.sections[i] < 0) return fail(ABW_EINVAL, "%s: sections[%d]=%d is negative", op, i, a.sections[i]);
    sum += a.sections[i];
  }
  if (sum != rotary_dim / 2)
    return fail(ABW_EINVAL, "%s: sections add up to %lld, not to rotary_dim / 2 = %d", op, sum, rotary_dim / 2);
  a.base = static_cast<double>(rope_base);
  a.rotary_dim = rotary_dim;
  a.positions = positions;
  a.n_axes = n_axes;
  return ABW_OK;
}

abw_status check_qk(const char *op, int B, int T, int Hq, int Hkv, int D, abw_dtype dtype, float eps) {
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0) return fail(ABW_EINVAL, "%s: negative size", op);
  if (D < 2 || (D & 1)) return fail(ABW_EINVAL, "%s: D=%d must be even and >= 2", op, D);
  if (D > 512) return fail(ABW_ENOTSUP, "%s: D=%d > 512", op, D);
  if (static_cast<long long>(Hq > Hkv ? Hq : Hkv) * D > 0x7fffffff)
    return fail(ABW_ENOTSUP, "%s: more than 2^31 elements a token", op);
  if (dtype != ABW_F32 && dtype != ABW_BF16) return fail(ABW_EINVAL, "%s: bad dtype", op);
  if (!(eps >= 0.0f)) return fail(ABW_EINVAL, "%s: eps must be >= 0", op);
  return ABW_OK;
}

size_t dt_size(abw_dtype d) { return d == ABW_BF16 ? 2 : 4; }

}  // namespace

namespace abw {

unsigned long long context_id() {
  // cuCtxGetCurrent / cuCtxGetId through the runtime's driver entry points
  // (no link against libcuda).  The id is unique for the life of the
  // process, so a context created after cudaDeviceReset never matches a
  // cached entry of the one it replaced, even at the same handle address.
  using GetCur = CUresult (*)(CUcontext *);
  using GetId = CUresult (*)(CUcontext, unsigned long long *);
  static GetCur get_cur = nullptr;
  static GetId get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_cur = reinterpret_cast<GetCur>(p);
    p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<GetId>(p);
  });
  CUcontext c = nullptr;
  unsigned long long id = 0;
  if (!get_cur || !get_id || get_cur(&c) != CUDA_SUCCESS || c == nullptr || get_id(c, &id) != CUDA_SUCCESS)
    return 0;
  return id;
}

cudaError_t ensure_dynamic_smem(const void *func, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long ctx = context_id();
  struct Entry {
    const void *func;
    int dev, bytes;
    unsigned long long ctx;
  };
  static std::mutex mu;
  static Entry seen[64];
  static int nseen = 0;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < nseen; ++i) {
    if (seen[i].func != func || seen[i].dev != dev) continue;
    if (ctx != 0 && seen[i].ctx == ctx && seen[i].bytes >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) {
      seen[i].bytes = bytes;
      seen[i].ctx = ctx;
    }
    return e;
  }
  e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && nseen < 64) seen[nseen++] = Entry{func, dev, bytes, ctx};
  return e;
}

WaitCtl wait_ctl() {
  WaitCtl w{nullptr, g_wait_limit_ns.load()};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return w;
  const unsigned long long ctx = context_id();
  std::lock_guard<std::mutex> lk(g_dev_mu);
  if (g_err_addr[dev] == nullptr || ctx == 0 || g_err_ctx[dev] != ctx) {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_abw_err_word) != cudaSuccess) return w;
    g_err_addr[dev] = static_cast<unsigned int *>(p);
    g_err_ctx[dev] = ctx;
  }
  w.err = g_err_addr[dev];
  return w;
}

bool encode_tiled(CUtensorMap *map, CUtensorMapDataType dt, uint32_t rank, const void *base,
                  const uint64_t *dims, const uint64_t *strides_bytes, const uint32_t *box,
                  CUtensorMapSwizzle swizzle, const char **why) {
  using Fn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                          const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                          CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Fn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<Fn>(p);
  });
  if (!fn) {
    if (why) *why = "cuTensorMapEncodeTiled unavailable";
    return false;
  }
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(map, dt, rank, const_cast<void *>(base), dims, strides_bytes, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    if (why) *why = "cuTensorMapEncodeTiled failed";
    return false;
  }
  return true;
}

bool move_tiled(CUtensorMap *map, const void *base) {
  using Fn = CUresult (*)(CUtensorMap *, void *);
  static Fn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapReplaceAddress", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<Fn>(p);
  });
  return fn && fn(map, const_cast<void *>(base)) == CUDA_SUCCESS;
}

}  // namespace abw

// ============================================================================
// extern "C" entry points
// ============================================================================
extern "C" {

const char *abw_last_error(void) { return g_last_error.c_str(); }

int abw_version(void) { return 100; }

void abw_set_wait_limit_ns(unsigned long long ns) { g_wait_limit_ns.store(ns); }

abw_status abw_device_check(abw_stream stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return from_cuda(e, "abw_device_check");
  abw::WaitCtl w = abw::wait_ctl();
  if (!w.err) return fail(ABW_ECUDA, "abw_device_check: device error word unavailable");
  unsigned int words[2] = {0, 0};
  e = cudaMemcpyAsync(words, w.err, sizeof(words), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(w.err, 0, sizeof(words), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return from_cuda(e, "abw_device_check");
  const unsigned int word = words[0], site = words[1];
  if (word & (abw::kErrWaitTimeout | abw::kErrSelfTest)) {
    const abw::WaitSite s = abw::unpack_site(site);
    return fail(ABW_ETIMEOUT,
                "a device-side bounded wait ran out (error word 0x%x; first in the %s kernel, barrier slot %u, "
                "warp %u, block %u)",
                word, abw::site_kernel(s.kernel), s.slot, s.warp, s.block);
  }
  if (word & abw::kErrSmemAlign)
    return fail(ABW_ECUDA, "a kernel's dynamic shared memory was not 1024-byte aligned; it did no work");
  return ABW_OK;
}

abw_status abw_selftest_wait_timeout(unsigned long long limit_ns, abw_stream stream) {
  abw::WaitCtl w = abw::wait_ctl();
  if (!w.err) return fail(ABW_ECUDA, "abw_selftest_wait_timeout: device error word unavailable");
  w.limit_ns = limit_ns;
  return from_cuda(abw::launch_selftest_wait(w, reinterpret_cast<cudaStream_t>(stream)),
                   "abw_selftest_wait_timeout");
}

abw_status softmax_bwd(const float *s, const float *dy, float *dx, int rows, int n, abw_stream stream) {
  if (rows < 0 || n < 1) return fail(ABW_EINVAL, "softmax_bwd: rows=%d n=%d (need rows >= 0, n >= 1)", rows, n);
  if (rows == 0) return ABW_OK;
  const size_t bytes = static_cast<size_t>(rows) * n * 4;
  Range in[] = {{"s", s, bytes}, {"dy", dy, bytes}};
  Range out[] = {{"dx", dx, bytes}};
  abw_status st = check_buffers("softmax_bwd", in, 2, out, 1);
  if (st != ABW_OK) return st;
  return from_cuda(abw::launch_softmax_bwd(s, dy, dx, rows, n, reinterpret_cast<cudaStream_t>(stream)),
                   "softmax_bwd");
}

abw_status rope_bwd(const float *dy, float *dx, int B, int T, int H, int D, const float *theta, int pos0,
                    float base, int interleaved, abw_stream stream) {
  if (B < 0 || T < 0 || H < 0) return fail(ABW_EINVAL, "rope_bwd: negative size");
  if (D < 2 || (D & 1)) return fail(ABW_EINVAL, "rope_bwd: D=%d must be even and >= 2", D);
  if (D > 512) return fail(ABW_ENOTSUP, "rope_bwd: D=%d > 512", D);
  if (!theta && !(base > 0.0f)) return fail(ABW_EINVAL, "rope_bwd: base must be > 0 when theta is NULL");
  if (!theta && pos0 < 0) return fail(ABW_EINVAL, "rope_bwd: pos0 must be >= 0");
  if (B == 0 || T == 0 || H == 0) return ABW_OK;
  const size_t bytes = static_cast<size_t>(B) * T * H * D * 4;
  const size_t tbytes = theta ? static_cast<size_t>(B) * T * (D / 2) * 4 : 0;
  Range in[] = {{"dy", dy, bytes}, {"theta", theta, tbytes}};
  if (dx != dy) {
    Range out[] = {{"dx", dx, bytes}};
    abw_status st = check_buffers("rope_bwd", in, 2, out, 1);
    if (st != ABW_OK) return st;
  } else {
    Range out[] = {{"dx", dx, bytes}};
    abw_status st = check_buffers("rope_bwd", in + 1, 1, out, 1);   // in place: only theta must not overlap
    if (st != ABW_OK) return st;
  }
  return from_cuda(abw::launch_rope_bwd(dy, dx, B, T, H, D, theta, pos0, static_cast<double>(base),
                                        interleaved ? 1 : 0, reinterpret_cast<cudaStream_t>(stream)),
                   "rope_bwd");
}

abw_status rmsnorm_bwd(const void *x, abw_dtype x_dtype, const float *gamma, const float *dy, void *dx,
                       abw_dtype dx_dtype, int rows, int n, float eps, abw_stream stream) {
  if (rows < 0 || n < 1) return fail(ABW_EINVAL, "rmsnorm_bwd: rows=%d n=%d", rows, n);
  if ((x_dtype != ABW_F32 && x_dtype != ABW_BF16) || (dx_dtype != ABW_F32 && dx_dtype != ABW_BF16))
    return fail(ABW_EINVAL, "rmsnorm_bwd: bad dtype");
  if (!(eps >= 0.0f)) return fail(ABW_EINVAL, "rmsnorm_bwd: eps must be >= 0");
  if (rows == 0) return ABW_OK;
  const size_t rn = static_cast<size_t>(rows) * n;
  Range in[] = {{"x", x, rn * dt_size(x_dtype)}, {"gamma", gamma, static_cast<size_t>(n) * 4}, {"dy", dy, rn * 4}};
  Range out[] = {{"dx", dx, rn * dt_size(dx_dtype)}};
  abw_status st = check_buffers("rmsnorm_bwd", in, 3, out, 1);
  if (st != ABW_OK) return st;
  return from_cuda(abw::launch_rmsnorm_bwd(x, x_dtype == ABW_BF16, gamma, dy, dx, dx_dtype == ABW_BF16, rows, n,
                                           eps, reinterpret_cast<cudaStream_t>(stream)),
                   "rmsnorm_bwd");
}

abw_status rmsnorm_bwd_dgamma(const void *x, abw_dtype x_dtype, const float *gamma, const float *dy, void *dx,
                              abw_dtype dx_dtype, float *dgamma, int rows, int n, float eps, abw_stream stream) {
  if (rows < 0 || n < 1) return fail(ABW_EINVAL, "rmsnorm_bwd_dgamma: rows=%d n=%d", rows, n);
  if ((x_dtype != ABW_F32 && x_dtype != ABW_BF16) || (dx_dtype != ABW_F32 && dx_dtype != ABW_BF16))
    return fail(ABW_EINVAL, "rmsnorm_bwd_dgamma: bad dtype");
  if (!(eps >= 0.0f)) return fail(ABW_EINVAL, "rmsnorm_bwd_dgamma: eps must be >= 0");
  const size_t rn = static_cast<size_t>(rows) * n;
  Range in[] = {{"x", x, rn * dt_size(x_dtype)},
                {"gamma", gamma, dx ? static_cast<size_t>(n) * 4 : 0},
                {"dy", dy, rn * 4}};
  Range out[] = {{"dgamma", dgamma, static_cast<size_t>(n) * 4}, {"dx", dx, dx ? rn * dt_size(dx_dtype) : 0}};
  abw_status st = check_buffers("rmsnorm_bwd_dgamma", in, 3, out, 2);
  if (st != ABW_OK) return st;
  return from_cuda(abw::launch_rmsnorm_bwd_dgamma(x, x_dtype == ABW_BF16, gamma, dy, dx, dx_dtype == ABW_BF16,
                                                  dgamma, rows, n, eps, reinterpret_cast<cudaStream_t>(stream)),
                   "rmsnorm_bwd_dgamma");
}

abw_status relu2_mul_bwd(const void *gate, const void *up, abw_dtype act_dtype, const float *dh, float *dgate,
                         float *dup, long long n, abw_stream stream) {
  if (n < 0) return fail(ABW_EINVAL, "relu2_mul_bwd: n=%lld", n);
  if (act_dtype != ABW_F32 && act_dtype != ABW_BF16) return fail(ABW_EINVAL, "relu2_mul_bwd: bad dtype");
  if (n == 0) return ABW_OK;
  const size_t nb = static_cast<size_t>(n);
  Range in[] = {{"gate", gate, nb * dt_size(act_dtype)}, {"up", up, nb * dt_size(act_dtype)}, {"dh", dh, nb * 4}};
  Range out[] = {{"dgate", dgate, nb * 4}, {"dup", dup, nb * 4}};
  abw_status st = check_buffers("relu2_mul_bwd", in, 3, out, 2);
  if (st != ABW_OK) return st;
  return from_cuda(abw::launch_relu2_mul_bwd(gate, up, act_dtype == ABW_BF16, dh, dgate, dup, n,
                                             reinterpret_cast<cudaStream_t>(stream)),
                   "relu2_mul_bwd");
}

size_t lora_bwd_workspace_bytes(int rows, int r) {
  if (rows < 0 || r < 1) return 0;
  return abw::lora_workspace_bytes(rows, r);
}

abw_status lora_bwd(const void *x, abw_dtype x_dtype, const float *dy, const float *A, const float *B, float *dA,
                    float *dB, int rows, int n_in, int n_out, int r, float scale, void *workspace,
                    size_t workspace_bytes, abw_stream stream) {
  if (rows < 0 || n_in < 1 || n_out < 1) return fail(ABW_EINVAL, "lora_bwd: rows=%d n_in=%d n_out=%d", rows, n_in, n_out);
  if (x_dtype != ABW_F32 && x_dtype != ABW_BF16) return fail(ABW_EINVAL, "lora_bwd: bad dtype");
  if (r < 1 || r > 16) return fail(ABW_ENOTSUP, "lora_bwd: rank r=%d unsupported (1 <= r <= 16)", r);
  if (n_in % 4 != 0 || n_out % 4 != 0)
    return fail(ABW_ENOTSUP, "lora_bwd: n_in=%d, n_out=%d must be multiples of 4", n_in, n_out);
  if (!(scale == scale)) return fail(ABW_EINVAL, "lora_bwd: scale is NaN");
  const size_t need = abw::lora_workspace_bytes(rows, r);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(ABW_EWORKSPACE, "lora_bwd: workspace %zu bytes at %p, need %zu", workspace_bytes, workspace, need);
  const size_t rb = static_cast<size_t>(rows);
  Range in[] = {{"x", x, rb * n_in * dt_size(x_dtype)}, {"dy", dy, rb * n_out * 4},
                {"A", A, static_cast<size_t>(r) * n_in * 4}, {"B", B, static_cast<size_t>(n_out) * r * 4}};
  Range out[] = {{"dA", dA, static_cast<size_t>(r) * n_in * 4}, {"dB", dB, static_cast<size_t>(n_out) * r * 4},
                 {"workspace", workspace, need}};
  abw_status st = check_buffers("lora_bwd", in, 4, out, 3);
  if (st != ABW_OK) return st;
  return from_cuda(abw::launch_lora_bwd(x, x_dtype == ABW_BF16, dy, A, B, dA, dB, rows, n_in, n_out, r, scale,
                                        workspace, reinterpret_cast<cudaStream_t>(stream)),
                   "lora_bwd");
}

abw_status attn_bwd_decode(const float *q, const void *k, const void *v, const float *dout, float *dq, float *dk,
                           float *dv, int B, int Hq, int Hkv, int S, int D, abw_dtype kv_dtype, float scale,
                           float rope_base, int q_pos, abw_stream stream) {
  if (B < 0 || Hq < 0 || Hkv < 0 || D < 0) return fail(ABW_EINVAL, "attn_bwd_decode: negative size");
  if (S < 1) return fail(ABW_EINVAL, "attn_bwd_decode: S=%d (softmax over no keys is undefined)", S);
  if (kv_dtype != ABW_F32 && kv_dtype != ABW_BF16) return fail(ABW_EINVAL, "attn_bwd_decode: bad kv dtype");
  if (Hkv == 0 || Hq % Hkv != 0) return fail(ABW_EINVAL, "attn_bwd_decode: Hq=%d not a multiple of Hkv=%d", Hq, Hkv);
  if (Hq / Hkv > 8) return fail(ABW_ENOTSUP, "attn_bwd_decode: Hq/Hkv=%d > 8", Hq / Hkv);
  const size_t es = dt_size(kv_dtype);
  if (D < 2 || (D & 1) || (D * es) % 16 != 0 || D * es > 512)
    return fail(ABW_ENOTSUP, "attn_bwd_decode: D=%d unsupported (even, D*sizeof(kv) %% 16 == 0, <= 512 B)", D);
  if (!(scale == scale)) return fail(ABW_EINVAL, "attn_bwd_decode: scale is NaN");
  if (B == 0 || Hq == 0) return ABW_OK;
  const size_t qb = static_cast<size_t>(B) * Hq * D * 4;
  const size_t kvn = static_cast<size_t>(B) * S * Hkv * D;
  Range in[] = {{"q", q, qb}, {"k", k, kvn * es}, {"v", v, kvn * es}, {"dout", dout, qb}};
  Range out[] = {{"dq", dq, qb}, {"dk", dk, kvn * 4}, {"dv", dv, kvn * 4}};
  abw_status st = check_buffers("attn_bwd_decode", in, 4, out, 3);
  if (st != ABW_OK) return st;
  abw::WaitCtl w = abw::wait_ctl();
  if (!w.err) return fail(ABW_ECUDA, "attn_bwd_decode: no CUDA device");
  const char *why = nullptr;
  const double rb = (rope_base > 0.0f && q_pos >= 0) ? static_cast<double>(rope_base) : 0.0;
  return from_cuda(abw::launch_attn_bwd_decode(q, k, v, dout, dq, dk, dv, B, Hq, Hkv, S, D, kv_dtype == ABW_BF16,
                                               scale, rb, q_pos, w, reinterpret_cast<cudaStream_t>(stream), &why),
                   "attn_bwd_decode", why);
}

abw_status attn_fwd_causal(const void *q, const void *k, const void *v, void *o, float *lse, int B, int T, int Hq,
                           int Hkv, int D, float scale, abw_stream stream) {
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0) return fail(ABW_EINVAL, "attn_fwd_causal: negative size");
  if (Hkv == 0 || Hq % Hkv != 0) return fail(ABW_EINVAL, "attn_fwd_causal: Hq=%d not a multiple of Hkv=%d", Hq, Hkv);
  if (D != 128) return fail(ABW_ENOTSUP, "attn_fwd_causal: D=%d unsupported (D == 128)", D);
  if (!(scale == scale)) return fail(ABW_EINVAL, "attn_fwd_causal: scale is NaN");
  if (B == 0 || T == 0 || Hq == 0) return ABW_OK;
  const size_t qn = static_cast<size_t>(B) * T * Hq * D, kn = static_cast<size_t>(B) * T * Hkv * D;
  Range in[] = {{"q", q, qn * 2}, {"k", k, kn * 2}, {"v", v, kn * 2}};
  Range out[] = {{"o", o, qn * 2}, {"lse", lse, static_cast<size_t>(B) * Hq * T * 4}};
  abw_status st = check_buffers("attn_fwd_causal", in, 3, out, 2);
  if (st != ABW_OK) return st;
  abw::WaitCtl w = abw::wait_ctl();
  if (!w.err) return fail(ABW_ECUDA, "attn_fwd_causal: no CUDA device");
  const char *why = nullptr;
  return from_cuda(abw::launch_attn_fwd_causal(q, k, v, o, lse, B, T, Hq, Hkv, D, scale, w,
                                               reinterpret_cast<cudaStream_t>(stream), &why),
                   "attn_fwd_causal", why);
}

size_t attn_bwd_causal_workspace_bytes(int B, int T, int Hq, int D) {
  if (B < 0 || T < 0 || Hq < 0 || D < 0) return 0;
  return abw::causal_workspace_bytes(B, T, Hq, D);
}

abw_status attn_bwd_causal(const void *q, const void *k, const void *v, const void *o, const void *dout,
                           const float *lse, float *dq, float *dk, float *dv, int B, int T, int Hq, int Hkv, int D,
                           float scale, float rope_base, int pos0, void *workspace, size_t workspace_bytes,
                           abw_stream stream) {
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0) return fail(ABW_EINVAL, "attn_bwd_causal: negative size");
  if (Hkv == 0 || Hq % Hkv != 0) return fail(ABW_EINVAL, "attn_bwd_causal: Hq=%d not a multiple of Hkv=%d", Hq, Hkv);
  if (D != 128) return fail(ABW_ENOTSUP, "attn_bwd_causal: D=%d unsupported (D == 128)", D);
  if (rope_base > 0.0f && pos0 < 0) return fail(ABW_EINVAL, "attn_bwd_causal: pos0 must be >= 0");
  if (!(scale == scale)) return fail(ABW_EINVAL, "attn_bwd_causal: scale is NaN");
  if (B == 0 || T == 0 || Hq == 0) return ABW_OK;
  const size_t need = abw::causal_workspace_bytes(B, T, Hq, D);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(ABW_EWORKSPACE, "attn_bwd_causal: workspace %zu bytes at %p, need %zu", workspace_bytes, workspace,
                need);
  const size_t qn = static_cast<size_t>(B) * T * Hq * D, kn = static_cast<size_t>(B) * T * Hkv * D;
  Range in[] = {{"q", q, qn * 2},    {"k", k, kn * 2},
                {"v", v, kn * 2},    {"o", o, qn * 2},
                {"dout", dout, qn * 2}, {"lse", lse, static_cast<size_t>(B) * Hq * T * 4}};
  Range out[] = {{"dq", dq, qn * 4}, {"dk", dk, kn * 4}, {"dv", dv, kn * 4}, {"workspace", workspace, need}};
  abw_status st = check_buffers("attn_bwd_causal", in, 6, out, 4);
  if (st != ABW_OK) return st;
  abw::WaitCtl w = abw::wait_ctl();
  if (!w.err) return fail(ABW_ECUDA, "attn_bwd_causal: no CUDA device");
  const char *why = nullptr;
  const double rb = rope_base > 0.0f ? static_cast<double>(rope_base) : 0.0;
  return from_cuda(abw::launch_attn_bwd_causal(q, k, v, nullptr, o, dout, lse, dq, dk, dv, B, T, Hq, Hkv, D, scale, rb, pos0,
                                               workspace, workspace_bytes, w,
                                               reinterpret_cast<cudaStream_t>(stream), &why),
                   "attn_bwd_causal", why);
}

abw_status attn_bwd_causal_saved_p(const void *q, const void *k, const void *v, const void *p_attn, const void *o,
                                   const void *dout, float *dq, float *dk, float *dv, int B, int T, int Hq, int Hkv,
                                   int D, float scale, float rope_base, int pos0, void *workspace,
                                   size_t workspace_bytes, abw_stream stream) {
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0) return fail(ABW_EINVAL, "attn_bwd_causal_saved_p: negative size");
  if (Hkv == 0 || Hq % Hkv != 0)
    return fail(ABW_EINVAL, "attn_bwd_causal_saved_p: Hq=%d not a multiple of Hkv=%d", Hq, Hkv);
  if (D != 128) return fail(ABW_ENOTSUP, "attn_bwd_causal_saved_p: D=%d unsupported (D == 128)", D);
  if (rope_base > 0.0f && pos0 < 0) return fail(ABW_EINVAL, "attn_bwd_causal_saved_p: pos0 must be >= 0");
  if (!(scale == scale)) return fail(ABW_EINVAL, "attn_bwd_causal_saved_p: scale is NaN");
  if (B == 0 || T == 0 || Hq == 0) return ABW_OK;
  const size_t need = abw::causal_workspace_bytes(B, T, Hq, D);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(ABW_EWORKSPACE, "attn_bwd_causal_saved_p: workspace %zu bytes at %p, need %zu", workspace_bytes,
                workspace, need);
  const size_t qn = static_cast<size_t>(B) * T * Hq * D, kn = static_cast<size_t>(B) * T * Hkv * D;
  const size_t pn = static_cast<size_t>(B) * Hq * T * T;
  Range in[] = {{"q", q, qn * 2},    {"k", k, kn * 2},      {"v", v, kn * 2},
                {"p_attn", p_attn, pn * 2}, {"o", o, qn * 2}, {"dout", dout, qn * 2}};
  Range out[] = {{"dq", dq, qn * 4}, {"dk", dk, kn * 4}, {"dv", dv, kn * 4}, {"workspace", workspace, need}};
  abw_status st = check_buffers("attn_bwd_causal_saved_p", in, 6, out, 4);
  if (st != ABW_OK) return st;
  abw::WaitCtl w = abw::wait_ctl();
  if (!w.err) return fail(ABW_ECUDA, "attn_bwd_causal_saved_p: no CUDA device");
  const char *why = nullptr;
  const double rb = rope_base > 0.0f ? static_cast<double>(rope_base) : 0.0;
  return from_cuda(abw::launch_attn_bwd_causal(q, k, v, p_attn, o, dout, nullptr, dq, dk, dv, B, T, Hq, Hkv, D, scale,
                                               rb, pos0, workspace, workspace_bytes, w,
                                               reinterpret_cast<cudaStream_t>(stream), &why),
                   "attn_bwd_causal_saved_p", why);
}

abw_status attn_bwd_causal_noalloc(const void *q, const void *k, const void *v, const void *o, const void *dout,
                                   const float *lse, float *dq, float *dk, float *dv, int B, int T, int Hq, int Hkv,
                                   int D, float scale, float rope_base, int pos0, abw_stream stream) {
  // Same checks and kernels as attn_bwd_causal; the workspace is the
  // library's built-in device scratch instead of a caller allocation.
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0) return fail(ABW_EINVAL, "attn_bwd_causal_noalloc: negative size");
  if (Hkv == 0 || Hq % Hkv != 0)
    return fail(ABW_EINVAL, "attn_bwd_causal_noalloc: Hq=%d not a multiple of Hkv=%d", Hq, Hkv);
  if (D != 128) return fail(ABW_ENOTSUP, "attn_bwd_causal_noalloc: D=%d unsupported (D == 128)", D);
  if (rope_base > 0.0f && pos0 < 0) return fail(ABW_EINVAL, "attn_bwd_causal_noalloc: pos0 must be >= 0");
  if (!(scale == scale)) return fail(ABW_EINVAL, "attn_bwd_causal_noalloc: scale is NaN");
  if (B == 0 || T == 0 || Hq == 0) return ABW_OK;
  const size_t need = abw::causal_workspace_bytes(B, T, Hq, D);
  if (need > abw::kNoAllocScratchBytes)
    return fail(ABW_EWORKSPACE,
                "attn_bwd_causal_noalloc: these sizes need %zu bytes of scratch, more than the built-in %zu "
                "(about B*Hq*T^2 bytes); use attn_bwd_causal with a workspace",
                need, static_cast<size_t>(abw::kNoAllocScratchBytes));
  const size_t qn = static_cast<size_t>(B) * T * Hq * D, kn = static_cast<size_t>(B) * T * Hkv * D;
  Range in[] = {{"q", q, qn * 2},    {"k", k, kn * 2},
                {"v", v, kn * 2},    {"o", o, qn * 2},
                {"dout", dout, qn * 2}, {"lse", lse, static_cast<size_t>(B) * Hq * T * 4}};
  Range out[] = {{"dq", dq, qn * 4}, {"dk", dk, kn * 4}, {"dv", dv, kn * 4}};
  abw_status st = check_buffers("attn_bwd_causal_noalloc", in, 6, out, 3);
  if (st != ABW_OK) return st;
  abw::WaitCtl w = abw::wait_ctl();
  if (!w.err) return fail(ABW_ECUDA, "attn_bwd_causal_noalloc: no CUDA device");
  const char *why = nullptr;
  void *scratch = nullptr;
  cudaError_t e = abw::noalloc_scratch(&scratch, &why);
  if (e != cudaSuccess) return from_cuda(e, "attn_bwd_causal_noalloc", why);
  const double rb = rope_base > 0.0f ? static_cast<double>(rope_base) : 0.0;
  return from_cuda(abw::launch_attn_bwd_causal(q, k, v, nullptr, o, dout, lse, dq, dk, dv, B, T, Hq, Hkv, D, scale, rb, pos0,
                                               scratch, abw::kNoAllocScratchBytes, w,
                                               reinterpret_cast<cudaStream_t>(stream), &why),
                   "attn_bwd_causal_noalloc", why);
}

abw_status qk_norm_rope_fwd(const void *q, const void *k, abw_dtype dtype, const float *gamma_q, const float *gamma_k,
                            void *q_out, void *k_out, int B, int T, int Hq, int Hkv, int D, long long q_stride,
                            long long k_stride, float eps, float rope_base, int rotary_dim, int interleaved,
                            const int *positions, int n_axes, const int *sections, int pos0, abw_stream stream) {
  abw_status st = check_qk("qk_norm_rope_fwd", B, T, Hq, Hkv, D, dtype, eps);
  if (st != ABW_OK) return st;
  if (q_stride < 0 || k_stride < 0) return fail(ABW_EINVAL, "qk_norm_rope_fwd: negative token stride");
  abw::QkNormRopeArgs a = {};
  a.D = D;
  st = check_rotation("qk_norm_rope_fwd", a, rope_base, rotary_dim, interleaved, positions, n_axes, sections, pos0);
  if (st != ABW_OK) return st;
  if (B == 0 || T == 0 || Hq + Hkv == 0) return ABW_OK;
  const size_t es = dt_size(dtype), ntok = static_cast<size_t>(B) * T;
  const size_t qr = static_cast<size_t>(Hq) * D * es, kr = static_cast<size_t>(Hkv) * D * es;
  const size_t gb = static_cast<size_t>(D) * 4;
  Rows in[] = {{"q", q, ntok, qr, q_stride ? q_stride * es : qr, es},
               {"k", k, ntok, kr, k_stride ? k_stride * es : kr, es},
               dense("gamma_q", gamma_q, gamma_q && Hq ? gb : 0),
               dense("gamma_k", gamma_k, gamma_k && Hkv ? gb : 0),
               dense("positions", a.positions, a.positions ? ntok * 4 * a.n_axes : 0, 4)};
  Rows out[] = {dense("q_out", q_out, ntok * qr), dense("k_out", k_out, ntok * kr)};
  st = check_rows("qk_norm_rope_fwd", in, 5, out, 2);
  if (st != ABW_OK) return st;
  a.x[0] = q, a.x[1] = k;
  a.out[0] = q_out, a.out[1] = k_out;
  a.gamma[0] = gamma_q, a.gamma[1] = gamma_k;
  a.bf16 = dtype == ABW_BF16;
  a.B = B, a.T = T, a.H[0] = Hq, a.H[1] = Hkv;
  a.x_stride[0] = token_stride(q_stride, B, T, static_cast<long long>(Hq) * D);
  a.x_stride[1] = token_stride(k_stride, B, T, static_cast<long long>(Hkv) * D);
  a.out_stride[0] = static_cast<long long>(Hq) * D;
  a.out_stride[1] = static_cast<long long>(Hkv) * D;
  a.eps = eps;
  return from_cuda(abw::launch_qk_norm_rope(a, reinterpret_cast<cudaStream_t>(stream)), "qk_norm_rope_fwd");
}

size_t qk_norm_rope_bwd_workspace_bytes(int D) {
  return D < 1 || D > 512 ? 0 : abw::qk_norm_rope_bwd_workspace_bytes(D);
}

abw_status qk_norm_rope_bwd(const void *q, const void *k, abw_dtype dtype, const void *dq_out, const void *dk_out,
                            abw_dtype dy_dtype, const float *gamma_q, const float *gamma_k, void *dq, void *dk,
                            float *dgamma_q, float *dgamma_k, int B, int T, int Hq, int Hkv, int D, long long q_stride,
                            long long k_stride, long long dq_stride, long long dk_stride, float eps, float rope_base,
                            int rotary_dim, int interleaved, const int *positions, int n_axes, const int *sections,
                            int pos0, void *workspace, size_t workspace_bytes, abw_stream stream) {
  abw_status st = check_qk("qk_norm_rope_bwd", B, T, Hq, Hkv, D, dtype, eps);
  if (st != ABW_OK) return st;
  if (dy_dtype != ABW_F32 && dy_dtype != ABW_BF16) return fail(ABW_EINVAL, "qk_norm_rope_bwd: bad dy dtype");
  if (q_stride < 0 || k_stride < 0 || dq_stride < 0 || dk_stride < 0)
    return fail(ABW_EINVAL, "qk_norm_rope_bwd: negative token stride");
  abw::QkNormRopeArgs a = {};
  a.D = D;
  st = check_rotation("qk_norm_rope_bwd", a, rope_base, rotary_dim, interleaved, positions, n_axes, sections, pos0);
  if (st != ABW_OK) return st;
  const bool norm = gamma_q || gamma_k;
  const size_t need = norm ? abw::qk_norm_rope_bwd_workspace_bytes(D) : 0;
  if (need && (workspace == nullptr || workspace_bytes < need))
    return fail(ABW_EWORKSPACE, "qk_norm_rope_bwd: workspace %zu bytes at %p, need %zu", workspace_bytes, workspace,
                need);
  const size_t es = dt_size(dtype), ds = dt_size(dy_dtype), ntok = static_cast<size_t>(B) * T;
  const size_t qn = static_cast<size_t>(Hq) * D, kn = static_cast<size_t>(Hkv) * D, gb = static_cast<size_t>(D) * 4;
  Rows in[] = {{"q", q, ntok, qn * es, q_stride ? q_stride * es : qn * es, es},
               {"k", k, ntok, kn * es, k_stride ? k_stride * es : kn * es, es},
               dense("dq_out", dq_out, ntok * qn * ds),
               dense("dk_out", dk_out, ntok * kn * ds),
               dense("gamma_q", gamma_q, gamma_q && Hq ? gb : 0),
               dense("gamma_k", gamma_k, gamma_k && Hkv ? gb : 0),
               dense("positions", a.positions, a.positions ? ntok * 4 * a.n_axes : 0, 4)};
  Rows out[] = {{"dq", dq, ntok, qn * es, dq_stride ? dq_stride * es : qn * es, es},
                {"dk", dk, ntok, kn * es, dk_stride ? dk_stride * es : kn * es, es},
                dense("dgamma_q", dgamma_q, dgamma_q ? gb : 0),
                dense("dgamma_k", dgamma_k, dgamma_k ? gb : 0),
                dense("workspace", workspace, need)};
  st = check_rows("qk_norm_rope_bwd", in, 7, out, 5);
  if (st != ABW_OK) return st;
  if (Hq + Hkv == 0 && !dgamma_q && !dgamma_k) return ABW_OK;
  a.x[0] = q, a.x[1] = k;
  a.dy[0] = dq_out, a.dy[1] = dk_out;
  a.out[0] = dq, a.out[1] = dk;
  a.gamma[0] = gamma_q, a.gamma[1] = gamma_k;
  a.dgamma[0] = gamma_q ? dgamma_q : nullptr;
  a.dgamma[1] = gamma_k ? dgamma_k : nullptr;
  a.backward = 1;
  a.bf16 = dtype == ABW_BF16;
  a.dy_bf16 = dy_dtype == ABW_BF16;
  a.B = B, a.T = T, a.H[0] = Hq, a.H[1] = Hkv;
  a.x_stride[0] = token_stride(q_stride, B, T, static_cast<long long>(qn));
  a.x_stride[1] = token_stride(k_stride, B, T, static_cast<long long>(kn));
  a.out_stride[0] = token_stride(dq_stride, B, T, static_cast<long long>(qn));
  a.out_stride[1] = token_stride(dk_stride, B, T, static_cast<long long>(kn));
  a.eps = eps;
  a.ws = workspace;
  return from_cuda(abw::launch_qk_norm_rope(a, reinterpret_cast<cudaStream_t>(stream)), "qk_norm_rope_bwd");
}

size_t lin_attn_fwd_workspace_bytes(int B, int T, int Hkv, int D) {
  return B < 0 || T < 0 || Hkv < 0 || D < 0 ? 0 : abw::lin_attn_workspace_bytes(B, T, Hkv, D, 0);
}

size_t lin_attn_bwd_workspace_bytes(int B, int T, int Hkv, int D) {
  return B < 0 || T < 0 || Hkv < 0 || D < 0 ? 0 : abw::lin_attn_workspace_bytes(B, T, Hkv, D, 1);
}

abw_status lin_attn_fwd(const void *q, const void *k, const void *v, const float *log_decay,
                        const float *initial_state, const int *lengths, void *o, float *final_state, int B, int T,
                        int Hq, int Hkv, int D, long long q_stride, long long k_stride, long long v_stride,
                        long long o_stride, float scale, void *workspace, size_t workspace_bytes, abw_stream stream) {
  abw_status st = check_lin("lin_attn_fwd", B, T, Hq, Hkv, D, scale);
  if (st != ABW_OK) return st;
  if (q_stride < 0 || k_stride < 0 || v_stride < 0 || o_stride < 0)
    return fail(ABW_EINVAL, "lin_attn_fwd: negative token stride");
  if (B == 0) return ABW_OK;
  const size_t need = abw::lin_attn_workspace_bytes(B, T, Hkv, D, 0);
  if (need && (workspace == nullptr || workspace_bytes < need))
    return fail(ABW_EWORKSPACE, "lin_attn_fwd: workspace %zu bytes at %p, need %zu", workspace_bytes, workspace, need);
  const size_t sbytes = static_cast<size_t>(B) * Hkv * D * D * 4;
  Rows in[] = {lin_rows("q", q, B, T, Hq, D, q_stride),
               lin_rows("k", k, B, T, Hkv, D, k_stride),
               lin_rows("v", v, B, T, Hkv, D, v_stride),
               dense("log_decay", log_decay, static_cast<size_t>(Hkv) * 4, 4),
               dense("lengths", lengths, lengths ? static_cast<size_t>(B) * 4 : 0, 4),
               dense("initial_state", initial_state, initial_state && initial_state != final_state ? sbytes : 0)};
  Rows out[] = {lin_rows("o", o, B, T, Hq, D, o_stride),
                dense("final_state", final_state, final_state ? sbytes : 0),
                dense("workspace", workspace, need)};
  st = check_rows("lin_attn_fwd", in, 6, out, 3);
  if (st != ABW_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {                                 // no tokens: the state passes through
    if (!final_state || final_state == initial_state) return ABW_OK;
    return from_cuda(initial_state ? cudaMemcpyAsync(final_state, initial_state, sbytes, cudaMemcpyDeviceToDevice, cs)
                                   : cudaMemsetAsync(final_state, 0, sbytes, cs),
                     "lin_attn_fwd");
  }
  abw::WaitCtl w = abw::wait_ctl();
  if (!w.err) return fail(ABW_ECUDA, "lin_attn_fwd: no CUDA device");
  abw::LinAttnArgs a = {};
  a.q = q, a.k = k, a.v = v;
  a.log_decay = log_decay, a.initial_state = initial_state, a.lengths = lengths;
  a.o = o, a.final_state = final_state;
  a.B = B, a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.D = D;
  const long long qn = static_cast<long long>(Hq) * D, kn = static_cast<long long>(Hkv) * D;
  a.q_stride = token_stride(q_stride, B, T, qn), a.k_stride = token_stride(k_stride, B, T, kn);
  a.v_stride = token_stride(v_stride, B, T, kn), a.o_stride = token_stride(o_stride, B, T, qn);
  a.scale = scale;
  a.ws = workspace;
  const char *why = nullptr;
  return from_cuda(abw::launch_lin_attn(a, w, cs, &why), "lin_attn_fwd", why);
}

abw_status lin_attn_bwd(const void *q, const void *k, const void *v, const void *dout, const float *log_decay,
                        const float *initial_state, const float *dfinal_state, const int *lengths, void *dq, void *dk,
                        void *dv, float *dinitial_state, int B, int T, int Hq, int Hkv, int D, long long q_stride,
                        long long k_stride, long long v_stride, long long dq_stride, long long dk_stride,
                        long long dv_stride, float scale, void *workspace, size_t workspace_bytes, abw_stream stream) {
  abw_status st = check_lin("lin_attn_bwd", B, T, Hq, Hkv, D, scale);
  if (st != ABW_OK) return st;
  if (q_stride < 0 || k_stride < 0 || v_stride < 0 || dq_stride < 0 || dk_stride < 0 || dv_stride < 0)
    return fail(ABW_EINVAL, "lin_attn_bwd: negative token stride");
  if (B == 0) return ABW_OK;
  const size_t need = abw::lin_attn_workspace_bytes(B, T, Hkv, D, 1);
  if (need && (workspace == nullptr || workspace_bytes < need))
    return fail(ABW_EWORKSPACE, "lin_attn_bwd: workspace %zu bytes at %p, need %zu", workspace_bytes, workspace, need);
  const size_t sbytes = static_cast<size_t>(B) * Hkv * D * D * 4;
  Rows in[] = {lin_rows("q", q, B, T, Hq, D, q_stride),
               lin_rows("k", k, B, T, Hkv, D, k_stride),
               lin_rows("v", v, B, T, Hkv, D, v_stride),
               lin_rows("dout", dout, B, T, Hq, D, 0),
               dense("log_decay", log_decay, static_cast<size_t>(Hkv) * 4, 4),
               dense("lengths", lengths, lengths ? static_cast<size_t>(B) * 4 : 0, 4),
               dense("initial_state", initial_state, initial_state ? sbytes : 0),
               dense("dfinal_state", dfinal_state, dfinal_state && dfinal_state != dinitial_state ? sbytes : 0)};
  Rows out[] = {lin_rows("dq", dq, B, T, Hq, D, dq_stride),
                lin_rows("dk", dk, B, T, Hkv, D, dk_stride),
                lin_rows("dv", dv, B, T, Hkv, D, dv_stride),
                dense("dinitial_state", dinitial_state, dinitial_state ? sbytes : 0),
                dense("workspace", workspace, need)};
  st = check_rows("lin_attn_bwd", in, 8, out, 5);
  if (st != ABW_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (!dinitial_state || dinitial_state == dfinal_state) return ABW_OK;
    return from_cuda(dfinal_state ? cudaMemcpyAsync(dinitial_state, dfinal_state, sbytes, cudaMemcpyDeviceToDevice, cs)
                                  : cudaMemsetAsync(dinitial_state, 0, sbytes, cs),
                     "lin_attn_bwd");
  }
  abw::WaitCtl w = abw::wait_ctl();
  if (!w.err) return fail(ABW_ECUDA, "lin_attn_bwd: no CUDA device");
  abw::LinAttnArgs a = {};
  a.q = q, a.k = k, a.v = v, a.dout = dout;
  a.log_decay = log_decay, a.initial_state = initial_state, a.dfinal_state = dfinal_state, a.lengths = lengths;
  a.dq = dq, a.dk = dk, a.dv = dv, a.dinitial_state = dinitial_state;
  a.B = B, a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.D = D;
  const long long qn = static_cast<long long>(Hq) * D, kn = static_cast<long long>(Hkv) * D;
  a.q_stride = token_stride(q_stride, B, T, qn), a.k_stride = token_stride(k_stride, B, T, kn);
  a.v_stride = token_stride(v_stride, B, T, kn), a.dq_stride = token_stride(dq_stride, B, T, qn);
  a.dk_stride = token_stride(dk_stride, B, T, kn), a.dv_stride = token_stride(dv_stride, B, T, kn);
  a.scale = scale;
  a.ws = workspace;
  const char *why = nullptr;
  return from_cuda(abw::launch_lin_attn(a, w, cs, &why), "lin_attn_bwd", why);
}

abw_status lin_attn_decode(const void *q, const void *k, const void *v, abw_dtype dtype, float *state,
                           const float *log_decay, const int *slots, void *o, int B, int Hq, int Hkv, int D,
                           int n_states, float scale, abw_stream stream) {
  abw_status st = check_lin("lin_attn_decode", B, 1, Hq, Hkv, D, scale);
  if (st != ABW_OK) return st;
  if (Hq / Hkv > 8) return fail(ABW_ENOTSUP, "lin_attn_decode: Hq/Hkv=%d > 8", Hq / Hkv);
  if (dtype != ABW_F32 && dtype != ABW_BF16) return fail(ABW_EINVAL, "lin_attn_decode: bad dtype");
  if (n_states < 0 || (!slots && n_states < B))
    return fail(ABW_EINVAL, "lin_attn_decode: n_states=%d with B=%d and %s", n_states, B, slots ? "slots" : "no slots");
  if (B == 0) return ABW_OK;
  const size_t es = dt_size(dtype), n = static_cast<size_t>(B) * D * es, qb = n * Hq, kb = n * Hkv;
  Rows in[] = {dense("q", q, qb), dense("k", k, kb), dense("v", v, kb),
               dense("log_decay", log_decay, static_cast<size_t>(Hkv) * 4, 4),
               dense("slots", slots, slots ? static_cast<size_t>(B) * 4 : 0, 4)};
  Rows out[] = {dense("o", o, qb), dense("state", state, static_cast<size_t>(n_states) * Hkv * D * D * 4)};
  st = check_rows("lin_attn_decode", in, 5, out, 2);
  if (st != ABW_OK) return st;
  return from_cuda(abw::launch_lin_attn_decode(q, k, v, state, log_decay, slots, o, dtype == ABW_BF16, B, Hq, Hkv, D,
                                               n_states, scale, reinterpret_cast<cudaStream_t>(stream)),
                   "lin_attn_decode");
}

}  // extern "C"
