"""Attention backward chain for NVIDIA GB300 (sm_103a).

A thin PyTorch-facing binding of the C ABI in ``include/attn_bwd.h``: each
function checks dtypes, shapes and contiguity, allocates missing outputs with
torch (device memory only), and passes device pointers plus the current CUDA
stream to the library.  Every arithmetic step runs in the library's CUDA
kernels; nothing here computes, and there is no fallback path.

Functions (same names as the C ABI):
  softmax_bwd, rope_bwd, rmsnorm_bwd, rmsnorm_bwd_dgamma, relu2_mul_bwd,
  lora_bwd, attn_bwd_decode, attn_fwd_causal, attn_bwd_causal,
  attn_bwd_causal_saved_p, attn_bwd_causal_workspace_bytes, device_check,
  qk_norm_rope_fwd, qk_norm_rope_bwd, lin_attn_fwd, lin_attn_bwd,
  lin_attn_decode and their *_workspace_bytes
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import _binding as _b

__all__ = ["softmax_bwd", "rope_bwd", "rmsnorm_bwd", "rmsnorm_bwd_dgamma", "relu2_mul_bwd", "lora_bwd",
           "attn_bwd_decode", "attn_fwd_causal", "attn_bwd_causal", "attn_bwd_causal_saved_p",
           "attn_bwd_causal_workspace_bytes", "device_check", "AbwError", "library",
           "qk_norm_rope_fwd", "qk_norm_rope_bwd", "qk_norm_rope_bwd_workspace_bytes", "lin_attn_fwd",
           "lin_attn_fwd_workspace_bytes", "lin_attn_bwd", "lin_attn_bwd_workspace_bytes", "lin_attn_decode"]

AbwError = _b.AbwError

_DT = {torch.float32: _b.F32, torch.bfloat16: _b.BF16}


def library():
    """The loaded ctypes library (built for sm_103a on first use)."""
    return _b.load()


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _s(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _req(t, name, dtypes, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")


def device_check(stream=None) -> None:
    """Synchronize and raise if a kernel's bounded wait ran out."""
    _b.check(library().abw_device_check(_s(stream)), "abw_device_check")


def softmax_bwd(s, dy, dx=None, stream=None):
    """dx = s * (dy - sum(s * dy)) over the last axis; s, dy fp32."""
    _req(s, "s", (torch.float32,))
    _req(dy, "dy", (torch.float32,), s.shape)
    n = s.shape[-1] if s.dim() else 1
    rows = s.numel() // max(n, 1)
    if dx is None:
        dx = torch.empty_like(s)
    _req(dx, "dx", (torch.float32,), s.shape)
    _b.check(library().softmax_bwd(_p(s), _p(dy), _p(dx), rows, n, _s(stream)), "softmax_bwd")
    return dx


def rope_bwd(dy, theta=None, pos0=0, base=10000.0, interleaved=True, dx=None, stream=None):
    """R(-theta) on the rotary pairs of dy [B][T][H][D] fp32; theta [B*T][D/2]
    fp32 or None (then theta = (pos0 + t) base^(-2i/D)).  dx may be dy."""
    _req(dy, "dy", (torch.float32,))
    if dy.dim() != 4:
        raise ValueError("dy must be [B][T][H][D]")
    B, T, H, D = dy.shape
    if theta is not None:
        _req(theta, "theta", (torch.float32,), (B * T, D // 2))
    if dx is None:
        dx = torch.empty_like(dy)
    _req(dx, "dx", (torch.float32,), dy.shape)
    _b.check(library().rope_bwd(_p(dy), _p(dx), B, T, H, D, _p(theta), int(pos0), float(base),
                                1 if interleaved else 0, _s(stream)), "rope_bwd")
    return dx


def rmsnorm_bwd(x, gamma, dy, eps=1e-6, dx=None, dx_dtype=torch.float32, stream=None):
    """RMSNorm backward per row: x [rows][n] fp32/bf16, gamma [n] fp32,
    dy [rows][n] fp32 -> dx [rows][n] (fp32 or bf16)."""
    _req(x, "x", (torch.float32, torch.bfloat16))
    n = x.shape[-1]
    rows = x.numel() // n
    _req(gamma, "gamma", (torch.float32,), (n,))
    _req(dy, "dy", (torch.float32,), x.shape)
    if dx is None:
        dx = torch.empty(x.shape, dtype=dx_dtype, device=x.device)
    _req(dx, "dx", (torch.float32, torch.bfloat16), x.shape)
    _b.check(library().rmsnorm_bwd(_p(x), _DT[x.dtype], _p(gamma), _p(dy), _p(dx), _DT[dx.dtype], rows, n,
                                   float(eps), _s(stream)), "rmsnorm_bwd")
    return dx


def rmsnorm_bwd_dgamma(x, gamma, dy, eps=1e-6, dx=None, dgamma=None, dx_dtype=torch.float32, want_dx=True,
                       stream=None):
    """RMSNorm backward with the scale gradient.  x [rows][n] fp32/bf16,
    gamma [n] fp32, dy [rows][n] fp32.  Returns (dx or None, dgamma [n] fp32)."""
    _req(x, "x", (torch.float32, torch.bfloat16))
    n = x.shape[-1]
    rows = x.numel() // n
    _req(dy, "dy", (torch.float32,), x.shape)
    if want_dx:
        _req(gamma, "gamma", (torch.float32,), (n,))
        if dx is None:
            dx = torch.empty(x.shape, dtype=dx_dtype, device=x.device)
        _req(dx, "dx", (torch.float32, torch.bfloat16), x.shape)
    else:
        dx = None
    if dgamma is None:
        dgamma = torch.empty(n, dtype=torch.float32, device=x.device)
    _req(dgamma, "dgamma", (torch.float32,), (n,))
    _b.check(library().rmsnorm_bwd_dgamma(_p(x), _DT[x.dtype], _p(gamma) if want_dx else None, _p(dy), _p(dx),
                                          _DT[dx.dtype] if dx is not None else _b.F32, _p(dgamma), rows, n,
                                          float(eps), _s(stream)), "rmsnorm_bwd_dgamma")
    return dx, dgamma


def relu2_mul_bwd(gate, up, dh, dgate=None, dup=None, stream=None):
    """Backward of hidden = ReLU(gate)^2 * up: gate, up fp32/bf16 (same
    dtype), dh fp32, all the same shape.  Returns (dgate, dup) fp32."""
    _req(gate, "gate", (torch.float32, torch.bfloat16))
    _req(up, "up", (gate.dtype,), gate.shape)
    _req(dh, "dh", (torch.float32,), gate.shape)
    dgate = torch.empty(gate.shape, dtype=torch.float32, device=gate.device) if dgate is None else dgate
    dup = torch.empty(gate.shape, dtype=torch.float32, device=gate.device) if dup is None else dup
    _req(dgate, "dgate", (torch.float32,), gate.shape)
    _req(dup, "dup", (torch.float32,), gate.shape)
    _b.check(library().relu2_mul_bwd(_p(gate), _p(up), _DT[gate.dtype], _p(dh), _p(dgate), _p(dup), gate.numel(),
                                     _s(stream)), "relu2_mul_bwd")
    return dgate, dup


def lora_bwd_workspace_bytes(rows, r) -> int:
    return int(library().lora_bwd_workspace_bytes(rows, r))


def lora_bwd(x, dy, A, B, scale, dA=None, dB=None, workspace=None, stream=None):
    """LoRA adapter gradients of y = scale * B (A x): x [rows][n_in]
    fp32/bf16, dy [rows][n_out] fp32, A [r][n_in], B [n_out][r] fp32.
    Returns (dA, dB) fp32."""
    _req(x, "x", (torch.float32, torch.bfloat16))
    _req(A, "A", (torch.float32,))
    r, n_in = A.shape
    rows = x.numel() // n_in
    _req(x, "x", (x.dtype,), (rows, n_in))
    _req(B, "B", (torch.float32,))
    n_out = B.shape[0]
    _req(B, "B", (torch.float32,), (n_out, r))
    _req(dy, "dy", (torch.float32,), (rows, n_out))
    dA = torch.empty_like(A) if dA is None else dA
    dB = torch.empty_like(B) if dB is None else dB
    _req(dA, "dA", (torch.float32,), A.shape)
    _req(dB, "dB", (torch.float32,), B.shape)
    need = lora_bwd_workspace_bytes(rows, r)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _req(workspace, "workspace", (torch.uint8,))
    _b.check(library().lora_bwd(_p(x), _DT[x.dtype], _p(dy), _p(A), _p(B), _p(dA), _p(dB), rows, n_in, n_out, r,
                                float(scale), _p(workspace), workspace.numel(), _s(stream)), "lora_bwd")
    return dA, dB


def attn_bwd_decode(q, k, v, dout, scale=None, rope_base=0.0, q_pos=-1, dq=None, dk=None, dv=None,
                    stream=None):
    """One query per sequence over a KV cache with grouped KV heads.
    q, dout [B][Hq][D] fp32; k, v [B][S][Hkv][D] fp32/bf16.
    Returns (dq [B][Hq][D], dk, dv [B][S][Hkv][D]) fp32."""
    _req(q, "q", (torch.float32,))
    B, Hq, D = q.shape
    _req(k, "k", (torch.float32, torch.bfloat16))
    _, S, Hkv, _ = k.shape
    _req(k, "k", (k.dtype,), (B, S, Hkv, D))
    _req(v, "v", (k.dtype,), (B, S, Hkv, D))
    _req(dout, "dout", (torch.float32,), (B, Hq, D))
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty(k.shape, dtype=torch.float32, device=k.device) if dk is None else dk
    dv = torch.empty(v.shape, dtype=torch.float32, device=v.device) if dv is None else dv
    _req(dq, "dq", (torch.float32,), q.shape)
    _req(dk, "dk", (torch.float32,), k.shape)
    _req(dv, "dv", (torch.float32,), v.shape)
    _b.check(library().attn_bwd_decode(_p(q), _p(k), _p(v), _p(dout), _p(dq), _p(dk), _p(dv), B, Hq, Hkv, S, D,
                                       _DT[k.dtype], float(scale), float(rope_base), int(q_pos), _s(stream)),
             "attn_bwd_decode")
    return dq, dk, dv


def attn_fwd_causal(q, k, v, scale=None, o=None, lse=None, stream=None):
    """Causal attention forward: q [B][T][Hq][D], k, v [B][T][Hkv][D] bf16.
    Returns (o [B][T][Hq][D] bf16, lse [B][Hq][T] fp32), the activations
    attn_bwd_causal consumes."""
    bf = (torch.bfloat16,)
    _req(q, "q", bf)
    B, T, Hq, D = q.shape
    _req(k, "k", bf)
    Hkv = k.shape[2]
    _req(k, "k", bf, (B, T, Hkv, D))
    _req(v, "v", bf, (B, T, Hkv, D))
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty(B, Hq, T, dtype=torch.float32, device=q.device) if lse is None else lse
    _req(o, "o", bf, q.shape)
    _req(lse, "lse", (torch.float32,), (B, Hq, T))
    _b.check(library().attn_fwd_causal(_p(q), _p(k), _p(v), _p(o), _p(lse), B, T, Hq, Hkv, D, float(scale),
                                       _s(stream)), "attn_fwd_causal")
    return o, lse


def attn_bwd_causal_workspace_bytes(B, T, Hq, D) -> int:
    return int(library().attn_bwd_causal_workspace_bytes(B, T, Hq, D))


def attn_bwd_causal(q, k, v, o, dout, lse, scale=None, rope_base=0.0, pos0=0, dq=None, dk=None, dv=None,
                    workspace=None, stream=None):
    """Causal attention backward.  q, o, dout [B][T][Hq][D] bf16; k, v
    [B][T][Hkv][D] bf16; lse [B][Hq][T] fp32.  Returns fp32 (dq, dk, dv)."""
    bf = (torch.bfloat16,)
    _req(q, "q", bf)
    B, T, Hq, D = q.shape
    _req(k, "k", bf)
    Hkv = k.shape[2]
    _req(k, "k", bf, (B, T, Hkv, D))
    _req(v, "v", bf, (B, T, Hkv, D))
    _req(o, "o", bf, q.shape)
    _req(dout, "dout", bf, q.shape)
    _req(lse, "lse", (torch.float32,), (B, Hq, T))
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    dq = torch.empty(q.shape, dtype=torch.float32, device=q.device) if dq is None else dq
    dk = torch.empty(k.shape, dtype=torch.float32, device=k.device) if dk is None else dk
    dv = torch.empty(v.shape, dtype=torch.float32, device=v.device) if dv is None else dv
    _req(dq, "dq", (torch.float32,), q.shape)
    _req(dk, "dk", (torch.float32,), k.shape)
    _req(dv, "dv", (torch.float32,), v.shape)
    need = attn_bwd_causal_workspace_bytes(B, T, Hq, D)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _req(workspace, "workspace", (torch.uint8,))
    _b.check(library().attn_bwd_causal(_p(q), _p(k), _p(v), _p(o), _p(dout), _p(lse), _p(dq), _p(dk), _p(dv),
                                       B, T, Hq, Hkv, D, float(scale), float(rope_base), int(pos0),
                                       _p(workspace), workspace.numel(), _s(stream)),
             "attn_bwd_causal")
    return dq, dk, dv


def attn_bwd_causal_saved_p(q, k, v, p_attn, o, dout, scale=None, rope_base=0.0, pos0=0, dq=None, dk=None, dv=None,
                            workspace=None, stream=None):
    """Causal attention backward from the saved attention weights p_attn
    [B][Hq][T][T] bf16 (row = query) instead of the log-sum-exp.  q, o, dout
    [B][T][Hq][D] bf16; k, v [B][T][Hkv][D] bf16.  Returns fp32 (dq, dk, dv)."""
    bf = (torch.bfloat16,)
    _req(q, "q", bf)
    B, T, Hq, D = q.shape
    _req(k, "k", bf)
    Hkv = k.shape[2]
    _req(k, "k", bf, (B, T, Hkv, D))
    _req(v, "v", bf, (B, T, Hkv, D))
    _req(p_attn, "p_attn", bf, (B, Hq, T, T))
    _req(o, "o", bf, q.shape)
    _req(dout, "dout", bf, q.shape)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    dq = torch.empty(q.shape, dtype=torch.float32, device=q.device) if dq is None else dq
    dk = torch.empty(k.shape, dtype=torch.float32, device=k.device) if dk is None else dk
    dv = torch.empty(v.shape, dtype=torch.float32, device=v.device) if dv is None else dv
    _req(dq, "dq", (torch.float32,), q.shape)
    _req(dk, "dk", (torch.float32,), k.shape)
    _req(dv, "dv", (torch.float32,), v.shape)
    need = attn_bwd_causal_workspace_bytes(B, T, Hq, D)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _req(workspace, "workspace", (torch.uint8,))
    _b.check(library().attn_bwd_causal_saved_p(_p(q), _p(k), _p(v), _p(p_attn), _p(o), _p(dout), _p(dq), _p(dk),
                                               _p(dv), B, T, Hq, Hkv, D, float(scale), float(rope_base), int(pos0),
                                               _p(workspace), workspace.numel(), _s(stream)),
             "attn_bwd_causal_saved_p")
    return dq, dk, dv


# --------------------------------------------------------------------------
# Per-head norm with rotation, and linear attention
#
# A call on a few tokens takes the GPU some microseconds, so what the host
# does for it counts: one pass of checks per tensor (the reason is looked for
# only when one fails), the raw stream handle, cached workspace sizes.
# --------------------------------------------------------------------------
_BF16, _F32 = torch.bfloat16, torch.float32
_lib = None

# torch's own entries, some microseconds a call cheaper than the public functions
# that stand in for them in a torch that lacks them.
_PUBLIC = {
    "_cuda_getCurrentRawStream": lambda index: torch.cuda.current_stream(index).cuda_stream,
    "_cuda_getDevice": torch.cuda.current_device,
    "_cuda_cudaCachingAllocator_raw_alloc": lambda size, stream: torch.cuda.caching_allocator_alloc(size, stream=stream),
    "_cuda_cudaCachingAllocator_raw_delete": torch.cuda.caching_allocator_delete,
}
_raw_stream, _device_index, _raw_alloc, _raw_delete = (getattr(torch._C, name, public) for name, public in _PUBLIC.items())


def _fns():
    global _lib
    if _lib is None:
        _lib = library()
    return _lib


def _dense(t, name, dt, shape, dev):
    """Checks a dense tensor and returns its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dt and t.shape == shape and t.device == dev
            and t.is_contiguous()):
        _req(t, name, (dt,), shape)
        raise ValueError(f"{name} is on {t.device}, other tensors on {dev}")
    return t.data_ptr()


def _first(t, name, dim, dtypes):
    """Checks what the first tensor of a call decides: type, rank, device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} dtype {t.dtype} not in {dtypes}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} axes, not {t.dim()}")
    return t.device


def _rows(t, name, dt, shape, dev):
    """Checks a [B][T][H][D] tensor whose tokens may be apart (a part of a
    packed projection) and returns its token stride in elements, 0 if dense."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dt and t.shape == shape and t.device == dev):
        if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dt and t.shape == shape:
            raise ValueError(f"{name} is on {t.device}, other tensors on {dev}")
        _req(t.contiguous() if isinstance(t, torch.Tensor) else t, name, (dt,), shape)
    if t.is_contiguous():
        return 0
    B, T, H, D = shape
    sb, st, sh, sd = t.stride()
    token = st if T > 1 else sb
    if (D > 1 and sd != 1) or (H > 1 and sh != D) or (B > 1 and T > 1 and sb != T * st) or token < H * D:
        raise ValueError(f"{name} must have dense [H][D] rows at one stride from token to token")
    return token


def _empty(shape, dtype, device, stream):
    """Memory for the launch stream (the caching allocator reuses a block in
    the order of the stream it was allocated on)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _call(op, fn, dev, stream, need, workspace, *args):
    """Launches on the tensors' device, on `stream` or its current stream.
    `need` bytes of workspace, where the caller gave none, are held for the
    launch alone: the caching allocator hands them out again in that stream's
    order."""
    index = dev.index
    if stream is None:
        handle = _raw_stream(index)
    elif stream.device == dev:
        handle = stream.cuda_stream
    else:
        raise ValueError(f"{op}: stream on {stream.device}, tensors on {dev}")
    if index != _device_index():
        with torch.cuda.device(dev):
            return _call(op, fn, dev, stream, need, workspace, *args)
    if need is None:
        status = fn(*args, handle)
    elif workspace is not None:
        at = _dense(workspace, "workspace", torch.uint8, getattr(workspace, "shape", ()), dev)
        status = fn(*args, at, workspace.numel(), handle)
    elif need == 0:
        status = fn(*args, None, 0, handle)
    else:
        at = _raw_alloc(need, handle)
        try:
            status = fn(*args, at, need, handle)
        finally:
            _raw_delete(at)
    if status:
        _b.check(status, op)


def _int32(x, name):
    """x as the C int it becomes (ctypes would wrap it without a word)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name}={x} does not fit 32 bits")
    return x


def _rotation(B, T, D, rope_base, rotary_dim, positions, sections, pos0, dev):
    """(rotary_dim, address of the positions, axes, sections as a host array,
    pos0)."""
    if not rope_base:
        return 0, None, 1, None, 0
    axes, host = 1, None
    if sections is not None:
        axes = len(sections)
        host = (ctypes.c_int * axes)(*(_int32(n, "sections") for n in sections))
    at = None
    if positions is not None:
        flat = axes == 1 and isinstance(positions, torch.Tensor) and positions.dim() == 2
        at = _dense(positions, "positions", torch.int32, (B, T) if flat else (axes, B, T), dev)
    return D if rotary_dim is None else _int32(rotary_dim, "rotary_dim"), at, axes, host, _int32(pos0, "pos0")


def qk_norm_rope_fwd(q, k, gamma_q=None, gamma_k=None, eps=1e-6, rope_base=0.0, rotary_dim=None, interleaved=True,
                     positions=None, sections=None, pos0=0, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head (gamma_q, gamma_k [D] fp32; None:
    no norm) and the rotation of its first ``rotary_dim`` components (all, if
    None; rope_base 0: none).  q [B][T][Hq][D], k [B][T][Hkv][D] or None,
    fp32 or bf16, possibly parts of a packed projection.  positions
    [axes][B][T] int32 (None: pos0 + t); ``sections`` gives each axis its
    number of pairs.  Returns dense (q_out, k_out) of the inputs' dtype."""
    dev = _first(q, "q", 4, (_F32, _BF16))
    dt, qshape = q.dtype, q.shape
    B, T, Hq, D = qshape
    qs = _rows(q, "q", dt, qshape, dev)
    if q_out is None:
        q_out = _empty(qshape, dt, dev, stream)
        qo = q_out.data_ptr()
    else:
        qo = _dense(q_out, "q_out", dt, qshape, dev)
    Hkv = ks = 0
    kp = ko = None
    if k is not None:
        Hkv = k.shape[2] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
        kshape = (B, T, Hkv, D)
        ks = _rows(k, "k", dt, kshape, dev)
        kp = k.data_ptr()
        if k_out is None:
            k_out = _empty(kshape, dt, dev, stream)
            ko = k_out.data_ptr()
        else:
            ko = _dense(k_out, "k_out", dt, kshape, dev)
    else:
        k_out = None
    gq = None if gamma_q is None else _dense(gamma_q, "gamma_q", _F32, (D,), dev)
    gk = None if gamma_k is None else _dense(gamma_k, "gamma_k", _F32, (D,), dev)
    R, pos, axes, host, pos0 = _rotation(B, T, D, rope_base, rotary_dim, positions, sections, pos0, dev)
    _call("qk_norm_rope_fwd", _fns().qk_norm_rope_fwd, dev, stream, None, None, q.data_ptr(), kp, _DT[dt], gq, gk, qo,
          ko, B, T, Hq, Hkv, D, qs, ks, float(eps), float(rope_base), R, 1 if interleaved else 0, pos, axes, host,
          pos0)
    return q_out, k_out


@functools.lru_cache(maxsize=None)
def qk_norm_rope_bwd_workspace_bytes(D) -> int:
    return int(library().qk_norm_rope_bwd_workspace_bytes(D))


def qk_norm_rope_bwd(q, k, dq_out, dk_out, gamma_q=None, gamma_k=None, eps=1e-6, rope_base=0.0, rotary_dim=None,
                     interleaved=True, positions=None, sections=None, pos0=0, dq=None, dk=None, dgamma_q=None,
                     dgamma_k=None, workspace=None, stream=None):
    """Gradients of qk_norm_rope_fwd.  dq_out, dk_out are dense, fp32 or bf16
    (the same for both).  dq, dk have the inputs' dtype and may be parts of a
    packed gradient.  Returns (dq, dk, dgamma_q, dgamma_k), None where there
    is no k or no gamma."""
    dts = (_F32, _BF16)
    dev = _first(q, "q", 4, dts)
    _first(dq_out, "dq_out", 4, dts)
    dt, yt, qshape = q.dtype, dq_out.dtype, q.shape
    B, T, Hq, D = qshape
    qs = _rows(q, "q", dt, qshape, dev)
    yq = _dense(dq_out, "dq_out", yt, qshape, dev)
    dqs = 0
    if dq is None:
        dq = _empty(qshape, dt, dev, stream)
    else:
        dqs = _rows(dq, "dq", dt, qshape, dev)
    Hkv = ks = dks = 0
    kp = yk = dkp = gq = gk = dgq = dgk = None
    if k is not None:
        Hkv = k.shape[2] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
        kshape = (B, T, Hkv, D)
        ks = _rows(k, "k", dt, kshape, dev)
        yk = _dense(dk_out, "dk_out", yt, kshape, dev)
        if dk is None:
            dk = _empty(kshape, dt, dev, stream)
        else:
            dks = _rows(dk, "dk", dt, kshape, dev)
        kp, dkp = k.data_ptr(), dk.data_ptr()
    else:
        dk = gamma_k = None
    if gamma_q is not None:
        gq = _dense(gamma_q, "gamma_q", _F32, (D,), dev)
        if dgamma_q is None:
            dgamma_q = _empty((D,), _F32, dev, stream)
            dgq = dgamma_q.data_ptr()
        else:
            dgq = _dense(dgamma_q, "dgamma_q", _F32, (D,), dev)
    else:
        dgamma_q = None
    if gamma_k is not None:
        gk = _dense(gamma_k, "gamma_k", _F32, (D,), dev)
        if dgamma_k is None:
            dgamma_k = _empty((D,), _F32, dev, stream)
            dgk = dgamma_k.data_ptr()
        else:
            dgk = _dense(dgamma_k, "dgamma_k", _F32, (D,), dev)
    else:
        dgamma_k = None
    R, pos, axes, host, pos0 = _rotation(B, T, D, rope_base, rotary_dim, positions, sections, pos0, dev)
    need = qk_norm_rope_bwd_workspace_bytes(D) if gq or gk else 0
    _call("qk_norm_rope_bwd", _fns().qk_norm_rope_bwd, dev, stream, need, workspace, q.data_ptr(), kp, _DT[dt], yq, yk,
          _DT[yt], gq, gk, dq.data_ptr(), dkp, dgq, dgk, B, T, Hq, Hkv, D, qs, ks, dqs, dks, float(eps),
          float(rope_base), R, 1 if interleaved else 0, pos, axes, host, pos0)
    return dq, dk, dgamma_q, dgamma_k


@functools.lru_cache(maxsize=1024)
def lin_attn_fwd_workspace_bytes(B, T, Hkv, D) -> int:
    return int(library().lin_attn_fwd_workspace_bytes(B, T, Hkv, D))


@functools.lru_cache(maxsize=1024)
def lin_attn_bwd_workspace_bytes(B, T, Hkv, D) -> int:
    return int(library().lin_attn_bwd_workspace_bytes(B, T, Hkv, D))


def _lin_inputs(q, k, v, log_decay, initial_state, lengths):
    """Checks what both directions take: (device, sizes, [B][T][Hkv][D],
    [B][Hkv][D][D], strides, addresses)."""
    dev = _first(q, "q", 4, (_BF16,))
    _first(k, "k", 4, (_BF16,))
    qshape = q.shape
    B, T, Hq, D = qshape
    Hkv = k.shape[2]
    kshape, sshape = (B, T, Hkv, D), (B, Hkv, D, D)
    strides = (_rows(q, "q", _BF16, qshape, dev), _rows(k, "k", _BF16, kshape, dev), _rows(v, "v", _BF16, kshape, dev))
    at = (q.data_ptr(), k.data_ptr(), v.data_ptr(), _dense(log_decay, "log_decay", _F32, (Hkv,), dev),
          None if initial_state is None else _dense(initial_state, "initial_state", _F32, sshape, dev),
          None if lengths is None else _dense(lengths, "lengths", torch.int32, (B,), dev))
    return dev, (B, T, Hq, Hkv, D), kshape, sshape, strides, at


def lin_attn_fwd(q, k, v, log_decay, scale=None, initial_state=None, lengths=None, want_final_state=False, o=None,
                 final_state=None, workspace=None, stream=None):
    """Causal linear attention with a decay for each KV head: S = a S + k v^T,
    o = scale S^T q, a = exp(log_decay).  q [B][T][Hq][D], k, v
    [B][T][Hkv][D] bf16 (possibly parts of a packed projection), log_decay
    [Hkv] fp32 <= 0, initial_state [B][Hkv][D][D] fp32 or None, lengths [B]
    int32 or None (tokens of each sequence; o is 0 behind them).  Returns
    (o [B][T][Hq][D] bf16, final_state fp32 or None); final_state may be the
    initial_state tensor."""
    dev, dims, _, sshape, strides, (qp, kp, vp, ldp, s0, ln) = _lin_inputs(q, k, v, log_decay, initial_state, lengths)
    B, T, Hq, Hkv, D = dims
    os = 0
    if o is None:
        o = _empty(q.shape, _BF16, dev, stream)
    else:
        os = _rows(o, "o", _BF16, q.shape, dev)
    if final_state is None and want_final_state:
        final_state = _empty(sshape, _F32, dev, stream)
    fin = None if final_state is None else _dense(final_state, "final_state", _F32, sshape, dev)
    _call("lin_attn_fwd", _fns().lin_attn_fwd, dev, stream, lin_attn_fwd_workspace_bytes(B, T, Hkv, D), workspace, qp,
          kp, vp, ldp, s0, ln, o.data_ptr(), fin, *dims, *strides, os,
          1.0 / math.sqrt(D) if scale is None else float(scale))
    return o, final_state


def lin_attn_bwd(q, k, v, dout, log_decay, scale=None, initial_state=None, dfinal_state=None, lengths=None,
                 want_dinitial_state=False, dq=None, dk=None, dv=None, dinitial_state=None, workspace=None,
                 stream=None):
    """Gradients of lin_attn_fwd: dout [B][T][Hq][D] bf16, dfinal_state
    [B][Hkv][D][D] fp32 or None.  Returns (dq, dk, dv) bf16 (given ones may be
    parts of a packed gradient) and dinitial_state fp32 or None."""
    dev, dims, kshape, sshape, strides, at = _lin_inputs(q, k, v, log_decay, initial_state, lengths)
    qp, kp, vp, ldp, s0, ln = at
    B, T, Hq, Hkv, D = dims
    dop = _dense(dout, "dout", _BF16, q.shape, dev)
    dfp = None if dfinal_state is None else _dense(dfinal_state, "dfinal_state", _F32, sshape, dev)
    outs = (0 if dq is None else _rows(dq, "dq", _BF16, q.shape, dev),
            0 if dk is None else _rows(dk, "dk", _BF16, kshape, dev),
            0 if dv is None else _rows(dv, "dv", _BF16, kshape, dev))
    dq = _empty(q.shape, _BF16, dev, stream) if dq is None else dq
    dk = _empty(kshape, _BF16, dev, stream) if dk is None else dk
    dv = _empty(kshape, _BF16, dev, stream) if dv is None else dv
    if dinitial_state is None and want_dinitial_state:
        dinitial_state = _empty(sshape, _F32, dev, stream)
    dsp = None if dinitial_state is None else _dense(dinitial_state, "dinitial_state", _F32, sshape, dev)
    _call("lin_attn_bwd", _fns().lin_attn_bwd, dev, stream, lin_attn_bwd_workspace_bytes(B, T, Hkv, D), workspace, qp,
          kp, vp, dop, ldp, s0, dfp, ln, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dsp, *dims, *strides, *outs,
          1.0 / math.sqrt(D) if scale is None else float(scale))
    return dq, dk, dv, dinitial_state


def lin_attn_decode(q, k, v, state, log_decay, scale=None, slots=None, o=None, stream=None):
    """One token per sequence of lin_attn_fwd's recurrence: q [B][Hq][D], k, v
    [B][Hkv][D] fp32 or bf16; state [n][Hkv][D][D] fp32 is updated in place.
    slots [B] int32 or None: row b works on state slots[b] (None: b); a row
    whose slot is outside 0 .. n - 1 is empty (o 0, no state touched).
    Returns o [B][Hq][D] of q's dtype."""
    dev = _first(q, "q", 3, (_F32, _BF16))
    dt, qshape = q.dtype, q.shape
    B, Hq, D = qshape
    Hkv = k.shape[1] if isinstance(k, torch.Tensor) and k.dim() == 3 else 0
    n = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() == 4 else 0
    kshape = (B, Hkv, D)
    qp, kp, vp = (_dense(q, "q", dt, qshape, dev), _dense(k, "k", dt, kshape, dev), _dense(v, "v", dt, kshape, dev))
    sp, lp = _dense(state, "state", _F32, (n, Hkv, D, D), dev), _dense(log_decay, "log_decay", _F32, (Hkv,), dev)
    sl = None if slots is None else _dense(slots, "slots", torch.int32, (B,), dev)
    if o is None:
        o = _empty(qshape, dt, dev, stream)
        op = o.data_ptr()
    else:
        op = _dense(o, "o", dt, qshape, dev)
    _call("lin_attn_decode", _fns().lin_attn_decode, dev, stream, None, None, qp, kp, vp, _DT[dt], sp, lp, sl, op, B,
          Hq, Hkv, D, n, 1.0 / math.sqrt(D) if scale is None else float(scale))
    return o
