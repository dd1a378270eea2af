"""Refusals of the per-head norm with rotation and of the linear attention,
through the C ABI: every one is answered on the host, before any launch."""
import ctypes

import numpy as np
import pytest

from transformer_attention_backward_gb300 import _binding as B


@pytest.fixture(scope="module")
def lib():
    return B.load()


@pytest.fixture(scope="module")
def mem():
    """One aligned host buffer: addresses for checks that never dereference."""
    raw = np.zeros(1 << 20, dtype=np.uint8)
    at = (raw.ctypes.data + 255) & ~255
    return raw, at


def p(mem, off):
    return ctypes.c_void_p(mem[1] + off)


def sections(*n):
    return (ctypes.c_int * len(n))(*n)


def qk_fwd(lib, mem=None, dt=1, T=4, Hq=2, Hkv=1, D=16, qs=0, ks=0, eps=1e-6, base=100.0, rot=16, axes=1, sec=None,
           q=0, k=4096, qo=8192, ko=12288):
    a = [None] * 4 if mem is None else [p(mem, x) for x in (q, k, qo, ko)]
    return lib.qk_norm_rope_fwd(a[0], a[1], dt, None, None, a[2], a[3], 1, T, Hq, Hkv, D, qs, ks, eps, base, rot, 1,
                                None, axes, sec, 0, None)


def test_qk_norm_rope_fwd_refusals(lib, mem):
    assert qk_fwd(lib, D=15, rot=14) == B.EINVAL
    assert qk_fwd(lib, D=514) == B.ENOTSUP
    assert qk_fwd(lib, dt=5) == B.EINVAL
    assert qk_fwd(lib, eps=-1.0) == B.EINVAL
    assert qk_fwd(lib, eps=float("nan")) == B.EINVAL
    assert qk_fwd(lib, base=-1.0) == B.EINVAL
    assert qk_fwd(lib, base=float("nan")) == B.EINVAL
    assert qk_fwd(lib, base=float("inf")) == B.EINVAL
    for rot in (0, 3, 18):
        assert qk_fwd(lib, rot=rot) == B.EINVAL
    assert qk_fwd(lib, axes=0) == B.EINVAL
    assert qk_fwd(lib, axes=5, sec=sections(1, 1, 1, 1, 4)) == B.EINVAL
    assert qk_fwd(lib, axes=2) == B.EINVAL                                 # no sections
    assert qk_fwd(lib, axes=2, sec=sections(4, 3)) == B.EINVAL             # do not add up
    assert "add up" in B.last_error()
    assert qk_fwd(lib, axes=2, sec=sections(9, -1)) == B.EINVAL
    assert qk_fwd(lib, T=-1) == B.EINVAL
    assert qk_fwd(lib, qs=-32) == B.EINVAL
    assert qk_fwd(lib) == B.EINVAL and "NULL" in B.last_error()
    assert qk_fwd(lib, T=0) == B.OK
    assert qk_fwd(lib, mem, qs=16) == B.EINVAL and "stride" in B.last_error()   # below a row of 2 x 16
    assert qk_fwd(lib, mem, q=1) == B.EINVAL                               # half an element
    assert qk_fwd(lib, mem, qo=8200) == B.EINVAL                           # outputs are 16-byte aligned
    assert qk_fwd(lib, mem, qo=64) == B.EINVAL and "overlaps" in B.last_error()
    assert qk_fwd(lib, mem, ko=8192) == B.EINVAL


def qk_bwd(lib, mem, dq, dk, dqs, dks, ws=65536, need=None, gamma=True, T=4):
    need = lib.qk_norm_rope_bwd_workspace_bytes(16) if need is None else need
    g = p(mem, 32768) if gamma else None
    return lib.qk_norm_rope_bwd(p(mem, 0), p(mem, 64), 1, p(mem, 8192), p(mem, 12288), 0, g, g, p(mem, dq), p(mem, dk),
                                p(mem, 36864) if gamma else None, None, 1, T, 2, 1, 16, 48, 48, dqs, dks, 1e-6, 100.0,
                                16, 1, None, 1, None, 0, p(mem, ws) if ws else None, need, None)


def test_qk_norm_rope_bwd_refusals(lib, mem):
    need = lib.qk_norm_rope_bwd_workspace_bytes(16)
    assert need > 0 and lib.qk_norm_rope_bwd_workspace_bytes(0) == 0
    assert qk_bwd(lib, mem, 16384, 16448, 48, 48, ws=0) == B.EWORKSPACE
    assert qk_bwd(lib, mem, 16384, 16448, 48, 48, need=need - 1) == B.EWORKSPACE
    # rows of a packed gradient interleave; rows that share bytes do not pass
    assert qk_bwd(lib, mem, 16384, 16416, 48, 48) == B.EINVAL and "overlap" in B.last_error()
    assert qk_bwd(lib, mem, 16384, 16448, 48, 32) == B.EINVAL and "overlap" in B.last_error()
    assert qk_bwd(lib, mem, 0, 16448, 48, 48) == B.EINVAL                  # dq over q


def lin_fwd(lib, mem=None, T=130, Hq=4, Hkv=2, D=64, qs=0, os=0, scale=0.1, need=None, q=0, o=400000, fin=None, init=None):
    wsb = lib.lin_attn_fwd_workspace_bytes(1, T, Hkv, D) if need is None else need
    a = (lambda x: None if mem is None or x is None else p(mem, x))
    return lib.lin_attn_fwd(a(q), a(100000 // 16 * 16), a(160000), a(220000 // 16 * 16), a(init), None, a(o), a(fin), 1,
                            T, Hq, Hkv, D, qs, 0, 0, os, scale, a(600000 // 16 * 16) if mem else None, wsb, None)


def test_lin_attn_fwd_refusals(lib, mem):
    assert lin_fwd(lib, D=96) == B.ENOTSUP
    assert lin_fwd(lib, Hkv=3) == B.EINVAL
    assert lin_fwd(lib, Hkv=0) == B.EINVAL
    assert lin_fwd(lib, Hq=0) == B.EINVAL and "Hq=0" in B.last_error()    # keys would move the state
    assert lin_fwd(lib, T=-1, need=0) == B.EINVAL
    assert lin_fwd(lib, scale=float("nan")) == B.EINVAL
    assert lin_fwd(lib, qs=-8) == B.EINVAL
    assert lin_fwd(lib) == B.EWORKSPACE
    assert lin_fwd(lib, mem, need=100) == B.EWORKSPACE
    assert lin_fwd(lib, mem, qs=260) == B.ENOTSUP                          # 520 bytes: not a multiple of 16
    assert lin_fwd(lib, mem, qs=128) == B.EINVAL                           # below a row
    assert lin_fwd(lib, mem, q=8) == B.EINVAL
    assert lin_fwd(lib, mem, o=64) == B.EINVAL and "overlaps" in B.last_error()
    assert lin_fwd(lib, mem, fin=480000, init=480016) == B.EINVAL          # half in place
    assert lin_fwd(lib, mem, T=0) == B.OK                                  # nothing to do, no state
    assert lib.lin_attn_fwd_workspace_bytes(2, 300, 5, 128) == 2 * 5 * 3 * 128 * 128 * 2
    assert lib.lin_attn_bwd_workspace_bytes(2, 300, 5, 128) == 2 * lib.lin_attn_fwd_workspace_bytes(2, 300, 5, 128)
    assert lib.lin_attn_bwd_workspace_bytes(-1, 300, 5, 128) == 0


def test_lin_attn_bwd_refusals(lib):
    def call(D=64, Hkv=2, T=16, scale=0.1, dks=0, ws=None, Hq=4):
        return lib.lin_attn_bwd(None, None, None, None, None, None, None, None, None, None, None, None, 1, T, Hq, Hkv, D,
                                0, 0, 0, 0, dks, 0, scale, ws, 1 << 30, None)
    assert call(Hq=0) == B.EINVAL and "Hq=0" in B.last_error()
    assert call(D=32) == B.ENOTSUP
    assert call(Hkv=3) == B.EINVAL
    assert call(scale=float("nan")) == B.EINVAL
    assert call(dks=-8) == B.EINVAL
    assert call() == B.EWORKSPACE
    assert call(ws=ctypes.c_void_p(256)) == B.EINVAL and "NULL" in B.last_error()
    assert call(T=0) == B.EINVAL                                           # log_decay is wanted all the same


def test_lin_attn_decode_refusals(lib, mem):
    def call(D=64, Hq=4, Hkv=2, Bn=3, n=3, slots=None, dt=1, state=4096):
        return lib.lin_attn_decode(p(mem, 0), p(mem, 1536), p(mem, 2304), dt, p(mem, state), p(mem, 500000 // 16 * 16),
                                   slots, p(mem, 520000 // 16 * 16), Bn, Hq, Hkv, D, n, 0.1, None)
    assert call(D=256) == B.ENOTSUP
    assert call(Hq=18) == B.ENOTSUP                                        # group of 9
    assert call(Hq=5) == B.EINVAL
    assert call(Hq=0) == B.EINVAL
    assert call(dt=3) == B.EINVAL
    assert call(n=2) == B.EINVAL                                           # fewer states than rows, no slots
    assert call(n=-1) == B.EINVAL
    assert call(state=16) == B.EINVAL and "overlaps" in B.last_error()
    assert call(Bn=0, n=0) == B.OK
