"""Refusals of the windowed attention and of the paged cache's calls, through
the C ABI: every one is answered on the host, before any launch."""
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
    return raw, (raw.ctypes.data + 255) & ~255


def p(mem, off):
    return None if mem is None or off is None else ctypes.c_void_p(mem[1] + off)


def fwd(lib, mem=None, T=16, Hq=4, Hkv=2, D=64, qs=0, os=0, window=8, sinks=0, scale=0.1, q=0, k=16384, o=32768, lse=65536,
        Bn=1, lengths=None):
    return lib.attn_fwd_window(p(mem, q), p(mem, k), p(mem, 24576), p(mem, lengths), p(mem, o), p(mem, lse), Bn, T, Hq, Hkv, D,
                               qs, 0, 0, os, window, sinks, scale, None)


def test_attn_fwd_window_refusals(lib, mem):
    assert fwd(lib, D=96) == B.ENOTSUP
    assert fwd(lib, Hkv=3) == B.EINVAL
    assert fwd(lib, Hkv=0) == B.EINVAL
    assert fwd(lib, Hq=0) == B.EINVAL
    assert fwd(lib, T=-1) == B.EINVAL
    assert fwd(lib, window=0) == B.EINVAL and "window" in B.last_error()
    assert fwd(lib, window=-3) == B.EINVAL
    assert fwd(lib, sinks=-1) == B.EINVAL
    assert fwd(lib, scale=float("nan")) == B.EINVAL
    assert fwd(lib, qs=-8) == B.EINVAL
    assert fwd(lib) == B.EINVAL and "NULL" in B.last_error()
    assert fwd(lib, T=0) == B.OK and fwd(lib, Bn=0) == B.OK
    assert fwd(lib, mem, qs=260) == B.ENOTSUP                              # 520 bytes: not a multiple of 16
    assert fwd(lib, mem, qs=128) == B.EINVAL and "stride" in B.last_error()
    assert fwd(lib, mem, q=8) == B.EINVAL
    assert fwd(lib, mem, o=64) == B.EINVAL and "overlaps" in B.last_error()
    assert fwd(lib, mem, lse=32832) == B.EINVAL and "overlap" in B.last_error()
    assert fwd(lib, mem, lse=65538) == B.EINVAL
    assert fwd(lib, mem, lengths=2) == B.EINVAL


def bwd(lib, mem=None, T=16, Hq=4, Hkv=2, D=64, window=8, sinks=0, dks=0, dk=120000 // 16 * 16, dq=98304, ws=200000 // 256 * 256,
        need=None):
    need = lib.attn_bwd_window_workspace_bytes(1, T, Hq, Hkv, D, window, sinks) if need is None else need
    a = lambda x: p(mem, x)
    return lib.attn_bwd_window(a(0), a(16384), a(24576), a(32768), a(49152), a(65536), None, a(dq), a(dk), a(140000 // 16 * 16),
                               1, T, Hq, Hkv, D, 0, 0, 0, 0, 0, dks, 0, window, sinks, 0.1, a(ws), need, None)


def test_attn_bwd_window_refusals(lib, mem):
    size = lib.attn_bwd_window_workspace_bytes
    assert size(1, 16, 4, 2, 64, 8, 0) > 0
    for bad in [(0, 16, 4, 2, 64, 8, 0), (1, -1, 4, 2, 64, 8, 0), (1, 16, 5, 2, 64, 8, 0), (1, 16, 4, 0, 64, 8, 0),
                (1, 16, 4, 2, 80, 8, 0), (1, 16, 4, 2, 64, 0, 0), (1, 16, 4, 2, 64, 8, -1)]:
        assert size(*bad) == 0
    assert bwd(lib, D=32) == B.ENOTSUP
    assert bwd(lib, Hkv=3) == B.EINVAL
    assert bwd(lib, window=0) == B.EINVAL
    assert bwd(lib, sinks=-1) == B.EINVAL
    assert bwd(lib, dks=-8) == B.EINVAL
    assert bwd(lib, T=0) == B.OK
    assert bwd(lib) == B.EWORKSPACE
    assert bwd(lib, mem, need=size(1, 16, 4, 2, 64, 8, 0) - 1) == B.EWORKSPACE
    assert bwd(lib, mem, dk=98304 + 64) == B.EINVAL and "overlap" in B.last_error()
    assert bwd(lib, mem, dq=0) == B.EINVAL and "overlaps" in B.last_error()


def write(lib, mem=None, Bn=2, T=4, Hkv=2, D=64, n=4, page=8, most=2, ks=0, k=0, kp=16384, vp=65536, table=200000 // 16 * 16,
          starts=210000 // 16 * 16):
    return lib.kv_pages_write(p(mem, k), p(mem, 8192), p(mem, kp), p(mem, vp), p(mem, table), p(mem, starts), None, Bn, T, Hkv,
                              D, n, page, most, ks, 0, None)


def test_kv_pages_write_refusals(lib, mem):
    assert write(lib, Bn=-1) == B.EINVAL and write(lib, T=-1) == B.EINVAL and write(lib, n=-1) == B.EINVAL
    assert write(lib, most=-1) == B.EINVAL
    assert write(lib, page=0) == B.EINVAL and "page_size" in B.last_error()
    assert write(lib, page=1 << 20, most=1 << 11) == B.ENOTSUP
    assert write(lib, D=68) == B.ENOTSUP and write(lib, D=0) == B.ENOTSUP
    assert write(lib, ks=-8) == B.EINVAL
    assert write(lib) == B.EINVAL and "NULL" in B.last_error()
    assert write(lib, T=0) == B.OK and write(lib, Bn=0) == B.OK
    assert write(lib, mem, n=0) == B.OK                                    # no page: nothing to write
    assert write(lib, mem, ks=64) == B.EINVAL                              # below a row of 2 x 64
    assert write(lib, mem, ks=132) == B.ENOTSUP
    assert write(lib, mem, kp=16392) == B.EINVAL
    assert write(lib, mem, vp=16384) == B.EINVAL and "overlap" in B.last_error()
    assert write(lib, mem, k=16384) == B.EINVAL and "overlaps" in B.last_error()
    assert write(lib, mem, starts=210002) == B.EINVAL


def decode(lib, mem=None, dt=1, Bn=2, Hq=4, Hkv=2, D=64, n=4, page=8, most=2, window=0, sinks=0, scale=0.1, q=0, o=8192,
           sums=None, need=None, ws=300000 // 16 * 16):
    need = 1 << 30 if need is None else need
    return lib.attn_decode_paged(p(mem, q), dt, p(mem, 16384), p(mem, 65536), p(mem, 131072), p(mem, 140000 // 16 * 16),
                                 p(mem, sums), p(mem, o), Bn, Hq, Hkv, D, n, page, most, window, sinks, scale, p(mem, ws), need,
                                 None)


def test_tables_end_where_positions_leave_32_bits(lib, mem):
    """The walks over positions step past the last one by up to a block's
    stretch of them; 2^31 - 2^16 positions leave the room for it."""
    for most in (0x7fff0001, 0x7fffffff):
        assert decode(lib, page=1, most=most) == B.ENOTSUP and write(lib, page=1, most=most) == B.ENOTSUP
        assert evict(lib, page=1, most=most) == B.ENOTSUP and evict(lib, page=1, fresh=most) == B.ENOTSUP
    most = 0x7fff0000                                                       # on to the next check: NULL
    assert decode(lib, page=1, most=most) == B.EWORKSPACE and write(lib, page=1, most=most) == B.EINVAL
    assert evict(lib, page=1, most=most) == B.EINVAL and evict(lib, page=1, fresh=most) == B.EINVAL


def test_attn_decode_paged_refusals(lib, mem):
    size = lib.attn_decode_paged_workspace_bytes
    assert decode(lib, D=32) == B.ENOTSUP and decode(lib, D=256) == B.ENOTSUP
    assert decode(lib, Hq=5) == B.EINVAL and decode(lib, Hkv=0) == B.EINVAL and decode(lib, Hq=0) == B.EINVAL
    assert decode(lib, dt=7) == B.EINVAL
    assert decode(lib, page=0) == B.EINVAL and decode(lib, n=-1) == B.EINVAL and decode(lib, most=-2) == B.EINVAL
    assert decode(lib, page=1 << 16, most=1 << 15) == B.ENOTSUP
    assert decode(lib, window=-1) == B.EINVAL and decode(lib, sinks=-1) == B.EINVAL
    assert decode(lib, scale=float("nan")) == B.EINVAL
    assert decode(lib, Bn=0) == B.OK
    assert decode(lib) == B.EWORKSPACE
    need = size(2, 4, 2, 64, 8, 2, 0, 0, 0)
    assert need > 0 and decode(lib, mem, need=need - 1) == B.EWORKSPACE
    assert size(2, 4, 2, 64, 8, 2, 0, 0, 1) > need
    assert size(2, 4, 2, 64, 8, 1000, 100, 4, 1) < size(2, 4, 2, 64, 8, 1000, 0, 0, 1)   # no more scores than a window
    for bad in [(0, 4, 2, 64, 8, 2, 0, 0, 0), (2, 5, 2, 64, 8, 2, 0, 0, 0), (2, 4, 0, 64, 8, 2, 0, 0, 0),
                (2, 4, 2, 65, 8, 2, 0, 0, 0), (2, 4, 2, 64, 0, 2, 0, 0, 0), (2, 4, 2, 64, 8, 2, -1, 0, 0)]:
        assert size(*bad) == 0
    assert decode(lib, mem, o=64) == B.EINVAL and "overlaps" in B.last_error()
    assert decode(lib, mem, o=8200) == B.EINVAL
    assert decode(lib, mem, sums=16384) == B.EINVAL and "overlaps" in B.last_error()
    assert decode(lib, mem, ws=8192) == B.EINVAL


def evict(lib, mem=None, Bn=2, Hkv=2, D=64, n=4, page=8, most=2, fresh=1, budget=8, sinks=2, recent=3, kept=210000 // 16 * 16,
          new_n=220000 // 16 * 16, lengths=140000 // 16 * 16):
    return lib.kv_pages_evict(p(mem, 16384), p(mem, 65536), p(mem, 131072), p(mem, lengths), p(mem, 150000 // 16 * 16),
                              p(mem, 160000 // 16 * 16), p(mem, kept), p(mem, new_n), p(mem, 230000 // 16 * 16), Bn, Hkv, D, n,
                              page, most, fresh, budget, sinks, recent, None)


def test_kv_pages_evict_refusals(lib, mem):
    assert evict(lib, D=60) == B.ENOTSUP
    assert evict(lib, Hkv=0) == B.EINVAL and evict(lib, Bn=-1) == B.EINVAL and evict(lib, page=0) == B.EINVAL
    assert evict(lib, budget=0, sinks=0, recent=0) == B.EINVAL
    assert evict(lib, sinks=-1) == B.EINVAL and evict(lib, recent=-1) == B.EINVAL
    assert evict(lib, sinks=6) == B.EINVAL and "hold" in B.last_error()     # 6 + 3 > 8
    assert evict(lib, sinks=0x7fffffff, recent=0x7fffffff) == B.EINVAL
    assert evict(lib, budget=9) == B.EINVAL and "new_table" in B.last_error()
    assert evict(lib, fresh=-1) == B.EINVAL and evict(lib, most=1 << 30) == B.ENOTSUP
    assert evict(lib) == B.EINVAL and "NULL" in B.last_error()
    assert evict(lib, Bn=0) == B.OK
    assert evict(lib, mem, kept=150000 // 16 * 16) == B.EINVAL and "overlaps" in B.last_error()
    assert evict(lib, mem, new_n=140000 // 16 * 16) == B.EINVAL             # lengths in place
    assert evict(lib, mem, kept=210002) == B.EINVAL
