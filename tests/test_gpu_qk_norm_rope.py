"""GPU parity of qk_norm_rope_fwd / _bwd (per-head norm and rotation in one
pass) against the float64 oracle.

Tolerance of one element: half a step of its type (2^-8 of its size in bf16)
for the one rounding on the way out, plus the fp32 arithmetic before it: a sum
of D squares (D 2^-24, halved by the root), the angle (2^-23) and some ten
products and sums of 2^-24 each, on values as large as the row's largest; the
backward takes two such sums and subtracts, so it gets three times that.
dgamma sums n rows in fp32: n 2^-24 of the sum of the terms' sizes at most."""
import numpy as np
import pytest
import torch

import oracle as O
from tests.helpers import to_np

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def abw():
    import transformer_attention_backward_gb300 as m
    m.library()
    return m


def close(got, ref, dtype, D, factor=1.0):
    g = to_np(got)
    assert g.shape == ref.shape and np.all(np.isfinite(g))
    if g.size == 0:
        return
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    row = np.max(np.abs(ref), axis=-1, keepdims=True)
    tol = half * np.abs(ref) + factor * (D / 2 + 16) * 2.0 ** -24 * 2 ** 0.5 * row
    bad = np.abs(g - ref) > tol
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(g - ref) / (tol + 1e-300))))


def inputs(seed, B, T, Hq, Hkv, D, dtype, axes=1, far=100, packed=True, dy=F):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(B, T, Hq + 2 * Hkv, D, generator=g).to(dtype)
    out = {"qkv": qkv, "gq": 1 + 0.1 * torch.randn(D, generator=g), "gk": 1 + 0.1 * torch.randn(D, generator=g),
           "pos": torch.randint(-far, far, (axes, B, T), generator=g, dtype=torch.int32),
           "dq": torch.randn(B, T, Hq, D, generator=g).to(dy), "dk": torch.randn(B, T, Hkv, D, generator=g).to(dy)}
    out["q"], out["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
    return out


def views(qkv, Hq, Hkv):
    d = qkv.cuda()
    return d[:, :, :Hq], d[:, :, Hq:Hq + Hkv]


def check(abw, B, T, Hq, Hkv, D, rot, sections, base, inter, dtype, dy, norm=(True, True), positions=True, pos0=0,
          eps=1e-6, far=100, seed=0):
    axes = 1 if sections is None else len(sections)
    t = inputs(seed, B, T, Hq, Hkv, D, dtype, axes, far, dy=dy)
    q, k = views(t["qkv"], Hq, Hkv)
    gq, gk = (t["gq"] if norm[0] else None), (t["gk"] if norm[1] else None)
    pos = t["pos"].numpy() if positions else np.broadcast_to(pos0 + np.arange(T), (axes, B, T))
    theta = O.section_angles(pos, rot, base, sections or [rot // 2]) if base else None
    how = dict(eps=eps, rope_base=base, rotary_dim=rot, interleaved=inter, pos0=pos0, sections=sections,
               positions=t["pos"].cuda() if positions else None)
    dev = lambda x: None if x is None else x.cuda()
    has_k = Hkv > 0
    y = abw.qk_norm_rope_fwd(q, k if has_k else None, dev(gq), dev(gk), **how)
    for got, x, g in ((y[0], t["q"], gq), (y[1], t["k"], gk)):
        if got is None:
            continue
        ref = O.qk_norm_rope_forward(to_np(x), None if g is None else to_np(g), eps, theta, rot, inter)
        close(got, ref, dtype, D)
    # gradients into a packed buffer with a part of its own in between
    pack = torch.full((B, T, Hq + Hkv + 1, D), 7.0, dtype=dtype, device="cuda")
    gr = abw.qk_norm_rope_bwd(q, k if has_k else None, t["dq"].cuda(), t["dk"].cuda(), dev(gq), dev(gk),
                              dq=pack[:, :, :Hq], dk=pack[:, :, Hq + 1:] if has_k else None, **how)
    assert bool((pack[:, :, Hq] == 7.0).all())
    for dx, dg, x, g, d in ((gr[0], gr[2], t["q"], gq, t["dq"]), (gr[1], gr[3], t["k"], gk, t["dk"])):
        if dx is None:
            continue
        rx, rg = O.qk_norm_rope_backward(to_np(x), None if g is None else to_np(g), to_np(d), eps, theta, rot, inter)
        close(dx, rx, dtype, D, 3.0)
        assert (dg is None) == (g is None)
        if g is not None:
            dn = O.rope_turn(to_np(d), theta, rot, inter, -1.0) if theta is not None else to_np(d)
            xx = to_np(x)
            size = np.abs(dn * xx / np.sqrt((xx * xx).mean(-1, keepdims=True) + eps)).sum((0, 1, 2))
            tol = (min(B * T * x.shape[2], 4096) + D) * 2.0 ** -24 * size
            assert np.all(np.abs(to_np(dg) - rg) <= tol)
    return y, gr


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("dtype,dy", [(BF, F), (BF, BF), (F, F), (F, BF)])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 32), (80, 48), (256, 192), (512, 512)])
def test_heads_and_types(abw, D, rot, dtype, dy, inter):
    check(abw, 2, 9, 5, 2, D, rot, None, 10000.0, inter, dtype, dy, seed=D + rot)


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("D,rot", [(2, 2), (6, 4), (10, 10), (96, 2), (34, 14), (128, 90), (510, 510)])
def test_sizes_no_vector_fits(abw, D, rot, inter):
    check(abw, 1, 7, 3, 1, D, rot, None, 100.0, inter, BF, F, seed=D)
    check(abw, 2, 3, 2, 2, D, rot, None, 100.0, inter, F, F, seed=D + 1)


@pytest.mark.parametrize("sections,rot", [([16, 24, 24], 128), ([10, 6], 32), ([0, 8, 0, 8], 32), ([64], 128), ([1, 30, 1], 64)])
def test_axes(abw, sections, rot):
    for inter in (True, False):
        check(abw, 2, 33, 4, 2, 128, rot, sections, 10000.0, inter, BF, BF, seed=rot)


@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (64, 1, 20, 5), (1, 1, 32, 0), (3, 700, 20, 5), (1, 5000, 1, 1), (2, 129, 3, 3)])
def test_tokens_and_heads(abw, B, T, Hq, Hkv):
    check(abw, B, T, Hq, Hkv, 128, 128, None, 500000.0, True, BF, F, seed=B * T)


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("dtype,dy", [(BF, F), (BF, BF), (F, F), (F, BF)])
@pytest.mark.parametrize("D,rot,Hq,Hkv", [(64, 64, 260, 3), (80, 48, 130, 2), (256, 192, 70, 70), (512, 512, 70, 1)])
def test_many_heads(abw, D, rot, Hq, Hkv, dtype, dy, inter):
    """Enough rows for a group of lanes that they come through shared memory."""
    check(abw, 1, 9, Hq, Hkv, D, rot, None, 10000.0, inter, dtype, dy, seed=D)


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("dtype,dy", [(BF, BF), (F, F)])
def test_many_tokens(abw, dtype, dy, inter):
    """The backward's groups go on from token to token, the last ones behind the end."""
    check(abw, 2, 6001, 4, 4, 128, 96, [16, 16, 16], 10000.0, inter, dtype, dy, seed=3)


@pytest.mark.parametrize("norm", [(False, False), (True, False), (False, True)])
def test_without_a_norm(abw, norm):
    check(abw, 2, 11, 4, 2, 128, 64, None, 10000.0, False, BF, F, norm=norm, seed=3)


def test_norm_alone(abw):
    check(abw, 2, 11, 4, 2, 96, 0, None, 0.0, True, F, F, seed=4)


def test_far_and_negative_positions(abw):
    """The angle of any 32-bit position: the double-precision oracle itself
    forms pos * freq to 2^-53, so its angles are off by up to 2^31 2^-53 =
    2.4e-7 rad: with its 2^-24 roundings that stays inside the tolerance."""
    check(abw, 2, 50, 3, 1, 128, 128, None, 10000.0, True, F, F, far=2 ** 31 - 1, seed=5)
    check(abw, 1, 40, 3, 1, 64, 64, None, 10000.0, False, F, F, positions=False, pos0=2 ** 31 - 41, seed=6)
    check(abw, 1, 40, 3, 1, 64, 64, None, 0.5, False, F, F, far=1000, seed=7)      # angles that grow with i


def test_rows_of_zeros_and_of_large_values(abw):
    q = torch.zeros(1, 4, 2, 128, dtype=F, device="cuda")
    q[0, 1] = 1e15
    g = torch.ones(128, device="cuda")
    y, _ = abw.qk_norm_rope_fwd(q, None, g, eps=1e-6)
    assert bool((y[0, 0] == 0).all()) and bool(torch.isfinite(y).all())
    assert torch.allclose(y[0, 1], torch.ones_like(y[0, 1]), rtol=1e-6)
    dx, _, dg, _ = abw.qk_norm_rope_bwd(q, None, torch.ones_like(q), None, g, eps=1e-6)
    assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dg).all())
    assert torch.allclose(dx[0, 0], torch.full_like(dx[0, 0], 1000.0), rtol=1e-5)   # dy / sqrt(eps)


def test_dgamma_is_zero_without_tokens_and_bits_repeat(abw):
    q = torch.empty(2, 0, 4, 64, dtype=BF, device="cuda")
    g = torch.ones(64, device="cuda")
    dg = torch.full((64,), 3.0, device="cuda")
    out = abw.qk_norm_rope_bwd(q, q, torch.empty_like(q), torch.empty_like(q), g, g, dgamma_q=dg)
    assert bool((out[2] == 0).all()) and bool((out[3] == 0).all())
    t = inputs(8, 4, 1500, 20, 5, 128, BF)
    q, k = views(t["qkv"], 20, 5)
    run = lambda: abw.qk_norm_rope_bwd(q, k, t["dq"].cuda(), t["dk"].cuda(), t["gq"].cuda(), t["gk"].cuda(), rope_base=1e4)
    a, b = run(), run()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_misaligned_rows_and_padded_strides(abw):
    """Rows that start off a 16-byte boundary, and tokens with a gap between."""
    t = inputs(9, 2, 20, 3, 1, 64, BF)
    wide = torch.zeros(2, 20, 64 * 4 + 2, dtype=BF, device="cuda")
    q, k = wide[:, :, :192].view(2, 20, 3, 64), wide[:, :, 194:].view(2, 20, 1, 64)
    q.copy_(t["q"]), k.copy_(t["k"])
    a = abw.qk_norm_rope_fwd(q, k, t["gq"].cuda(), t["gk"].cuda(), rope_base=1e4)
    b = abw.qk_norm_rope_fwd(t["q"].contiguous().cuda(), t["k"].contiguous().cuda(), t["gq"].cuda(), t["gk"].cuda(), rope_base=1e4)
    for x, y, src in zip(a, b, (t["q"], t["k"])):
        theta = O.section_angles(np.broadcast_to(np.arange(20), (1, 2, 20)), 64, 1e4, [32])
        g = t["gq"] if src is t["q"] else t["gk"]
        ref = O.qk_norm_rope_forward(to_np(src), to_np(g), 1e-6, theta, 64, True)
        close(x, ref, BF, 64)
        close(y, ref, BF, 64)


@pytest.mark.parametrize("D", [64, 66])
def test_offsets_past_32_bits(abw, D):
    """Tokens some 2^23 elements apart: the last ones start behind 2^31."""
    T, gap = 130, 1 << 23
    t = inputs(11, 2, T, 3, 1, D, BF)
    wide = torch.empty(2, T, gap, dtype=BF, device="cuda")
    outs = torch.empty(2, T, gap, dtype=BF, device="cuda")
    assert wide.numel() - gap > 2 ** 31
    part = lambda buf, at, h: buf[:, :, at * D:(at + h) * D].view(2, T, h, D)
    q, k = part(wide, 0, 3).copy_(t["q"]), part(wide, 3, 1).copy_(t["k"])
    g = (t["gq"].cuda(), t["gk"].cuda())
    qd, kd, dq, dk = t["q"].contiguous().cuda(), t["k"].contiguous().cuda(), t["dq"].cuda(), t["dk"].cuda()
    want = abw.qk_norm_rope_fwd(qd, kd, *g, rope_base=1e4) + abw.qk_norm_rope_bwd(qd, kd, dq, dk, *g, rope_base=1e4)
    got = abw.qk_norm_rope_fwd(q, k, *g, rope_base=1e4) + abw.qk_norm_rope_bwd(
        q, k, dq, dk, *g, rope_base=1e4, dq=part(outs, 0, 3), dk=part(outs, 3, 1))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_other_stream_and_graph(abw):
    t = inputs(10, 2, 300, 4, 2, 128, BF)
    q, k = views(t["qkv"], 4, 2)
    gq, gk, dq, dk = (t[x].cuda() for x in ("gq", "gk", "dq", "dk"))
    want = abw.qk_norm_rope_bwd(q, k, dq, dk, gq, gk, rope_base=1e4)
    fwd = abw.qk_norm_rope_fwd(q, k, gq, gk, rope_base=1e4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = abw.qk_norm_rope_bwd(q, k, dq, dk, gq, gk, rope_base=1e4, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = abw.qk_norm_rope_fwd(q, k, gq, gk, rope_base=1e4) + abw.qk_norm_rope_bwd(q, k, dq, dk, gq, gk, rope_base=1e4)
        graphs.append((gr, out))
    for gr, out in graphs + graphs[::-1]:
        for x in out:
            x.fill_(9.0)
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, fwd + want))


def test_binding_refusals(abw):
    q = torch.zeros(1, 4, 2, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        abw.qk_norm_rope_fwd(q.transpose(1, 2), None)
    with pytest.raises(ValueError):
        abw.qk_norm_rope_fwd(q, q[:, :, :, :32])
    with pytest.raises(TypeError):
        abw.qk_norm_rope_fwd(q, q.float())
    with pytest.raises(TypeError):
        abw.qk_norm_rope_fwd(q.half(), None)
    with pytest.raises(ValueError):
        abw.qk_norm_rope_fwd(q, None, torch.zeros(32, device="cuda"))
    with pytest.raises(ValueError):
        abw.qk_norm_rope_fwd(q, None, rope_base=1e4, positions=torch.zeros(1, 1, 5, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        abw.qk_norm_rope_fwd(q.cpu(), None)
    with pytest.raises(abw.AbwError):
        abw.qk_norm_rope_fwd(q, None, rope_base=1e4, rotary_dim=66)
    with pytest.raises(abw.AbwError):
        abw.qk_norm_rope_fwd(q, None, q_out=q)
