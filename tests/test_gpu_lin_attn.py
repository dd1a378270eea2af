"""GPU parity of the linear attention with a decay for each head (chunked
forward and backward, single-token form) against the float64 oracle.

Tolerances, on the 2-norm of an output's error over that of the output.  bf16
outputs: a score, a state element and the output are each rounded to bf16
once, at most 2^-8 of their size; the roundings are independent of one
another and of zero-mean inputs, so the three add up in squares: sqrt(3) 2^-8.
Single elements may be off by 8 times that share of the output's mean square
root (8 standard deviations and more).  fp32 states: the weighted rows enter
in three bf16 terms (2^-25 left), some 35 tensor-core additions of 2^-23 per
chunk and one per chunk of the state, decay powers to 2^-22: (40 + 2 chunks)
2^-23 at most."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from tests.helpers import to_np

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
TOL = 3 ** 0.5 * 2.0 ** -8


def tol32(T):
    return (40 + 2 * ((T + 127) // 128)) * 2.0 ** -23


@pytest.fixture(scope="module")
def abw():
    import transformer_attention_backward_gb300 as m
    m.library()
    return m


def near(got, ref, tol):
    g = to_np(got)
    assert g.shape == ref.shape and np.all(np.isfinite(g))
    if g.size == 0:
        return
    rms = math.sqrt(float(np.mean(ref * ref)))
    err = g - ref
    assert math.sqrt(float(np.mean(err * err))) <= tol * rms
    assert np.all(np.abs(err) <= 8 * tol * np.maximum(rms, np.abs(ref)))


def make(seed, B, T, Hq, Hkv, D, state=False, decay=None):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    t = {"q": n(B, T, Hq, D).to(BF), "k": n(B, T, Hkv, D).to(BF), "v": n(B, T, Hkv, D).to(BF), "do": n(B, T, Hq, D).to(BF)}
    h = torch.arange(1, Hkv + 1, dtype=torch.float32)
    t["ld"] = -(2.0 ** (-6.0 * h / Hkv)) if decay is None else torch.as_tensor(decay, dtype=F).expand(Hkv).contiguous()
    t["s0"], t["df"] = (n(B, Hkv, D, D), n(B, Hkv, D, D)) if state else (None, None)
    return t


def cuda(x):
    return None if x is None else x.cuda()


def npy(x):
    return None if x is None else to_np(x)


def check(abw, t, lengths=None, scale=0.125, want=None):
    """Forward and backward of one case against the oracle; the outputs."""
    d = {x: cuda(y) for x, y in t.items()}
    T, ln = t["q"].shape[1], None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    state = t["s0"] is not None if want is None else want
    o, fin = abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"], scale, initial_state=d["s0"], lengths=ln, want_final_state=state)
    gr = abw.lin_attn_bwd(d["q"], d["k"], d["v"], d["do"], d["ld"], scale, initial_state=d["s0"], dfinal_state=d["df"],
                          lengths=ln, want_dinitial_state=state)
    abw.device_check()
    f64 = {x: npy(y) for x, y in t.items()}
    ro, rf = O.lin_attn_forward(f64["q"], f64["k"], f64["v"], f64["ld"], scale, f64["s0"], lengths)
    rg = O.lin_attn_backward(f64["q"], f64["k"], f64["v"], f64["do"], f64["ld"], scale, f64["s0"], f64["df"], lengths)
    near(o, ro, TOL)
    for a, b in zip(gr[:3], rg[:3]):
        near(a, b, TOL)
    assert (fin is not None) == state and (gr[3] is not None) == state
    if state:
        near(fin, rf, tol32(T))
        near(gr[3], rg[3], tol32(T))
    return (o, fin) + tuple(gr)


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 127, 128, 129, 300, 513])
def test_lengths(abw, T, D, state):
    check(abw, make(T + D, 2, T, 4, 2, D, state))


@pytest.mark.parametrize("B,Hq,Hkv,D", [(1, 1, 1, 128), (3, 5, 5, 64), (1, 6, 2, 128), (2, 8, 1, 64), (1, 20, 5, 128), (1, 12, 1, 128)])
def test_heads(abw, B, Hq, Hkv, D):
    check(abw, make(Hq + D, B, 200, Hq, Hkv, D, True))


def test_more_items_than_sms(abw):
    """Persistent CTAs take several items each, ragged ones among them."""
    check(abw, make(1, 5, 330, 16, 4, 64, True), lengths=[330, 0, 129, 1, 256])
    check(abw, make(2, 3, 260, 40, 40, 64, False))
    check(abw, make(3, 4, 800, 24, 24, 128, False), lengths=[800, 513, 0, 385])     # a KV head of its own for each
    check(abw, make(4, 2, 900, 30, 30, 64, True), lengths=[900, 129])


@pytest.mark.parametrize("decay", [0.0, -1e-4, -0.05, -1.0, -30.0, -1000.0, -math.inf])
def test_decays(abw, decay):
    """From none to one that leaves the token itself; no power overflows."""
    t = make(7, 1, 300, 2, 2, 128, True, decay)
    check(abw, t)
    check(abw, make(8, 1, 140, 4, 2, 64, False, [decay, -0.3]))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths", [[0, 300, 1], [128, 129, 255], [-5, 1000, 256], [0, 0, 0]])
def test_padded_batch(abw, lengths, D):
    """What stands behind a sequence is not looked at, NaN and infinities
    included, and the outputs are 0 there."""
    t = make(9, 3, 300, 4, 2, D, True)
    clean = check(abw, t, lengths)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), 300)
        for x, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("do", -float("inf"))):
            t[x][b, n:] = bad
    d = {x: cuda(y) for x, y in t.items()}
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o = abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"], 0.125, initial_state=d["s0"], lengths=ln, want_final_state=True)
    g = abw.lin_attn_bwd(d["q"], d["k"], d["v"], d["do"], d["ld"], 0.125, initial_state=d["s0"], dfinal_state=d["df"],
                         lengths=ln, want_dinitial_state=True)
    abw.device_check()
    for a, b in zip(clean, o + g):
        assert torch.equal(a, b)
    for x in (o[0],) + g[:3]:
        for b, n in enumerate(lengths):
            assert bool((x[b, min(max(n, 0), 300):] == 0).all())


@pytest.mark.parametrize("T,Hq,Hkv,D", [(300, 6, 2, 128), (512, 4, 4, 64), (700, 3, 1, 64), (769, 2, 2, 128)])
def test_padded_batch_without_states(abw, T, Hq, Hkv, D):
    """No state comes in or goes out: short batches take their other chunks
    directly, longer ones through states (both directions differ in where
    that changes)."""
    lengths = [T, 129, 0, 1, 128, 257]
    t = make(T, 6, T, Hq, Hkv, D, decay=torch.tensor([-0.004, -0.5])[:Hkv] if Hkv < 3 else -0.03)
    clean = check(abw, t, lengths)
    for b, n in enumerate(lengths):
        for x, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("do", -float("inf"))):
            t[x][b, n:] = bad
    d = {x: cuda(y) for x, y in t.items()}
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o = abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"], 0.125, lengths=ln)
    g = abw.lin_attn_bwd(d["q"], d["k"], d["v"], d["do"], d["ld"], 0.125, lengths=ln)
    abw.device_check()
    for a, b in zip(clean, o + g):
        assert (a is None and b is None) or torch.equal(a, b)
    for decay in (0.0, -20.0, -math.inf):
        check(abw, make(T + 1, 1, T, Hq, Hkv, D, decay=decay))


def test_states_wanted_or_not(abw):
    """Every mix of states that come in and go out, over one chunk and more."""
    for T in (100, 200):
        t = make(T, 2, T, 2, 2, 128, True)
        d = {x: cuda(y) for x, y in t.items()}
        f = {x: npy(y) for x, y in t.items()}
        for s0 in (True, False):
            for out in (True, False):
                a, z = (d["s0"], f["s0"]) if s0 else (None, None)
                b, y = (d["df"], f["df"]) if not s0 or out else (None, None)
                o, fin = abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"], 0.1, initial_state=a, want_final_state=out)
                g = abw.lin_attn_bwd(d["q"], d["k"], d["v"], d["do"], d["ld"], 0.1, initial_state=a, dfinal_state=b,
                                     want_dinitial_state=out)
                ro, rf = O.lin_attn_forward(f["q"], f["k"], f["v"], f["ld"], 0.1, z)
                rg = O.lin_attn_backward(f["q"], f["k"], f["v"], f["do"], f["ld"], 0.1, z, y)
                near(o, ro, TOL)
                for p, r in zip(g[:3], rg[:3]):
                    near(p, r, TOL)
                if out:
                    near(fin, rf, tol32(T))
                    near(g[3], rg[3], tol32(T))


def test_packed_projection_and_gradient(abw):
    t = make(11, 2, 200, 4, 2, 128)
    want = check(abw, t)
    qkv = torch.cat([t["q"], t["k"], t["v"]], 2).cuda()
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    pack = torch.full((2, 200, 9, 128), 7.0, dtype=BF, device="cuda")
    wide = torch.full((2, 200, 5, 128), 7.0, dtype=BF, device="cuda")
    o, _ = abw.lin_attn_fwd(q, k, v, cuda(t["ld"]), 0.125, o=wide[:, :, :4])
    g = abw.lin_attn_bwd(q, k, v, cuda(t["do"]), cuda(t["ld"]), 0.125, dq=pack[:, :, :4], dk=pack[:, :, 4:6], dv=pack[:, :, 7:])
    for a, b in zip((want[0],) + want[2:5], (o,) + g[:3]):
        assert torch.equal(a, b)
    assert bool((pack[:, :, 6] == 7.0).all()) and bool((wide[:, :, 4] == 7.0).all())


def test_state_in_place_continues_a_prompt(abw):
    """A prompt in two calls, the state in one buffer, equals one call."""
    t = make(12, 2, 256 + 70, 4, 2, 128, True)
    d = {x: cuda(y) for x, y in t.items()}
    o, fin = abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"], 0.125, initial_state=d["s0"], want_final_state=True)
    st = d["s0"].clone()
    parts = []
    for lo, hi in ((0, 256), (256, 326)):
        part = [d[x][:, lo:hi].contiguous() for x in "qkv"]
        y, out = abw.lin_attn_fwd(*part, d["ld"], 0.125, initial_state=st, final_state=st)
        assert out is st
        parts.append(y)
    assert torch.equal(torch.cat(parts, 1), o) and torch.equal(st, fin)     # 256 is a chunk border: the same steps
    df = d["df"].clone()
    a = abw.lin_attn_bwd(d["q"], d["k"], d["v"], d["do"], d["ld"], 0.125, dfinal_state=d["df"], want_dinitial_state=True)
    b = abw.lin_attn_bwd(d["q"], d["k"], d["v"], d["do"], d["ld"], 0.125, dfinal_state=df, dinitial_state=df)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("Hkv", [2, 4])
def test_offsets_past_32_bits(abw, Hkv):
    """Tokens some 2^23 elements apart: the last ones start behind 2^31."""
    T, Hq, D, gap = 150, 4, 64, 1 << 23
    t = make(15, 2, T, Hq, Hkv, D, True)
    d = {x: cuda(y) for x, y in t.items()}
    wide = torch.empty(2, T, gap, dtype=BF, device="cuda")
    outs = torch.empty(2, T, gap, dtype=BF, device="cuda")
    assert wide.numel() - gap > 2 ** 31
    part = lambda buf, at, h: buf[:, :, at * D:(at + h) * D].view(2, T, h, D)
    q, k, v = (part(wide, at, h).copy_(d[x]) for x, at, h in (("q", 0, Hq), ("k", Hq, Hkv), ("v", Hq + Hkv, Hkv)))
    for s0, df in ((None, None), (d["s0"], d["df"])):
        how = dict(initial_state=s0)
        want = abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"], 0.125, want_final_state=s0 is not None, **how)
        got = abw.lin_attn_fwd(q, k, v, d["ld"], 0.125, want_final_state=s0 is not None, o=part(outs, 0, Hq), **how)
        how["dfinal_state"] = df
        want += abw.lin_attn_bwd(d["q"], d["k"], d["v"], d["do"], d["ld"], 0.125, **how)
        got += abw.lin_attn_bwd(q, k, v, d["do"], d["ld"], 0.125, dq=part(outs, Hq, Hq), dk=part(outs, 2 * Hq, Hkv),
                                dv=part(outs, 2 * Hq + Hkv, Hkv), **how)
        abw.device_check()
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("Hkv", [4, 8])
def test_waits_that_run_out(abw, Hkv):
    """A limit of zero: kernels that give up say so and leave the device as it
    was, so the next call is right."""
    from transformer_attention_backward_gb300 import _binding as B
    t = make(16, 2, 900, 8, Hkv, 128, True)
    d = {x: cuda(y) for x, y in t.items()}

    def run():
        return (abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"], 0.125, initial_state=d["s0"], want_final_state=True)
                + abw.lin_attn_bwd(d["q"], d["k"], d["v"], d["do"], d["ld"], 0.125, initial_state=d["s0"],
                                   dfinal_state=d["df"], want_dinitial_state=True))
    want = run()
    abw.device_check()
    lib = abw.library()
    lib.abw_set_wait_limit_ns(0)
    try:
        run()
        status = lib.abw_device_check(torch.cuda.current_stream().cuda_stream)
    finally:
        lib.abw_set_wait_limit_ns(2_000_000_000)
    assert status in (B.OK, B.ETIMEOUT)
    got = run()
    abw.device_check()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_tokens(abw):
    t = make(13, 2, 0, 4, 2, 64, True)
    d = {x: cuda(y) for x, y in t.items()}
    o, fin = abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"], initial_state=d["s0"], want_final_state=True)
    assert o.shape == (2, 0, 4, 64) and torch.equal(fin, d["s0"])
    _, fin = abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"], want_final_state=True)
    assert bool((fin == 0).all())
    g = abw.lin_attn_bwd(d["q"], d["k"], d["v"], d["do"], d["ld"], dfinal_state=d["df"], want_dinitial_state=True)
    assert torch.equal(g[3], d["df"])


@pytest.mark.parametrize("Hkv", [4, 8])
def test_bits_repeat_streams_and_graphs(abw, Hkv):
    t = make(14, 2, 400, 8, Hkv, 128, True)
    d = {x: cuda(y) for x, y in t.items()}

    def run(**kw):
        return (abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"], 0.125, initial_state=d["s0"], want_final_state=True, **kw)
                + abw.lin_attn_bwd(d["q"], d["k"], d["v"], d["do"], d["ld"], 0.125, initial_state=d["s0"],
                                   dfinal_state=d["df"], want_dinitial_state=True, **kw))

    want = run()
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    streams = [torch.cuda.Stream() for _ in range(2)]                       # two calls at once
    torch.cuda.synchronize()
    both = [run(stream=s) for s in streams]
    torch.cuda.synchronize()
    for got in both:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = run()
        graphs.append((gr, out))
    for gr, out in graphs + graphs[::-1]:
        for x in out:
            x.fill_(3.0)
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    abw.device_check()


# ------------------------------------------------------------ single tokens
def decode_inputs(seed, B, Hq, Hkv, D, dtype, pool=None):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    h = torch.arange(1, Hkv + 1, dtype=F)
    return (n(B, Hq, D).to(dtype), n(B, Hkv, D).to(dtype), n(B, Hkv, D).to(dtype), n(pool or B, Hkv, D, D), -(2.0 ** (-8 * h / Hkv)))


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("B,Hq,Hkv,D", [(1, 1, 1, 64), (1, 20, 5, 128), (3, 6, 2, 128), (2, 5, 1, 64), (7, 8, 1, 128), (4, 21, 3, 64), (70, 4, 4, 128)])
def test_decode(abw, B, Hq, Hkv, D, dtype):
    """fp32: D products and sums of 2^-24; bf16 out: one rounding more."""
    q, k, v, s, ld = decode_inputs(B + D, B, Hq, Hkv, D, dtype)
    st = s.cuda()
    o = abw.lin_attn_decode(q.cuda(), k.cuda(), v.cuda(), st, ld.cuda(), 0.2)
    ro, rs = O.lin_attn_decode(to_np(q), to_np(k), to_np(v), to_np(s), to_np(ld), 0.2)
    near(o, ro, 2.0 ** -8 if dtype == BF else D * 2.0 ** -24)
    near(st, rs, 4 * 2.0 ** -24)


def test_decode_slots(abw):
    q, k, v, s, ld = decode_inputs(3, 6, 8, 4, 128, BF, pool=9)
    slots = torch.tensor([8, -1, 0, 9, 3, -2 ** 31], dtype=torch.int32)
    st = s.cuda()
    o = abw.lin_attn_decode(q.cuda(), k.cuda(), v.cuda(), st, ld.cuda(), 0.2, slots=slots.cuda())
    ro, rs = O.lin_attn_decode(to_np(q), to_np(k), to_np(v), to_np(s), to_np(ld), 0.2, slots.tolist())
    near(o, ro, 2.0 ** -8)
    near(st, rs, 4 * 2.0 ** -24)
    for row in (1, 3, 5):
        assert bool((o[row] == 0).all())
    for at in (1, 2, 4, 5, 6, 7):
        assert torch.equal(st[at].cpu(), s[at])
    none = abw.lin_attn_decode(q.cuda(), k.cuda(), v.cuda(), st[:0], ld.cuda(), 0.2, slots=slots.cuda())
    assert bool((none == 0).all())


def test_decode_state_past_32_bits(abw):
    q, k, v, s, ld = decode_inputs(4, 2, 8, 8, 128, BF)
    pool = torch.empty(2 ** 31 // (8 * 128 * 128) + 2, 8, 128, 128, device="cuda")
    slots = torch.tensor([pool.shape[0] - 1, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = s.cuda()
    st = s.cuda()
    want = abw.lin_attn_decode(q.cuda(), k.cuda(), v.cuda(), st, ld.cuda())
    got = abw.lin_attn_decode(q.cuda(), k.cuda(), v.cuda(), pool, ld.cuda(), slots=slots)
    assert torch.equal(got, want) and torch.equal(pool[slots.long()], st)


def test_prompt_then_tokens(abw):
    """The chunked form's final state carries on in the single-token form,
    also from a captured graph that updates the state in place."""
    t = make(21, 2, 150 + 5, 8, 2, 128)
    d = {x: cuda(y) for x, y in t.items()}
    ro, rf = O.lin_attn_forward(npy(t["q"]), npy(t["k"]), npy(t["v"]), npy(t["ld"]), 0.125)
    part = [d[x][:, :150].contiguous() for x in "qkv"]
    _, st = abw.lin_attn_fwd(*part, d["ld"], 0.125, want_final_state=True)
    token = [d[x][:, 150].contiguous() for x in "qkv"]
    y = abw.lin_attn_decode(*token, st, d["ld"], 0.125)
    near(y, ro[:, 150], 2.0 ** -8)
    gr = torch.cuda.CUDAGraph()
    keep = st.clone()
    with torch.cuda.graph(gr):
        y = abw.lin_attn_decode(*token, st, d["ld"], 0.125)
    st.copy_(keep)
    for i in range(151, 155):
        for x, name in zip(token, "qkv"):
            x.copy_(d[name][:, i])
        gr.replay()
        near(y, ro[:, i], 2.0 ** -8)
    near(st, rf, tol32(155))


# ---------------------------------------------------------- used together
def chain_oracle(qkv, gq, gk, do, theta, ld, Hq, Hkv, scale, linear):
    """float64 forward and gradient of norm + rotation + attention."""
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    yq, yk = O.qk_norm_rope_forward(q, gq, 1e-6, theta, 128, False), O.qk_norm_rope_forward(k, gk, 1e-6, theta, 128, False)
    if linear:
        o, _ = O.lin_attn_forward(yq, yk, v, ld, scale)
        dq, dk, dv, _ = O.lin_attn_backward(yq, yk, v, do, ld, scale)
    else:
        o, _ = O.causal_forward(yq, yk, v, scale)
        dq, dk, dv = O.causal_backward(yq, yk, v, do, scale)
    xq, gg = O.qk_norm_rope_backward(q, gq, dq, 1e-6, theta, 128, False)
    xk, hh = O.qk_norm_rope_backward(k, gk, dk, 1e-6, theta, 128, False)
    return o, xq, xk, dv, gg, hh


@pytest.mark.parametrize("linear", [True, False])
def test_chain(abw, linear):
    """Projection -> norm and rotation on two axes -> attention (linear, and
    the softmax one that was there) -> back.  bf16 roundings on the longest
    path to a gradient: the normed q and k, P, the state or dS, o (which the
    softmax backward reads), the attention's gradient and the last one; eight,
    added in squares."""
    B, T, Hq, Hkv, D = 2, 333, 8, 2, 128
    g = torch.Generator().manual_seed(31)
    n = lambda *s: torch.randn(*s, generator=g)
    qkv, do = n(B, T, Hq + 2 * Hkv, D).to(BF), n(B, T, Hq, D).to(BF)
    gq, gk = 1 + 0.1 * n(D), 1 + 0.1 * n(D)
    ld, scale = torch.tensor([-0.02, -0.3]), 1 / math.sqrt(D)
    pos = torch.randint(0, 500, (2, B, T), generator=g, dtype=torch.int32)
    how = dict(rope_base=1e4, interleaved=False, positions=pos.cuda(), sections=[40, 24])
    x = qkv.cuda()
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    yq, yk = abw.qk_norm_rope_fwd(q, k, gq.cuda(), gk.cuda(), **how)
    dx = torch.empty_like(x)
    if linear:
        o, _ = abw.lin_attn_fwd(yq, yk, v, ld.cuda(), scale)
        dq, dk, _, _ = abw.lin_attn_bwd(yq, yk, v, do.cuda(), ld.cuda(), scale, dv=dx[:, :, Hq + Hkv:])
    else:
        vv = v.contiguous()
        o, lse = abw.attn_fwd_causal(yq, yk, vv, scale)
        dq, dk, dv = abw.attn_bwd_causal(yq, yk, vv, o, do.cuda(), lse, scale)
        dx[:, :, Hq + Hkv:] = dv
    _, _, gg, hh = abw.qk_norm_rope_bwd(q, k, dq, dk, gq.cuda(), gk.cuda(), dq=dx[:, :, :Hq], dk=dx[:, :, Hq:Hq + Hkv], **how)
    abw.device_check()
    theta = O.section_angles(pos.numpy(), 128, 1e4, [40, 24])
    ref = chain_oracle(to_np(qkv), to_np(gq), to_np(gk), to_np(do), theta, to_np(ld), Hq, Hkv, scale, linear)
    tol = 8 ** 0.5 * 2.0 ** -8
    for got, r in zip((o, dx[:, :, :Hq], dx[:, :, Hq:Hq + Hkv], dx[:, :, Hq + Hkv:], gg, hh), ref):
        near(got, r, tol)


def test_binding_refusals(abw):
    t = make(1, 1, 8, 4, 2, 64)
    d = {x: cuda(y) for x, y in t.items()}
    with pytest.raises(TypeError):
        abw.lin_attn_fwd(d["q"].float(), d["k"], d["v"], d["ld"])
    with pytest.raises(ValueError):
        abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"][:1])
    with pytest.raises(ValueError):
        abw.lin_attn_fwd(d["q"], d["k"], d["v"][:, :4], d["ld"])
    with pytest.raises(ValueError):
        abw.lin_attn_fwd(d["q"], d["k"].transpose(1, 2).contiguous().transpose(1, 2), d["v"], d["ld"])
    with pytest.raises(ValueError):
        abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"], initial_state=torch.zeros(1, 2, 64, 32, device="cuda"))
    with pytest.raises(abw.AbwError):
        abw.lin_attn_fwd(d["q"], d["k"], d["v"], d["ld"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        abw.lin_attn_bwd(d["q"], d["k"], d["v"], d["do"].float(), d["ld"])
    st = torch.zeros(1, 2, 64, 64, device="cuda")
    with pytest.raises(ValueError):
        abw.lin_attn_decode(d["q"][0, :1], d["k"][0, ::8, :, :32], d["v"][0, :1], st, d["ld"])
    with pytest.raises(abw.AbwError):
        abw.lin_attn_decode(d["q"][0], d["k"][0], d["v"][0], st, d["ld"])     # 8 rows, one state
