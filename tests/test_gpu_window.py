"""GPU parity of the softmax attention over a sliding window with first tokens
that stay visible, forward and backward, against the float64 oracle.

Tolerances, on the 2-norm of an output's error over that of the output.  A
rounding to bf16 is off by at most 2^-8 of the value, independent of the others
and of zero-mean inputs, so n of them on the way add up in squares: sqrt(n)
2^-8.  o: P and o itself (2).  dv: P and dv (2).  dq, dk: dS and the output (2).
The backward is defined on the o that the forward saved, so the oracle takes that
o, rounded as it is: delta = dout . o is off from sum P dP by some 2^-8 |dout| |o|
whatever computes it, and where one weight is close to 1, dP - delta is no larger
than that (the gradient of the unrounded function is tested by differences).  Single elements may be off by 8 times that share of
the output's mean square root, or of themselves, or of their row's: an element's
error is the sum of its terms' errors, so it grows as the row's own sum does (the
dk and dv of a first token sum over all queries, those of others over a window:
with window 1 some 700 terms beside two, sqrt(350) times the others' size).  Where
a query sees one key alone, dS = dP - delta is 0 and what is left are two fp32 sums
of the same D products in different orders: D additions, each off by 2^-24 of a
partial sum of up to 3 sqrt(D) (unit normal terms), sqrt(D) of that together, twice;
with scale and a factor |q| or |k|: 6 D 2^-24 scale max(|q|, |k|) absolute.  lse is fp32: products of bf16
values are exact, their sum and the scale good to some 2^-20 of sum |q k| (D
additions of 2^-24), exp and log to 2^-21 each."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from tests.helpers import to_np

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
TOL = 2 ** 0.5 * 2.0 ** -8
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def abw():
    import transformer_attention_backward_gb300 as m
    m.library()
    return m


def near(got, ref, tol, least=0.0):
    g = to_np(got)
    assert g.shape == ref.shape and np.all(np.isfinite(g))
    if g.size == 0:
        return
    rms = math.sqrt(float(np.mean(ref * ref)))
    err = g - ref
    assert math.sqrt(float(np.mean(err * err))) <= tol * rms + least
    row = np.sqrt(np.mean(ref * ref, axis=-1, keepdims=True))
    assert np.all(np.abs(err) <= 8 * tol * np.maximum(np.maximum(rms, row), np.abs(ref)) + least)


def make(seed, B, T, Hq, Hkv, D, q_size=1.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda h: torch.randn(B, T, h, D, generator=g)
    return {"q": (q_size * n(Hq)).to(BF), "k": n(Hkv).to(BF), "v": n(Hkv).to(BF), "do": n(Hq).to(BF)}


def call(abw, d, window, sinks, lengths=None, scale=0.125, **out):
    """Forward and backward on the GPU: (o, lse, dq, dk, dv)."""
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, lse = abw.attn_fwd_window(d["q"], d["k"], d["v"], window, sinks, scale, lengths=ln)
    g = abw.attn_bwd_window(d["q"], d["k"], d["v"], o, d["do"], lse, window, sinks, scale, lengths=ln, **out)
    return (o, lse) + tuple(g)


def check(abw, t, window, sinks=0, lengths=None, scale=0.125):
    got = call(abw, {x: y.cuda() for x, y in t.items()}, window, sinks, lengths, scale)
    abw.device_check()
    f = {x: to_np(y) for x, y in t.items()}
    ro, rl = O.attn_window_forward(f["q"], f["k"], f["v"], scale, window, sinks, lengths)
    near(got[0], ro, TOL)
    l = to_np(got[1])
    live = np.isfinite(rl)
    assert np.array_equal(np.isneginf(l), ~live)
    most = max(1.0, float(np.abs(f["q"]).max() * np.abs(f["k"]).max()) * t["q"].shape[-1] * abs(scale))
    assert np.all(np.abs(l[live] - rl[live]) <= 2.0 ** -20 * most)
    rg = O.attn_window_backward(f["q"], f["k"], f["v"], f["do"], scale, window, sinks, lengths, to_np(got[0]))
    least = 6 * t["q"].shape[-1] * 2.0 ** -24 * abs(scale) * float(max(np.abs(f["q"]).max(), np.abs(f["k"]).max()))
    for a, b in zip(got[2:], rg):
        near(a, b, TOL, least)
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 127, 128, 129, 255, 300, 513])
def test_lengths(abw, T, D):
    check(abw, make(T + D, 2, T, 4, 2, D), 100, 3)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (3, 130), (64, 4), (127, 0), (128, 0), (128, 128), (129, 1),
                                          (130, 129), (200, 257), (256, 4), (300, 0), (699, 2), (700, 0), (2 ** 31 - 1, 4),
                                          (50, 2 ** 31 - 1)])
def test_windows(abw, window, sinks):
    check(abw, make(window % 1000 + sinks % 77, 1, 700, 2, 1, 128), window, sinks)
    check(abw, make(window % 1000 + sinks % 79, 1, 420, 2, 2, 64), window, sinks)


@pytest.mark.parametrize("B,Hq,Hkv,D", [(1, 1, 1, 128), (3, 5, 5, 64), (1, 6, 2, 128), (2, 8, 1, 64), (1, 20, 5, 128), (1, 12, 1, 128)])
def test_heads(abw, B, Hq, Hkv, D):
    check(abw, make(Hq + D, B, 333, Hq, Hkv, D), 77, 2)


def test_more_items_than_sms(abw):
    """Persistent blocks take several items each, ragged ones among them."""
    check(abw, make(1, 5, 700, 16, 4, 64), 200, 4, [700, 0, 129, 1, 512])
    check(abw, make(2, 4, 800, 40, 40, 64), 300, 0)
    check(abw, make(3, 4, 900, 24, 24, 128), 130, 5, [900, 513, 0, 385])
    check(abw, make(4, 2, 1100, 20, 5, 128), 400, 2)


@pytest.mark.parametrize("B,T,Hq,Hkv,window,sinks,lengths", [
    (3, 600, 20, 20, 64, 400, None),             # more blocks of first tokens than SMs
    (2, 900, 40, 10, 128, 4, [900, 77]),         # theirs cut to parts, the others whole
    (2, 1100, 16, 16, 130, 200, None),
    (1, 1300, 6, 2, 300, 700, None),             # all cut
    (3, 700, 30, 30, 1, 4, [0, 700, 350])])
def test_long_items_among_short_ones(abw, B, T, Hq, Hkv, window, sinks, lengths):
    """First tokens' blocks of keys meet many times the others' queries."""
    check(abw, make(T, B, T, Hq, Hkv, 64), window, sinks, lengths)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths", [[0, 300, 1], [128, 129, 255], [-5, 1000, 256], [0, 0, 0]])
def test_padded_batch(abw, lengths, D):
    """What stands behind a sequence is not looked at, NaN and infinities
    included, and the outputs are 0 there (lse -infinity)."""
    t = make(9, 3, 300, 4, 2, D)
    clean = check(abw, t, 90, 4, lengths)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), 300)
        for x, bad in (("q", NAN), ("k", INF), ("v", NAN), ("do", -INF)):
            t[x][b, n:] = bad
    got = call(abw, {x: y.cuda() for x, y in t.items()}, 90, 4, lengths)
    abw.device_check()
    for a, b in zip(clean, got):
        assert torch.equal(a, b)
    for x in (got[0],) + got[2:]:
        for b, n in enumerate(lengths):
            assert bool((x[b, min(max(n, 0), 300):] == 0).all())
    # the backward looks at neither o nor lse there
    o, lse = got[0].clone(), got[1].clone()
    for b, n in enumerate(lengths):
        n = min(max(n, 0), 300)
        o[b, n:], lse[b, :, n:] = NAN, NAN
    d = {x: y.cuda() for x, y in t.items()}
    g = abw.attn_bwd_window(d["q"], d["k"], d["v"], o, d["do"], lse, 90, 4, 0.125,
                            lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    for a, b in zip(clean[2:], g):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128])
def test_packed_projection(abw, D):
    """Parts of one packed tensor in and out give what dense tensors give, and
    what stands between them stays as it was."""
    B, T, Hq, Hkv = 2, 280, 6, 2
    t = make(4, B, T, Hq, Hkv, D)
    d = {x: y.cuda() for x, y in t.items()}
    want = call(abw, d, 100, 2)
    H = Hq + 2 * Hkv + 1
    qkv = torch.full((B, T, H, D), 7.0, dtype=BF, device="cuda")
    cut = lambda x: (x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:Hq + 2 * Hkv])
    for part, x in zip(cut(qkv), "qkv"):
        part.copy_(d[x])
    q, k, v = cut(qkv)
    ob = torch.full((B, T, Hq + 1, D), 5.0, dtype=BF, device="cuda")
    o, lse = abw.attn_fwd_window(q, k, v, 100, 2, 0.125, o=ob[:, :, :Hq])
    grad = torch.full((B, T, H, D), 3.0, dtype=BF, device="cuda")
    dq, dk, dv = cut(grad)
    abw.attn_bwd_window(q, k, v, o, d["do"], lse, 100, 2, 0.125, dq=dq, dk=dk, dv=dv)
    abw.device_check()
    for a, b in zip((o, lse, dq, dk, dv), want):
        assert torch.equal(a, b)
    assert bool((ob[:, :, Hq:] == 5).all()) and bool((grad[:, :, H - 1:] == 3).all()) and bool((qkv[:, :, H - 1:] == 7).all())


def test_equal_calls_give_equal_bits(abw):
    d = {x: y.cuda() for x, y in make(5, 2, 1500, 20, 5, 128).items()}
    first = call(abw, d, 300, 4)
    for _ in range(20):
        for a, b in zip(first, call(abw, d, 300, 4)):
            assert torch.equal(a, b)
    abw.device_check()


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales(abw, scale):
    """Equal weights, turned signs, and scores far apart (the largest weight
    close to 1, others below 2^-100)."""
    check(abw, make(6, 1, 300, 2, 1, 128), 120, 1, scale=scale)
    if scale == 1.0:
        check(abw, make(6, 1, 300, 2, 1, 64, q_size=4.0), 120, 1, scale=scale)


def test_a_running_maximum_that_keeps_rising(abw):
    """Scores that grow from block to block move the maximum every time; ones
    that fall leave it at the first block's."""
    for sign in (1.0, -1.0):
        t = make(7, 1, 700, 2, 1, 128)
        t["q"][:] = t["q"].abs()
        t["k"] = (t["k"].abs() * (0.01 * sign * torch.arange(700.0))[None, :, None, None]).to(BF)
        check(abw, t, 600, 0, scale=0.125)


def test_gradients_are_the_difference_quotient(abw):
    """The GPU's own forward, f(x + d) - f(x - d) with f = sum o do, along each
    gradient's signs.  f is off by o's roundings, 2^-8 |o do| each and
    independent: 4 standard deviations of their sum, twice.  The terms of third
    order: scores move by up to m, and softmax's third derivatives are below 6
    of its first, so they stay below 6 m^2 / 6 of the difference."""
    B, T, Hq, Hkv, D, W, S = 1, 160, 2, 1, 64, 40, 3
    t = {x: y.cuda() for x, y in make(8, B, T, Hq, Hkv, D).items()}
    got = call(abw, t, W, S)
    noise = 4 * 2 * 2.0 ** -8 * float((got[0].double() * t["do"].double()).norm())

    def f(**x):
        a = {**t, **x}
        return float((abw.attn_fwd_window(a["q"], a["k"], a["v"], W, S, 0.125)[0].double() * t["do"].double()).sum())
    for name, grad in zip("qkv", got[2:]):
        d = 2.0 ** -5 * grad.sign().float()
        up, down = (t[name].float() + d).to(BF), (t[name].float() - d).to(BF)
        first = float((grad.double() * (up.double() - down.double())).sum())
        move = 0.0
        if name != "v":
            other = t["k" if name == "q" else "q"].double()
            dx = ((up.double() - down.double()) / 2).transpose(1, 2)
            move = float((dx @ other.transpose(1, 2).transpose(2, 3)).abs().max()) * 0.125
        assert first > 10 * noise
        assert abs(first - (f(**{name: up}) - f(**{name: down}))) <= noise + move ** 2 * first, name


def test_graph_and_streams(abw):
    d = {x: y.cuda() for x, y in make(10, 2, 400, 8, 2, 128).items()}
    want = [x.clone() for x in call(abw, d, 90, 4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(abw.attn_bwd_window_workspace_bytes(2, 400, 8, 2, 128, 90, 4), dtype=torch.uint8, device="cuda")
    o, lse = abw.attn_fwd_window(d["q"], d["k"], d["v"], 90, 4, 0.125, stream=side)
    got = abw.attn_bwd_window(d["q"], d["k"], d["v"], o, d["do"], lse, 90, 4, 0.125, workspace=ws, stream=side)
    side.synchronize()
    for a, b in zip((o, lse) + tuple(got), want):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):                                       # two graphs that share the workspace, run in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, lse = abw.attn_fwd_window(d["q"], d["k"], d["v"], 90, 4, 0.125)
            out = (o, lse) + tuple(abw.attn_bwd_window(d["q"], d["k"], d["v"], o, d["do"], lse, 90, 4, 0.125, workspace=ws))
        graphs.append((graph, out))
    ws.fill_(255)
    for _ in range(3):
        for graph, out in graphs:
            for x in out:
                x.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b)
    abw.device_check()


def test_binding_refusals(abw):
    d = {x: y.cuda() for x, y in make(11, 1, 8, 2, 1, 64).items()}
    with pytest.raises(abw.AbwError, match="window"):
        abw.attn_fwd_window(d["q"], d["k"], d["v"], 0)
    with pytest.raises(ValueError, match="32 bits"):
        abw.attn_fwd_window(d["q"], d["k"], d["v"], 2 ** 31)
    with pytest.raises(TypeError):
        abw.attn_fwd_window(d["q"].float(), d["k"], d["v"], 4)
    with pytest.raises(ValueError):
        abw.attn_fwd_window(d["q"], d["k"], d["v"][:, :, :, :32], 4)
    with pytest.raises(ValueError):
        abw.attn_fwd_window(d["q"], d["k"].cpu(), d["v"], 4)
    with pytest.raises(TypeError):
        abw.attn_fwd_window(d["q"], d["k"], d["v"], 4, lengths=torch.tensor([8], device="cuda"))
    o, lse = abw.attn_fwd_window(d["q"], d["k"], d["v"], 4)
    with pytest.raises(abw.AbwError, match="workspace"):
        abw.attn_bwd_window(d["q"], d["k"], d["v"], o, d["do"], lse, 4, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    for z in (abw.attn_fwd_window(*(d[x][:, :0] for x in "qkv"), 4)[0], abw.attn_fwd_window(*(d[x][:0] for x in "qkv"), 4)[0]):
        assert z.numel() == 0
