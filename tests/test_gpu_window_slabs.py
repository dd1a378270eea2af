"""The windowed backward where its heads' tiles do not fit the workspace at one
time and go through it in turn: some KV heads of one long sequence, or some
sequences of a batch.  Against the definition in 64 bits on the GPU, with the
tolerances of the calls that fit."""
import pytest
import torch

from tests.helpers import to_np
from tests.test_gpu_window import BF, TOL, abw, near   # noqa: F401  (abw: the fixture)
from tests.test_gpu_window_groups import exact

pytestmark = pytest.mark.gpu


def run(abw, B, T, Hq, Hkv, D, window, sinks, lengths=None, packed=False):
    scale = D ** -0.5
    g = torch.Generator(device="cuda").manual_seed(T + D)
    H = Hq + 2 * Hkv
    if packed:
        qkv = torch.randn(B, T, H + 1, D, generator=g, device="cuda").to(BF)
        grad = torch.full((B, T, H + 1, D), 3.0, dtype=BF, device="cuda")
    else:
        parts = [torch.randn(B, T, h, D, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv)]
    cut = lambda x: (x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:H])
    q, k, v = cut(qkv) if packed else parts
    do = torch.randn(B, T, Hq, D, generator=g, device="cuda").to(BF)
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, lse = abw.attn_fwd_window(q, k, v, window, sinks, lengths=ln)
    need = abw.attn_bwd_window_workspace_bytes(B, T, Hq, Hkv, D, window, sinks)
    room = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    out = dict(zip(("dq", "dk", "dv"), cut(grad))) if packed else {}
    got = abw.attn_bwd_window(q, k, v, o, do, lse, window, sinks, lengths=ln, workspace=room[:need], **out)
    abw.device_check()
    assert bool((room[need:] == 171).all())                 # nothing behind the workspace
    if packed:
        assert bool((grad[:, :, H:] == 3).all())
    G = Hq // Hkv
    for b in range(B):
        n = T if lengths is None else lengths[b]
        for x in got:
            assert not bool(x[b, n:].any())
        for h in range(Hkv if n else 0):                    # a KV head at a time
            hq, at = slice(h * G, h * G + G), slice(h, h + 1)
            _, _, *ref = exact(q[b, :n, hq], k[b, :n, at], v[b, :n, at], o[b, :n, hq], do[b, :n, hq], scale, window, sinks)
            least = 6 * D * 2.0 ** -24 * scale * float(max(q.abs().max(), k.abs().max()))
            for x, y, part in zip(got, ref, (hq, at, at)):
                near(x[b, :n, part], to_np(y), TOL, least)
    again = abw.attn_bwd_window(q, k, v, o, do, lse, window, sinks, lengths=ln)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("Hq,Hkv,D,window,sinks", [(7, 7, 64, 8192, 0), (10, 5, 128, 5000, 130)])
def test_heads_of_one_sequence_in_turn(abw, Hq, Hkv, D, window, sinks):
    """68 and 59 MB of tiles a query head (2,080 tiles of 32 KB where 8,192 tokens see all), 2.9 and 3.5 GB in all: 42
    heads as 21 and 21, 30 pairs as 15 and 15."""
    run(abw, 1, 8192, Hq * 6, Hkv * 6, D, window, sinks)


def test_sequences_in_turn(abw):
    """17 MB of tiles a query head, 554 MB a sequence: three of seven at a time."""
    run(abw, 7, 4096, 32, 8, 64, 4096, 5, [4096, 0, 130, 4095, 2048, 1, 3000], packed=True)


def test_a_long_and_a_padded_sequence(abw):
    """Heads of each sequence in turn, as one sequence does not fit."""
    run(abw, 2, 8192, 48, 48, 64, 8000, 3, [8192, 5000], packed=True)


def test_captured(abw):
    B, T, H, D, W = 2, 8192, 40, 64, 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn(B, T, H, D, generator=g, device="cuda").to(BF) for _ in range(4))
    o, lse = abw.attn_fwd_window(q, k, v, W)
    want = abw.attn_bwd_window(q, k, v, o, do, lse, W)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = abw.attn_bwd_window(q, k, v, o, do, lse, W)
    for _ in range(2):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    abw.device_check()
