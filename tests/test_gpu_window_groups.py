"""The windowed attention where its heads are more than one scheduling group
takes, the last group narrower than the others: the items of every group, against
the definition in 64 bits on the GPU.  A forward group has 144 MB of K and V (a
block of 128 keys of D components is 512 D bytes), 700 tokens that see all of each
other 6 blocks: 384 pairs of heads of 128 with a KV head for each two, 768 heads of
64 of their own.  A backward group has 72 MB of q and dout, here 7 blocks a query
head: 82 and 329 KV heads.  Tolerances as for one group."""
import pytest
import torch

from tests.helpers import to_np
from tests.test_gpu_window import BF, TOL, abw, near   # noqa: F401  (abw: the fixture)

pytestmark = pytest.mark.gpu


def exact(q, k, v, o, do, scale, window, sinks):
    """One sequence [T][H][D] in 64 bits: o, lse, dq, dk, dv (for the given o)."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    q, k, v, o, do = (x.double().transpose(0, 1) for x in (q, k, v, o, do))
    kk, vv = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
    i = torch.arange(T, device=q.device)
    gap = i[:, None] - i[None, :]
    hidden = (gap < 0) | ((gap >= window) & (i >= sinks)[None, :])
    s = (scale * q @ kk.transpose(1, 2)).masked_fill(hidden, float("-inf"))
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    ds = p * (do @ vv.transpose(1, 2) - (do * o).sum(-1, keepdim=True))
    shared = lambda x: x.reshape(-1, G, T, D).sum(1).transpose(0, 1)
    return ((p @ vv).transpose(0, 1), lse, scale * (ds @ kk).transpose(0, 1), shared(scale * ds.transpose(1, 2) @ q),
            shared(p.transpose(1, 2) @ do))


@pytest.mark.parametrize("B,Hq,Hkv,D,window,sinks,lengths", [
    (9, 96, 48, 128, 700, 0, None),              # 432 pairs of heads: 384 and 48; 432 KV heads: 5 of 82 and 22
    (10, 80, 80, 64, 700, 3, None),              # 800 heads: 768 and 32; 329, 329 and 142
    (10, 80, 80, 64, 690, 0, [700, 0, 1, 129, 640, 700, 384, 77, 700, 513]),
    (9, 96, 48, 128, 699, 130, [700, 350, 700, 0, 128, 700, 5, 600, 257])])
def test_groups(abw, B, Hq, Hkv, D, window, sinks, lengths):
    T, scale = 700, 0.125
    g = torch.Generator(device="cuda").manual_seed(B + D)
    q, k, v, do = (torch.randn(B, T, h, D, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv, Hq))
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, lse = abw.attn_fwd_window(q, k, v, window, sinks, scale, lengths=ln)
    grads = abw.attn_bwd_window(q, k, v, o, do, lse, window, sinks, scale, lengths=ln)
    abw.device_check()
    most = float(q.abs().max() * k.abs().max()) * D * scale
    for b in range(B):
        n = T if lengths is None else lengths[b]
        assert bool((lse[b, :, n:] == float("-inf")).all())
        for x in (o,) + tuple(grads):
            assert not bool(x[b, n:].any())
        if n == 0:
            continue
        ro, rl, *rg = exact(q[b, :n], k[b, :n], v[b, :n], o[b, :n], do[b, :n], scale, window, sinks)
        near(o[b, :n], to_np(ro), TOL)
        assert float((lse[b, :, :n].double() - rl).abs().max()) <= 2.0 ** -20 * most
        least = 6 * D * 2.0 ** -24 * scale * float(max(q.abs().max(), k.abs().max()))
        for x, y in zip(grads, rg):
            near(x[b, :n], to_np(y), TOL, least)
