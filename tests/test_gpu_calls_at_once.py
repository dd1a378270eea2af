"""The windowed attention and the paged cache's calls on several streams at one
time, each with memory of its own: they give what they give alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def abw():
    import transformer_attention_backward_gb300 as m
    m.library()
    return m


def attention(abw, seed, T, Hq, Hkv, D, window):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, do = (torch.randn(2, T, h, D, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv, Hq))

    def run(stream):
        o, lse = abw.attn_fwd_window(q, k, v, window, 4, stream=stream)
        return [o, lse] + list(abw.attn_bwd_window(q, k, v, o, do, lse, window, 4, stream=stream))
    return run


def serving(abw, seed, B, n, page):
    """A cache of its own: an attended step, then an eviction by its weights."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    most, budget = n // page, n // 4
    fresh = budget // page + 1
    order = torch.randperm(B * (most + fresh), generator=g, device="cuda").to(torch.int32)
    table, new = order[:B * most].reshape(B, most).contiguous(), order[B * most:].reshape(B, fresh).contiguous()
    k, v = (torch.randn(B * (most + fresh), page, 2, 128, generator=g, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(B, 8, 128, generator=g, device="cuda").to(BF)
    lens = torch.tensor([n - (b * 37) % n for b in range(B)], dtype=torch.int32, device="cuda")
    sums = torch.zeros(B, 2, n, device="cuda")

    def run(stream):
        with torch.cuda.stream(stream):
            sums.zero_()
        o = abw.attn_decode_paged(q, k, v, table, lens, weight_sums=sums, stream=stream)
        kept = abw.kv_pages_evict(k, v, table, lens, sums, budget, new, sinks=2, recent=9, stream=stream)
        rows = new.flatten().long()
        with torch.cuda.stream(stream):
            return [o, sums.clone(), *kept, k[rows], v[rows]]
    return run


def test_calls_at_once(abw):
    calls = [attention(abw, 1, 700, 8, 2, 128, 100), attention(abw, 2, 1500, 6, 6, 64, 1500), serving(abw, 3, 40, 640, 16),
             serving(abw, 4, 3, 48000, 64), attention(abw, 5, 130, 20, 5, 128, 64)]
    here = torch.cuda.current_stream()
    want = [[x.clone() for x in run(here)] for run in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [[] for _ in calls]
        for turn in range(3):                                # queued behind one another on each stream
            for i, (run, stream) in enumerate(zip(calls, streams)):
                got[i] = run(stream)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            # rows behind the last kept token are not written, and the same in both
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    abw.device_check()
