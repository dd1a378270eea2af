"""The windowed attention where a wait runs out, and where offsets pass 32 bits."""
import contextlib
import re

import pytest
import torch

from transformer_attention_backward_gb300 import _binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def abw():
    import transformer_attention_backward_gb300 as m
    m.library()
    return m


@contextlib.contextmanager
def no_waiting(lib):
    lib.abw_set_wait_limit_ns(0)
    try:
        yield
    finally:
        lib.abw_set_wait_limit_ns(2_000_000_000)


def call(abw, T, Hq, Hkv, D, window, sinks, backward, lengths=None):
    """One call, as a function without arguments."""
    g = torch.Generator().manual_seed(T + D)
    q, k, v, do = (torch.randn(2, T, h, D, generator=g).to(BF).cuda() for h in (Hq, Hkv, Hkv, Hq))
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, lse = abw.attn_fwd_window(q, k, v, window, sinks, lengths=ln)
    if backward:
        return lambda: list(abw.attn_bwd_window(q, k, v, o, do, lse, window, sinks, lengths=ln))
    return lambda: list(abw.attn_fwd_window(q, k, v, window, sinks, lengths=ln))


CASES = [(100, 4, 2, 128, 30, 2, None), (300, 3, 3, 64, 100, 0, [300, 130]), (1000, 8, 2, 128, 200, 4, None),
         (1500, 40, 40, 64, 300, 4, [1500, 777]), (2500, 6, 2, 128, 100, 4, [1, 2400])]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d-%d/%d-D%d" % c[:4])
def test_gives_up_says_where_and_the_next_call_is_right(abw, case, backward):
    """A limit of 0 is over before any wait: the call reports it, lets its copies
    land and leaves the device as it was."""
    run, lib = call(abw, *case[:6], backward, case[6]), abw.library()
    want = [x.clone() for x in run()]
    abw.device_check()
    for _ in range(10):
        with no_waiting(lib):
            run()
            status = lib.abw_device_check(torch.cuda.current_stream().cuda_stream)
        assert status == B.ETIMEOUT
        assert re.search("first in the window (kv|dq)" if backward else "first in the window forward", B.last_error()), B.last_error()
        got = run()
        abw.device_check()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits(abw):
    """Rows of a packed tensor of more than 2^31 elements: its last tokens give
    what they give in a tensor of their own (the window reaches no further
    back)."""
    T, wide, Hq, Hkv, D, W, tail = 66000, 520, 4, 2, 64, 40, 200        # 66000 x 520 x 64 = 2.2e9 elements
    big = torch.zeros(1, T, wide, D, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(1)
    parts = [torch.randn(1, tail, h, D, generator=g).to(BF).cuda() for h in (Hq, Hkv, Hkv)]
    views = [big[:, :, wide - 9:wide - 5], big[:, :, wide - 5:wide - 3], big[:, :, wide - 3:wide - 1]]
    for x, y in zip(views, parts):
        x[:, T - tail:] = y
    o, lse = abw.attn_fwd_window(*views, W)
    ro, rl = abw.attn_fwd_window(*parts, W)
    keep = slice(T - tail + W, T)                                      # queries whose window lies in the tail
    # blocks of 128 begin elsewhere, so P is rounded at other scales: o is off by a rounding of it and one of P
    assert float((o[:, keep].float() - ro[:, W:].float()).abs().max()) <= 2 * 2.0 ** -8 * float(ro.float().abs().max())
    assert float((lse[:, :, keep] - rl[:, :, W:]).abs().max()) <= 1e-5
    do = torch.zeros_like(o)
    do[:, T - 100:] = torch.randn(1, 100, Hq, D, generator=g).to(BF).cuda()
    grads = abw.attn_bwd_window(*views, o, do, lse, W, dq=torch.empty_like(o))
    rgrads = abw.attn_bwd_window(*parts, ro, do[:, T - tail:].contiguous(), rl, W)
    abw.device_check()
    for a, b in zip(grads, rgrads):
        x, y = a[:, T - 100:].float(), b[:, tail - 100:].float()
        assert float((x - y).norm()) <= 3 ** 0.5 * 2.0 ** -8 * float(y.norm())
        assert not bool(a[:, :T - 100 - W - 128].any())                # no gradient comes so far back
