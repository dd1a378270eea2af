"""What the tensor-core kernels do when a wait runs out: they say so, let their
copies land, and leave the device as it was, so that the next call is right.
Sizes whose loads all fit the rings (the loading role is through with its
loop before any other role gives up), and larger ones."""
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


def linear(abw, T, Hq, Hkv, D, state, backward, seed=0):
    """One call of the linear attention, as a function without arguments."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    q, k, v, do = (n(2, T, h, D).to(BF).cuda() for h in (Hq, Hkv, Hkv, Hq))
    ld = -(2.0 ** -(1.0 + torch.arange(Hkv))).cuda()
    s0, df = (n(2, Hkv, D, D).cuda(), n(2, Hkv, D, D).cuda()) if state else (None, None)
    if backward:
        return lambda: [x for x in abw.lin_attn_bwd(q, k, v, do, ld, 0.125, initial_state=s0, dfinal_state=df,
                                                    want_dinitial_state=state) if x is not None]
    return lambda: [x for x in abw.lin_attn_fwd(q, k, v, ld, 0.125, initial_state=s0, want_final_state=state) if x is not None]


def softmax(abw, T, Hq, Hkv, backward):
    """One call of the causal softmax attention."""
    g = torch.Generator().manual_seed(T)
    q, k, v, do = (torch.randn(2, T, h, 128, generator=g).to(BF).cuda() for h in (Hq, Hkv, Hkv, Hq))
    o, lse = abw.attn_fwd_causal(q, k, v)
    if backward:
        return lambda: list(abw.attn_bwd_causal(q, k, v, o, do, lse, rope_base=1e4))
    return lambda: list(abw.attn_fwd_causal(q, k, v))


def same(got, want):
    """Equal bits; the softmax backward's key blocks that several blocks share
    add their parts in any order: up to four of them, so a few roundings of
    the largest."""
    return all(torch.equal(a, b) or (a.dtype == torch.float32 and bool((a - b).abs().max() <= 4 * 2.0 ** -24 * b.abs().max()))
               for a, b in zip(got, want))


CALLS = [pytest.param(lambda m, a=a: linear(m, *a), id="lin-T%d-%d/%d-D%d-state%d-bwd%d" % a) for a in [
    (100, 4, 2, 128, False, False), (100, 4, 2, 64, True, False), (300, 4, 2, 128, False, True), (128, 4, 4, 128, True, True),
    (128, 2, 2, 64, True, True), (700, 4, 1, 128, True, True), (1500, 8, 8, 64, True, True), (900, 40, 40, 128, False, True)]]
CALLS += [pytest.param(lambda m, a=a: softmax(m, *a), id="softmax-T%d-%d/%d-bwd%d" % a) for a in [
    (100, 4, 2, False), (128, 4, 4, True), (1000, 4, 2, False), (1000, 8, 2, True)]]


@pytest.mark.parametrize("make", CALLS)
def test_next_call_is_right(abw, make):
    call, lib = make(abw), abw.library()
    want = [x.clone() for x in call()]
    abw.device_check()
    for _ in range(3):
        with no_waiting(lib):
            got = call()
            status = lib.abw_device_check(torch.cuda.current_stream().cuda_stream)
        assert status in (B.OK, B.ETIMEOUT)
        if status == B.OK:
            assert same(got, want)
        got = call()
        abw.device_check()
        assert same(got, want)


def one_chunk(abw, Hq, Hkv):
    """Gradients of one chunk from a given state: the walk only hands it on."""
    g = torch.Generator().manual_seed(Hq)
    q, k, v, do = (torch.randn(2, 100, h, 128, generator=g).to(BF).cuda() for h in (Hq, Hkv, Hkv, Hq))
    s0, ld = torch.randn(2, Hkv, 128, 128, generator=g).cuda(), torch.full((Hkv,), -0.1, device="cuda")
    return lambda: list(abw.lin_attn_bwd(q, k, v, do, ld, 0.125, initial_state=s0)[:3])


KERNELS = [("linear attention output", lambda m: linear(m, 100, 4, 2, 128, False, False)),
           ("linear attention output", lambda m: linear(m, 500, 4, 2, 64, False, True)),
           ("linear attention output", lambda m: one_chunk(m, 4, 2)),
           ("linear attention state", lambda m: linear(m, 100, 4, 2, 64, True, False)),
           ("linear attention state", lambda m: linear(m, 3000, 4, 4, 128, True, True)),
           ("linear attention gradient", lambda m: one_chunk(m, 4, 4)),
           ("causal forward", lambda m: softmax(m, 128, 4, 2, False)),
           ("causal forward", lambda m: softmax(m, 2000, 4, 2, False)),
           ("causal (kv|dq)", lambda m: softmax(m, 128, 4, 2, True)),          # dq's blocks start in kv's tail
           ("causal (kv|dq)", lambda m: softmax(m, 2000, 4, 2, True))]


@pytest.mark.parametrize("kernel,make", KERNELS, ids=lambda x: x.replace(" ", "_") if isinstance(x, str) else "")
def test_gives_up_and_says_where(abw, kernel, make):
    """A limit of 0 is over before any wait: every such call reports it, and
    names the kernel that came first."""
    call, lib = make(abw), abw.library()
    want = [x.clone() for x in call()]
    abw.device_check()
    for _ in range(20):
        with no_waiting(lib):
            call()
            status = lib.abw_device_check(torch.cuda.current_stream().cuda_stream)
        assert status == B.ETIMEOUT
        assert re.search(f"first in the {kernel}", B.last_error()), B.last_error()
        got = call()
        abw.device_check()
        assert same(got, want)


def test_names_the_warp(abw):
    """Blocks of up to 19 warps: the walk's products are issued by warps 1 and
    18, and one of the two is the first to report."""
    call, lib = linear(abw, 600, 8, 8, 128, True, False), abw.library()
    for _ in range(40):
        with no_waiting(lib):
            call()
            assert lib.abw_device_check(torch.cuda.current_stream().cuda_stream) == B.ETIMEOUT
        assert re.search(r"warp (1|18), block", B.last_error()), B.last_error()
