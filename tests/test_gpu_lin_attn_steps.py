"""The single-token form over many tokens, heads that hardly decay: the decay of
one token, as one fp32 number, is off by up to 2^-25, the same way every time."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_states_after_many_tokens(dtype):
    """Error of a state's 2-norm after N tokens: two roundings of 2^-24 a token,
    which the tokens' random products keep independent, so sqrt(2 N) 2^-24, and 8
    2^-24 for the products themselves.  A decay off by 2^-25 would take N 2^-25."""
    import transformer_attention_backward_gb300 as abw
    H, D, N = 6, 64, 4000
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    ld = torch.tensor([-1e-6, -3.3e-6, -9e-6, -2.1e-5, -7.7e-5, -2e-4], device="cuda")
    state, k, v = n(1, H, D, D), n(N, H, D).to(dtype), n(N, H, D).to(dtype)
    want = state[0].double()
    q = torch.zeros(1, H, D, device="cuda", dtype=dtype)
    for t in range(N):
        abw.lin_attn_decode(q, k[t:t + 1], v[t:t + 1], state, ld, 1.0)
    a = ld.double()
    age = torch.arange(N - 1, -1, -1, device="cuda", dtype=torch.float64)
    w = torch.exp(age[:, None] * a[None])
    want = torch.exp(N * a)[:, None, None] * want + torch.einsum("th,thd,the->hde", w, k.double(), v.double())
    rel = ((state[0].double() - want).pow(2).mean((1, 2)) / want.pow(2).mean((1, 2))).sqrt()
    assert float(rel.max()) <= (math.sqrt(2 * N) + 8) * 2.0 ** -24, rel.tolist()


def test_one_token_of_strong_and_no_decay():
    """a = 1 adds to the state, a = 0 leaves the token alone, an infinity stays."""
    import transformer_attention_backward_gb300 as abw
    ld = torch.tensor([0.0, -math.inf, -1e-5, -0.6, -0.7, -90.0], device="cuda")
    s0 = torch.randn(1, 6, 64, 64, device="cuda")
    k, v = torch.randn(1, 6, 64, device="cuda"), torch.randn(1, 6, 64, device="cuda")
    state = s0.clone()
    abw.lin_attn_decode(torch.zeros_like(k), k, v, state, ld, 1.0)
    want = torch.exp(ld.double())[:, None, None] * s0[0].double() + k[0].double()[:, :, None] * v[0].double()[:, None, :]
    size = torch.exp(ld.double())[:, None, None] * s0[0].double().abs() + (k[0].double()[:, :, None] * v[0].double()[:, None, :]).abs()
    assert bool(((state[0].double() - want).abs() <= 4 * 2.0 ** -24 * size + 1e-37).all())
    for h in (0, 2, 3):
        state[0, h, 5, 6] = math.inf
    abw.lin_attn_decode(torch.zeros_like(k), torch.zeros_like(k), v, state, ld, 1.0)
    assert all(bool(torch.isposinf(state[0, h, 5, 6])) for h in (0, 2, 3)) and not bool(torch.isnan(state).any())
