"""The binding's short cuts into torch have public functions behind them, for a
torch that lacks them."""
import pytest
import torch

import transformer_attention_backward_gb300 as m


def test_none_is_called_without_a_look():
    source = open(m.__file__).read()
    assert source.count("torch._C") == source.count("getattr(torch._C, name, public)") == 1


@pytest.mark.gpu
def test_public_functions_do_the_same(monkeypatch):
    g = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn(2, 300, h, 64, generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2, 4))
    ld, s0 = torch.tensor([-0.1, -0.01], device="cuda"), torch.randn(2, 2, 64, 64, generator=g).cuda()

    def run():
        return m.lin_attn_fwd(q, k, v, ld, initial_state=s0, want_final_state=True) + m.lin_attn_bwd(q, k, v, do, ld)[:3]

    want = run()
    for name, function in zip(("_raw_stream", "_device_index", "_raw_alloc", "_raw_delete"), m._PUBLIC.values()):
        monkeypatch.setattr(m, name, function)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = run()
    torch.cuda.synchronize()
    m.device_check()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
