"""A budget that the new pages do not hold is refused before any memory of its
size is asked for."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("budget", [49, 20_000_000, 0, -1])
def test_refused_without_memory(budget):
    import transformer_attention_backward_gb300 as abw
    B, Hkv, page, D = 2, 2, 16, 64
    k, v = (torch.zeros(20, page, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.arange(8, dtype=torch.int32, device="cuda").reshape(B, 4)
    new = torch.arange(8, 14, dtype=torch.int32, device="cuda").reshape(B, 3)
    lens = torch.tensor([9, 60], dtype=torch.int32, device="cuda")
    sums = torch.zeros(B, Hkv, 64, device="cuda")
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    with pytest.raises((ValueError, abw.AbwError), match="budget"):
        abw.kv_pages_evict(k, v, table, lens, sums, budget, new)
    assert torch.cuda.max_memory_allocated() == held
