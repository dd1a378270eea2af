"""Python integers that no C int holds are refused: ctypes would pass their low
32 bits, and the call would turn by other angles than asked."""
import pytest
import torch

import transformer_attention_backward_gb300 as m


def rotation(rotary_dim=None, sections=None, pos0=0, base=1e4):
    return m._rotation(2, 3, 64, base, rotary_dim, None, sections, pos0, torch.device("cpu"))


def test_pos0():
    assert rotation(pos0=2 ** 31 - 1)[4] == 2 ** 31 - 1 and rotation(pos0=-2 ** 31)[4] == -2 ** 31
    for bad in (2 ** 31, -2 ** 31 - 1, 2 ** 32 + 5):
        with pytest.raises(ValueError, match="pos0"):
            rotation(pos0=bad)
    assert rotation(pos0=2 ** 40, base=0.0)[4] == 0             # no rotation: not looked at


def test_rotary_dim_and_sections():
    assert rotation()[0] == 64 and rotation(rotary_dim=32, sections=[10, 6])[0] == 32
    with pytest.raises(ValueError, match="rotary_dim"):
        rotation(rotary_dim=2 ** 32 + 64)
    with pytest.raises(ValueError, match="sections"):
        rotation(sections=[2 ** 32 + 16, 16])


@pytest.mark.gpu
def test_far_start_is_refused():
    q = torch.zeros(1, 4, 2, 64, device="cuda")
    with pytest.raises(ValueError):
        m.qk_norm_rope_fwd(q, None, rope_base=1e4, pos0=2 ** 31)
    with pytest.raises(ValueError):
        m.qk_norm_rope_bwd(q, None, q, None, rope_base=1e4, pos0=2 ** 31)
    y, _ = m.qk_norm_rope_fwd(q, None, rope_base=1e4, pos0=2 ** 31 - 1)
    assert bool((y == 0).all())
