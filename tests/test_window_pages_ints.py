"""Workspace sizes for a window or a number of first tokens that no C int holds:
refused, as the calls themselves refuse them, and not those of the low 32 bits."""
import pytest

import transformer_attention_backward_gb300 as m


@pytest.mark.parametrize("window,sinks", [(2 ** 31, 0), (2 ** 32 + 8, 0), (8, 2 ** 31), (8, 2 ** 32), (-2 ** 31 - 1, 0)])
def test_refused(window, sinks):
    with pytest.raises(ValueError, match="32 bits"):
        m.attn_bwd_window_workspace_bytes(2, 300, 4, 2, 64, window, sinks)
    with pytest.raises(ValueError, match="32 bits"):
        m.attn_decode_paged_workspace_bytes(2, 4, 2, 64, 16, 100, window, sinks, True)


def test_the_largest_ones():
    most = 2 ** 31 - 1
    assert m.attn_bwd_window_workspace_bytes(2, 300, 4, 2, 64, most, 0) == m.attn_bwd_window_workspace_bytes(2, 300, 4, 2, 64, 300, 0)
    size = m.attn_decode_paged_workspace_bytes
    assert size(2, 4, 2, 64, 16, 100, most, most, True) == size(2, 4, 2, 64, 16, 100, None, 0, True) > 0
