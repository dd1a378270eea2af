"""The workspace of the windowed backward: it holds the products' tiles of as many
heads as fit 2 GiB, or of one KV head, however large the call."""
import pytest

from transformer_attention_backward_gb300 import _binding as B

ROOM = 2 << 30


def tiles(T, window, sinks):
    """Pairs of 128-token blocks that meet, counted."""
    nb, n = (T + 127) // 128, 0
    for i in range(nb):
        for j in range(i + 1):
            n += i * 128 - window < j * 128 + 127 or j * 128 < sinks
    return n


@pytest.mark.parametrize("Bn,T,Hq,Hkv,window,sinks", [
    (1, 32768, 32, 32, 4096, 0), (1, 32768, 32, 32, 32768, 0), (1, 131072, 32, 8, 1024, 4), (64, 4096, 32, 8, 512, 4),
    (1000, 2048, 20, 5, 2048, 0), (7, 8192, 32, 32, 1024, 4), (1, 65536, 24, 12, 700, 300), (1, 131072, 8, 1, 131072, 0),
    (1, 131072, 8, 8, 131072, 131072)])
def test_the_workspace_is_bounded(Bn, T, Hq, Hkv, window, sinks):
    need = B.load().attn_bwd_window_workspace_bytes(Bn, T, Hq, Hkv, 128, window, sinks)
    head = tiles(T, window, sinks) * 32768 * (Hq // Hkv)
    whole = Bn * Hkv * head
    assert whole > ROOM                                      # a call that does not fit in one go
    fit = max(1, ROOM // head)                               # KV heads at one time
    stats = 8 * fit * (Hq // Hkv) * ((T + 127) // 128 * 128) + 1024
    # what is left: fp32 parts of blocks of 128 keys that go to several of 152 CTAs, 128 KB each, two at most
    # for a CTA's share and one for each block and head
    parts = (2 * 152 + fit * (T // 128)) * 131072
    assert need <= max(ROOM, head) + stats + parts


@pytest.mark.parametrize("Bn,T,Hq,Hkv,window,sinks", [(4, 2048, 20, 20, 512, 4), (1, 8192, 32, 32, 1024, 4), (2, 512, 20, 5, 128, 4)])
def test_what_fits_goes_in_one(Bn, T, Hq, Hkv, window, sinks):
    need = B.load().attn_bwd_window_workspace_bytes(Bn, T, Hq, Hkv, 128, window, sinks)
    assert need >= Bn * Hq * tiles(T, window, sinks) * 32768
