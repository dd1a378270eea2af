"""The fp32 states of the linear attention over long sequences of heads that
hardly decay: whatever error the decay of a whole chunk carried would grow
with the number of chunks."""
import math

import numpy as np
import pytest
import torch

from tests.helpers import to_np

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def abw():
    import transformer_attention_backward_gb300 as m
    m.library()
    return m


@pytest.mark.parametrize("T,D", [(20000, 128), (100001, 64)])
def test_states_of_slow_decays(abw, T, D):
    """Error of a state's 2-norm.  Weighted rows: powers to 2^-22, three bf16
    terms to 2^-25, some 35 additions of 2^-23 in the tensor core, each of the
    size of its own chunk's sum, so 38 2^-23 of the state's.  The state takes
    one rounding of 2^-24 a step of 64 tokens, N of them, in either direction:
    sqrt(N) 2^-24.  The decay of a chunk has to be exact for that: off by
    2^-25, the rounding of one fp32 number, it would move what is n chunks old
    by n 2^-25.  Single elements: 8 times that share of the mean square root."""
    H, scale = 6, 0.125
    decay = [-1e-6, -2.3e-6, -5e-6, -1.1e-5, -2.7e-5, -6e-5]
    g = torch.Generator().manual_seed(T)
    q, k, v, do = (torch.randn(1, T, H, D, generator=g).to(BF) for _ in range(4))
    s0, df = torch.randn(1, H, D, D, generator=g), torch.randn(1, H, D, D, generator=g)
    ld = torch.tensor(decay)
    dev = [x.cuda() for x in (q, k, v, do, ld)]
    _, fin = abw.lin_attn_fwd(*dev[:3], dev[4], scale, initial_state=s0.cuda(), want_final_state=True)
    din = abw.lin_attn_bwd(*dev, scale, dfinal_state=df.cuda(), want_dinitial_state=True)[3]
    abw.device_check()
    tol = (38 + math.sqrt(2 * ((T + 127) // 128)) / 2) * 2.0 ** -23
    t = np.arange(T, dtype=np.float64)[:, None]
    for h in range(H):
        a = float(ld[h])                        # the fp32 number
        whole = math.exp(a * T)
        x, y = to_np(k[0, :, h]), to_np(v[0, :, h])
        want = (np.exp(a * (T - 1 - t)) * x).T @ y + whole * to_np(s0[0, h])
        x, y = to_np(q[0, :, h]), to_np(do[0, :, h])
        back = (scale * np.exp(a * (t + 1)) * x).T @ y + whole * to_np(df[0, h])
        for got, ref in ((fin, want), (din, back)):
            err = to_np(got[0, h]) - ref
            rms = math.sqrt(float(np.mean(ref * ref)))
            rel = math.sqrt(float(np.mean(err * err))) / rms
            assert rel <= tol, (h, rel, tol)
            assert np.all(np.abs(err) <= 8 * tol * np.maximum(rms, np.abs(ref)))
