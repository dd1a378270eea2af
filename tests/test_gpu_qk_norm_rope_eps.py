"""qk_norm_rope_fwd / _bwd with eps = 0, which the header allows: groups of
lanes that have no row (behind the last token, or where the heads do not fill
a group's steps) must leave dgamma alone.  Inputs without a row of zeros, so
every value is defined."""
import pytest
import torch

from tests.test_gpu_qk_norm_rope import abw, check  # noqa: F401  (abw: the fixture)

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,dy", [(BF, F), (BF, BF), (F, F), (F, BF)])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot", [
    (1, 1, 1, 1, 128, 128),        # one row: all other lane groups of the block are without one
    (3, 7, 5, 3, 64, 32),          # heads that their groups' steps do not divide
    (2, 301, 3, 1, 256, 256),
    (1, 9, 5, 2, 512, 64),
    (1, 3, 3, 2, 34, 14),          # one pair a lane
    (1, 9, 260, 3, 64, 64),        # rows through shared memory
    (2, 6001, 5, 4, 128, 96),      # ... whose groups go on from token to token
])
def test_groups_without_a_row(abw, B, T, Hq, Hkv, D, rot, dtype, dy):  # noqa: F811
    for inter in (True, False):
        check(abw, B, T, Hq, Hkv, D, rot, None, 10000.0, inter, dtype, dy, eps=0.0, seed=B + T + D)


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("dtype", [BF, F])
def test_a_nan_stays_one(abw, dtype, eps):  # noqa: F811
    """The norm of a row with a NaN is one, so all of its outputs and of dgamma."""
    q = torch.randn(2, 5, 3, 64, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    q[1, 2, 1, 7] = float("nan")
    g = torch.ones(64, device="cuda")
    y, _ = abw.qk_norm_rope_fwd(q, None, g, eps=eps, rope_base=1e4)
    dx, _, dg, _ = abw.qk_norm_rope_bwd(q, None, torch.ones_like(q, dtype=F), None, g, eps=eps, rope_base=1e4)
    assert bool(torch.isnan(y[1, 2, 1]).all()) and int(torch.isnan(y).sum()) == 64
    assert bool(torch.isnan(dx[1, 2, 1]).all()) and int(torch.isnan(dx).sum()) == 64
    assert bool(torch.isnan(dg).all())
