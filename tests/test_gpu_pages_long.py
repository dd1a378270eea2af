"""Paged caches whose tables hold more positions than the eviction keeps in shared
memory (40,960): the choice then forms a token's key again wherever it needs it.
The table's capacity decides, not the tokens in it.  Against the float64 oracle,
with the tolerances of the shorter tables."""
import pytest
import torch

from tests.test_gpu_pages import F, INF, NAN, abw, decode, evict, int32   # noqa: F401  (abw: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most,page", [(640, 64), (40961, 1), (641, 64), (1707, 24)])   # 40,960 and the next ones
@pytest.mark.parametrize("budget", [1, 3000])
def test_evict_at_the_border(abw, most, page, budget):
    n = most * page
    evict(abw, page + budget, [n, n - 1, 17], most, page, 1, 8, budget, min(4, budget // 2), min(64, budget // 2))


@pytest.mark.parametrize("page", [64, 24, 1000])
def test_evict_very_long(abw, page):
    most = 70000 // page + 1
    evict(abw, page, [70000, 41000], most, page, 2, 8, 9000, 4, 300)
    evict(abw, page, [most * page], most, page, 1, 64, 65001, 0, 1)        # nearly all


def test_evict_short_sequences_in_a_wide_table(abw):
    lengths = [0, 1, 31, 32, 33, 500, 1024, 1025, 3000]
    for page in (16, 24):
        evict(abw, page, lengths, 50000 // page, page, 1, 16, 500, 2, 30)
        evict(abw, page, lengths, 50000 // page, page, 1, 16, 1, 0, 0)


def test_evict_ties_and_odd_weights(abw):
    page, most = 24, 1800                                                  # 43,200 positions
    n = page * most
    g = torch.Generator().manual_seed(3)
    few = torch.randint(0, 3, (1, 2, n), generator=g).float()
    evict(abw, 3, [n], most, page, 2, 8, 20000, 2, 5, weights=few)
    evict(abw, 4, [n - 30], most, page, 2, 8, 999, 0, 0, weights=torch.zeros(1, 2, n))
    odd = torch.randn(1, 2, n, generator=g)
    odd[:, :, ::5], odd[:, :, 1::5], odd[:, :, 2::5], odd[:, :, 3::10], odd[:, :, 8::10] = NAN, -INF, INF, 0.0, -0.0
    for budget in (100, 10000, 24000, 30000):
        evict(abw, 5, [n - 7], most, page, 2, 8, budget, 1, 2, weights=odd)
    near_ones = 1.0 + torch.randint(0, 9, (1, 2, n), generator=g) * 2.0 ** -23
    evict(abw, 6, [n], most, page, 2, 8, 21000, 0, 3, weights=near_ones)


def test_evict_absent_pages(abw):
    gone = [(0, i) for i in range(0, 700, 3)] + [(0, 699), (1, 0), (1, 1)] + [(2, i) for i in range(700)]
    evict(abw, 7, [44800, 30000, 44800], 700, 64, 1, 8, 5000, 100, 100, absent=gone)
    evict(abw, 8, [44800, 300], 700, 64, 1, 8, 44000, 2, 2, absent=gone[:235], no_room=[(0, 1), (0, 400), (1, 0)])


def test_evict_does_not_depend_on_the_tables_width(abw):
    """A sequence keeps the same tokens in a table of its own length and in a
    wide one."""
    B, n, page, Hkv, D, budget = 3, 2000, 16, 2, 64, 700
    g = torch.Generator().manual_seed(9)
    pages = B * (n // page) + B * 44
    order = torch.randperm(pages, generator=g)
    table, new = int32(order[:B * 125].reshape(B, 125)), int32(order[B * 125:].reshape(B, 44))
    k, v = (torch.randn(pages, page, Hkv, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w = torch.rand(B, Hkv, n, generator=g).cuda()
    lens = int32([n, n - 700, n - 5])
    out = []
    for wide in (125, 2560, 2561, 6000):
        t = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
        t[:, :125] = table
        ww = torch.full((B, Hkv, wide * page), 1e30, device="cuda")
        ww[:, :, :n] = w
        kk, vv = k.clone(), v.clone()
        out.append(tuple(abw.kv_pages_evict(kk, vv, t, lens, ww, budget, new, sinks=3, recent=50)) + (kk, vv))
    abw.device_check()
    for other in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], other))


def test_decode_very_long(abw):
    decode(abw, 1, [70000, 41000, 5], 1094, 64, 4, 1, 64, weights=True)
    decode(abw, 2, [70000], 2917, 24, 3, 1, 64, F, weights=True)
    decode(abw, 3, [70000, 66000], 1094, 64, 4, 1, 128, window=50000, sinks=100, weights=True)
