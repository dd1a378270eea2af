"""GPU parity of the paged cache: writing to its pages, attention of one new
token over it, and eviction by attention weight, against the float64 oracle.

Tolerances, on the 2-norm of an output's error over that of the output.  p
enters its product with at least 16 bits, fp32 queries with 24: bf16 outputs are
off by their own rounding, 2^-8, with 2^-16 for p, fp32 ones by the sums alone.
A score is a sum of D exact (or fp32-exact) products, off by 2^-23 of a running
sum each; weights and fp32 outputs are off by that as often as they add: (D +
positions / 16 + 16) 2^-23 (one addition a 16-token tile, 2^-22 for exp2 and its
argument)."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from tests.helpers import to_np

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def abw():
    import transformer_attention_backward_gb300 as m
    m.library()
    return m


def int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def near(got, ref, tol):
    g = to_np(got)
    assert g.shape == ref.shape and np.all(np.isfinite(g))
    if g.size == 0:
        return
    rms = math.sqrt(float(np.mean(ref * ref)))
    err = g - ref
    assert math.sqrt(float(np.mean(err * err))) <= tol * rms
    assert np.all(np.abs(err) <= 8 * tol * np.maximum(rms, np.abs(ref)))


def cache(seed, B, most, page, Hkv, D, spare=3):
    """Pages and a table of `most` entries a row, in no order; numpy's view of
    both beside them."""
    g = torch.Generator().manual_seed(seed)
    n = B * most + spare
    order = torch.randperm(n, generator=g).numpy()
    k, v = (torch.randn(n, page, Hkv, D, generator=g).to(BF) for _ in range(2))
    return k, v, order[:B * most].reshape(B, most).copy(), order[B * most:].copy()


def decode(abw, seed, lengths, most, page, Hq, Hkv, D, dtype=BF, window=None, sinks=0, weights=False, absent=(), scale=0.125,
           q_size=1.0):
    B = len(lengths)
    k, v, table, _ = cache(seed, B, most, page, Hkv, D)
    for b, i in absent:
        table[b, i] = -1 if (b + i) % 2 else k.shape[0]
    g = torch.Generator().manual_seed(seed + 1)
    q = (q_size * torch.randn(B, Hq, D, generator=g)).to(dtype)
    sums = torch.rand(B, Hkv, most * page, generator=g) if weights else None
    ro, rs = O.attn_decode_paged(to_np(q), to_np(k), to_np(v), table, lengths, scale, window, sinks, None if sums is None else to_np(sums))
    # whatever is not seen may hold anything
    for b, n in enumerate(lengths):
        for p, pg, row in O.page_rows(table[b], page, k.shape[0], 0, most * page):
            if p >= n or (window is not None and p < n - window and p >= sinks):
                k[pg, row], v[pg, row] = NAN, INF
    ds = None if sums is None else sums.cuda()
    o = abw.attn_decode_paged(q.cuda(), k.cuda(), v.cuda(), int32(table), int32(lengths), scale, window=window, sinks=sinks,
                              weight_sums=ds)
    abw.device_check()
    fp32 = (D + most * page / 16 + 16) * 2.0 ** -23 * max(1.0, q_size)
    near(o, ro, 2.0 ** -8 if dtype == BF else fp32)
    if weights:
        same = rs == to_np(sums)
        assert torch.equal(ds.cpu()[torch.from_numpy(same)], sums[torch.from_numpy(same)])
        near(ds, rs, fp32)
    return o, ds


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 64, 65, 127, 500, 1333])
def test_decode_lengths(abw, n, D, dtype):
    decode(abw, n + D, [n], 84, 16, 4, 2, D, dtype, weights=True)


@pytest.mark.parametrize("page", [1, 2, 7, 16, 24, 64, 100, 1000])
def test_decode_page_sizes(abw, page):
    decode(abw, page, [1000, 77, 999], (1000 + page - 1) // page, page, 8, 2, 128, weights=page % 2 == 0)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (5, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 1), (24, 2), (20, 5), (96, 3), (64, 2)])
def test_decode_heads(abw, Hq, Hkv, dtype):
    decode(abw, Hq, [300, 45], 20, 16, Hq, Hkv, 128, dtype, weights=True)
    decode(abw, Hq, [300, 45], 20, 16, Hq, Hkv, 64, dtype)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (17, 4), (100, 20), (333, 0), (999, 1), (2000, 5), (10, 500), (2 ** 31 - 1, 7)])
def test_decode_windows(abw, window, sinks):
    decode(abw, window % 97, [1000, 5, 0, 101, 640], 63, 16, 4, 1, 128, window=window, sinks=sinks, weights=True)
    decode(abw, window % 89, [1000, 5, 0, 101, 640], 42, 24, 4, 2, 64, F, window=window, sinks=sinks)


def test_decode_absent_pages(abw):
    """Entries that are no page's number: their tokens are not seen, rows that
    see nothing are 0; lengths below 0 and beyond the table are cut."""
    gone = [(0, 0), (0, 3), (1, 4), (2, 0), (2, 1), (2, 2), (2, 3), (2, 4), (3, 2)]
    for weights in (False, True):
        o, _ = decode(abw, 3, [80, 70, 80, 33, -4, 5000], 5, 16, 8, 2, 128, absent=gone, weights=weights)
        assert bool((o[2] == 0).all()) and bool((o[4] == 0).all())
    decode(abw, 4, [80, 70], 5, 16, 8, 2, 64, F, window=20, sinks=17, absent=[(0, 0), (1, 1), (1, 4)], weights=True)


def test_decode_ragged_batches(abw):
    """Runs of equal length cross sequences and heads at any place; one long
    sequence beside many short ones, and more sequences than threads."""
    r = np.random.default_rng(1)
    decode(abw, 1, [3000] + [int(x) for x in r.integers(0, 40, size=30)], 188, 16, 4, 2, 64, weights=True)
    decode(abw, 2, [int(x) for x in r.integers(0, 60, size=300)], 4, 16, 4, 2, 64, weights=True)
    decode(abw, 3, [0] * 200 + [900] + [0] * 99, 57, 16, 8, 1, 128, weights=True)
    decode(abw, 4, [4000, 4096, 3111], 64, 64, 32, 8, 128, weights=True)
    decode(abw, 5, [6000], 94, 64, 3, 1, 128, F, weights=True)


def test_decode_scores_far_apart(abw):
    for dtype in (BF, F):
        decode(abw, 6, [700, 300], 44, 16, 4, 2, 128, dtype, scale=1.0, q_size=4.0, weights=dtype == BF)
        decode(abw, 7, [700, 300], 44, 16, 4, 2, 128, dtype, scale=0.0, weights=True)
        decode(abw, 8, [700, 300], 44, 16, 4, 2, 128, dtype, scale=-0.3, weights=True)


def test_decode_sums_over_steps(abw):
    """Equal calls add equal weights, bit for bit; the sum over a row grows by
    the number of its query heads each step."""
    k, v, table, _ = cache(9, 3, 20, 16, 2, 128)
    q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    a = torch.zeros(3, 2, 320, device="cuda")
    b = torch.zeros(3, 2, 320, device="cuda")
    args = (q, k.cuda(), v.cuda(), int32(table), int32([320, 100, 0]))
    for step in range(1, 6):
        oa = abw.attn_decode_paged(*args, weight_sums=a)
        ob = abw.attn_decode_paged(*args, weight_sums=b)
        assert torch.equal(oa, ob) and torch.equal(a, b)
        total = a.double().sum(-1).cpu()
        assert torch.allclose(total, torch.tensor([4.0, 4.0, 0.0])[:, None].double() * step, rtol=1e-4, atol=0)


@pytest.mark.parametrize("D", [8, 64, 128])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_write(abw, page, D):
    B, T, Hkv = 4, 50, 3
    most = (90 + page - 1) // page
    k, v, table, _ = cache(page + D, B, most, page, Hkv, D)
    table[1, 0], table[2, most // 2] = -1, k.shape[0]
    g = torch.Generator().manual_seed(5)
    kv = torch.randn(B, T, 2 * Hkv + 1, D, generator=g).to(BF)
    nk, nv = kv[:, :, :Hkv], kv[:, :, Hkv:2 * Hkv]
    for starts, lengths in (([0, 3, 17, 39], None), ([-7, 60, 2 ** 31 - 20, -2 ** 31], [50, 50, 50, 50]), ([5, 5, 5, 5], [0, -3, 1, 9000])):
        rk, rv = O.kv_pages_write(to_np(nk), to_np(nv), to_np(k), to_np(v), table, starts, lengths)
        dk, dv, dkv = k.cuda(), v.cuda(), kv.cuda()
        abw.kv_pages_write(dkv[:, :, :Hkv], dkv[:, :, Hkv:2 * Hkv], dk, dv, int32(table), int32(starts),
                           lengths=None if lengths is None else int32(lengths))
        assert np.array_equal(to_np(dk), rk) and np.array_equal(to_np(dv), rv)
    k, v, table, _ = cache(1, 2, 64, 16, 20, 128)
    nk, nv = (torch.randn(2, 1000, 20, 128, generator=g).to(BF) for _ in range(2))
    rk, rv = O.kv_pages_write(to_np(nk), to_np(nv), to_np(k), to_np(v), table, [24, 0], [1000, 513])
    dk, dv = k.cuda(), v.cuda()
    abw.kv_pages_write(nk.cuda(), nv.cuda(), dk, dv, int32(table), int32([24, 0]), lengths=int32([1000, 513]))
    assert np.array_equal(to_np(dk), rk) and np.array_equal(to_np(dv), rv)


def evict(abw, seed, lengths, most, page, Hkv, D, budget, sinks=0, recent=1, weights=None, absent=(), no_room=()):
    B = len(lengths)
    fresh = (budget + page - 1) // page + 1
    k, v, table, rest = cache(seed, B, most, page, Hkv, D, spare=B * fresh + 2)
    new = rest[:B * fresh].reshape(B, fresh).copy()
    for b, i in absent:
        table[b, i] = -1 if (b + i) % 2 else k.shape[0] + 5
    for b, i in no_room:
        new[b, i] = -1
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(3 * torch.randn(B, Hkv, most * page, generator=g)) if weights is None else weights
    ref = O.kv_pages_evict(to_np(k), to_np(v), table, lengths, w.double().numpy(), budget, new, sinks, recent)
    dk, dv, dw = k.cuda(), v.cuda(), w.cuda()
    got = abw.kv_pages_evict(dk, dv, int32(table), int32(lengths), dw, budget, int32(new), sinks=sinks, recent=recent)
    abw.device_check()
    assert torch.equal(dw.cpu().nan_to_num(1e30), w.nan_to_num(1e30))
    assert np.array_equal(got[0].cpu().numpy(), ref[2]) and np.array_equal(got[1].cpu().numpy(), ref[3])
    assert np.array_equal(to_np(got[2]), ref[4], equal_nan=True)
    assert np.array_equal(to_np(dk), ref[0]) and np.array_equal(to_np(dv), ref[1])


@pytest.mark.parametrize("page", [1, 16, 24, 100])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 4, 16), (64, 32, 32), (200, 0, 0), (500, 4, 100)])
def test_evict(abw, page, budget, sinks, recent):
    evict(abw, page + budget, [300, 0, 1, 64, 65, 200, 299], (300 + page - 1) // page, page, 2, 64, budget, sinks, recent)


def test_evict_long(abw):
    evict(abw, 1, [5000, 1024, 1025, 2049], 40, 128, 3, 128, 1024, 4, 200)
    evict(abw, 2, [20000], 20000, 1, 1, 8, 3001, 1, 1)


def test_evict_ties_and_odd_weights(abw):
    n = 3000
    g = torch.Generator().manual_seed(3)
    few = torch.randint(0, 3, (2, 2, n), generator=g).float()              # many equal ones
    evict(abw, 3, [n, 2500], 125, 24, 2, 64, 1000, 2, 5, weights=few)
    evict(abw, 4, [n, 2500], 125, 24, 2, 64, 999, 0, 0, weights=torch.zeros(2, 2, n))
    odd = torch.randn(2, 2, n, generator=g)
    odd[:, :, ::5], odd[:, :, 1::5], odd[:, :, 2::5], odd[:, :, 3::10], odd[:, :, 8::10] = NAN, -INF, INF, 0.0, -0.0
    for budget in (100, 700, 1300, 1500, 1900, 2600):
        evict(abw, 5, [n, 2990], 125, 24, 2, 64, budget, 1, 2, weights=odd)
    near_ones = 1.0 + torch.randint(0, 9, (2, 2, n), generator=g) * 2.0 ** -23
    evict(abw, 6, [n, 1800], 125, 24, 2, 64, 1500, 0, 3, weights=near_ones)


def test_evict_absent_pages(abw):
    evict(abw, 7, [160, 150, 160], 10, 16, 2, 64, 40, 20, 20, absent=[(0, 0), (0, 9), (1, 5), (2, 1), (2, 3), (2, 4)])
    evict(abw, 8, [160, 150], 10, 16, 2, 64, 130, 2, 2, absent=[(0, i) for i in range(9)] + [(1, 2)])
    evict(abw, 9, [160, 150], 10, 16, 2, 64, 40, 2, 2, no_room=[(0, 1), (1, 0)])


def test_write_attend_evict_in_turn(abw):
    """Steps of a served batch: a prompt, then tokens one at a time, with an
    eviction under way, against the oracle's calls."""
    B, Hq, Hkv, D, page, most, budget = 3, 8, 2, 64, 8, 12, 24
    r = torch.Generator().manual_seed(11)
    k, v, table, rest = cache(12, B, most, page, Hkv, D, spare=B * most + 1)
    new = np.full((B, most), -1)
    new[:, :5] = rest[:B * 5].reshape(B, 5)
    kp, vp = k.cuda(), v.cuda()
    ek, ev = to_np(k), to_np(v)
    n = [30, 1, 17]
    sums, es = torch.zeros(B, Hkv, most * page, device="cuda"), np.zeros((B, Hkv, most * page))
    pk, pv = (torch.randn(B, 30, Hkv, D, generator=r).to(BF) for _ in range(2))
    abw.kv_pages_write(pk.cuda(), pv.cuda(), kp, vp, int32(table), int32([0] * B), lengths=int32(n))
    ek, ev = O.kv_pages_write(to_np(pk), to_np(pv), ek, ev, table, [0] * B, n)
    for step in range(20):
        if step == 10:
            kept, nl, sums = abw.kv_pages_evict(kp, vp, int32(table), int32(n), sums, budget, int32(new), sinks=2, recent=6)
            # the choice itself is compared in other tests; here the oracle takes the weights that the GPU summed
            ek, ev, ekept, en, es = O.kv_pages_evict(ek, ev, table, n, to_np(gpu_sums), budget, new, 2, 6)
            assert np.array_equal(kept.cpu().numpy(), ekept) and np.array_equal(nl.cpu().numpy(), en)
            n, table = [int(x) for x in en], new
        tk, tv = (torch.randn(B, 1, Hkv, D, generator=r).to(BF) for _ in range(2))
        q = torch.randn(B, Hq, D, generator=r).to(BF)
        abw.kv_pages_write(tk.cuda(), tv.cuda(), kp, vp, int32(table), int32(n))
        ek, ev = O.kv_pages_write(to_np(tk), to_np(tv), ek, ev, table, n)
        n = [x + 1 for x in n]
        o = abw.attn_decode_paged(q.cuda(), kp, vp, int32(table), int32(n), weight_sums=sums)
        ro, es = O.attn_decode_paged(to_np(q), ek, ev, table, n, 0.125, None, 0, es)
        near(o, ro, 2.0 ** -8)
        near(sums, es, (D + 22) * 2.0 ** -23 * 20)
        gpu_sums = sums.clone()
        es = to_np(sums)
    assert np.array_equal(to_np(kp), ek) and np.array_equal(to_np(vp), ev)
    abw.device_check()


def test_graph_and_streams(abw):
    k, v, table, rest = cache(13, 4, 30, 16, 2, 128, spare=40)
    q = torch.randn(4, 8, 128, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    kp, vp, tb, new = k.cuda(), v.cuda(), int32(table), int32(rest[:16].reshape(4, 4))
    lens = int32([480, 100, 0, 333])
    sums = torch.zeros(4, 2, 480, device="cuda")
    want = abw.attn_decode_paged(q, kp, vp, tb, lens, weight_sums=sums)
    want_sums, want_kept = sums.clone(), [x.clone() for x in abw.kv_pages_evict(kp, vp, tb, lens, sums, 64, new, sinks=2, recent=9)]
    ws = torch.empty(abw.attn_decode_paged_workspace_bytes(4, 8, 2, 128, 16, 30, None, 0, True), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sums.zero_()
    o = abw.attn_decode_paged(q, kp, vp, tb, lens, weight_sums=sums, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(o, want) and torch.equal(sums, want_sums)
    graphs = []
    for _ in range(2):                                       # two graphs that share the workspace, run in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sums.zero_()
            o = abw.attn_decode_paged(q, kp, vp, tb, lens, weight_sums=sums, workspace=ws)
            kept = abw.kv_pages_evict(kp, vp, tb, lens, sums, 64, new, sinks=2, recent=9)
        graphs.append((graph, o, kept))
    for n in ([480, 100, 0, 333], [479, 480, 3, 1], [480, 100, 0, 333]):   # lengths are read when a graph runs
        lens.copy_(int32(n))
        for graph, o, kept in graphs:
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            if n[0] == 480:
                assert torch.equal(o, want) and torch.equal(sums, want_sums)
                assert all(torch.equal(a, b) for a, b in zip(kept, want_kept))
            else:
                again = torch.zeros_like(sums)
                assert torch.equal(o, abw.attn_decode_paged(q, kp, vp, tb, lens, weight_sums=again)) and torch.equal(sums, again)
    abw.device_check()


def test_binding_refusals(abw):
    k, v, table, rest = cache(14, 2, 4, 16, 2, 64, spare=6)
    kp, vp, tb, lens = k.cuda(), v.cuda(), int32(table), int32([9, 60])
    q, sums = torch.randn(2, 4, 64, device="cuda"), torch.zeros(2, 2, 64, device="cuda")
    with pytest.raises(ValueError, match="window"):
        abw.attn_decode_paged(q, kp, vp, tb, lens, window=0)
    with pytest.raises(ValueError, match="sums"):
        abw.attn_decode_paged(q, kp, vp, tb, lens, weight_sums=sums[:, :, :63].contiguous())
    with pytest.raises(TypeError):
        abw.attn_decode_paged(q, kp.float(), vp, tb, lens)
    with pytest.raises(TypeError):
        abw.attn_decode_paged(q, kp, vp, tb.long(), lens)
    with pytest.raises(ValueError):
        abw.attn_decode_paged(q, kp, vp, tb[:1], lens)
    with pytest.raises(ValueError):
        abw.attn_decode_paged(q[:, :, :32].contiguous(), kp, vp, tb, lens)
    with pytest.raises(abw.AbwError, match="multiple of Hkv"):
        abw.attn_decode_paged(q[:, :3].contiguous(), kp, vp, tb, lens)
    new = int32(rest[:6].reshape(2, 3))
    for bad in (dict(budget=49), dict(budget=0), dict(budget=8, sinks=5, recent=4), dict(budget=8, recent=-1)):
        with pytest.raises((ValueError, abw.AbwError)):
            abw.kv_pages_evict(kp, vp, tb, lens, sums, new_table=new, **bad)
    with pytest.raises(ValueError):
        abw.kv_pages_write(torch.zeros(3, 1, 2, 64, dtype=BF, device="cuda"), torch.zeros(3, 1, 2, 64, dtype=BF, device="cuda"),
                           kp, vp, tb, lens)
    assert abw.attn_decode_paged(q[:0], kp, vp, tb[:0], lens[:0]).shape == (0, 4, 64)
    assert abw.kv_pages_evict(kp, vp, tb[:0], lens[:0], sums[:0], 4, new[:0])[0].shape == (0, 2, 4)


def test_rows_past_32_bits(abw):
    """A cache of more than 2^31 elements: the last pages' rows."""
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 20 GB")
    n, page, Hkv, D = 70000, 64, 4, 128                       # 2.3e9 elements, 4.6 GB each
    kp = torch.zeros(n, page, Hkv, D, dtype=BF, device="cuda")
    vp = torch.zeros(n, page, Hkv, D, dtype=BF, device="cuda")
    table = int32([[n - 1, 0, n - 2], [n // 2, n - 3, 5]])
    g = torch.Generator().manual_seed(2)
    nk, nv = (torch.randn(2, 150, Hkv, D, generator=g).to(BF) for _ in range(2))
    q = torch.randn(2, 8, D, generator=g).to(BF)
    abw.kv_pages_write(nk.cuda(), nv.cuda(), kp, vp, table, int32([0, 0]))
    sums = torch.zeros(2, Hkv, 192, device="cuda")
    o = abw.attn_decode_paged(q.cuda(), kp, vp, table, int32([150, 150]), weight_sums=sums)
    small = [to_np(x[table.cpu().flatten().unique().long().cuda()]) for x in (kp, vp)]
    index = {int(p): i for i, p in enumerate(table.cpu().flatten().unique())}
    st = [[index[int(p)] for p in row] for row in table.cpu()]
    ro, rs = O.attn_decode_paged(to_np(q), *small, st, [150, 150], 128 ** -0.5, None, 0, np.zeros((2, Hkv, 192)))
    near(o, ro, 2.0 ** -8)
    near(sums, rs, (D + 28) * 2.0 ** -23)
    new = int32([[n - 5], [n - 4]])
    kept, _, _ = abw.kv_pages_evict(kp, vp, table, int32([150, 150]), sums, 40, new, recent=5)
    j = kept[1, 2, 17].item()
    assert torch.equal(kp[n - 4, 17, 2].cpu(), nk[1, j, 2]) and torch.equal(vp[n - 4, 17, 2].cpu(), nv[1, j, 2])
    abw.device_check()
