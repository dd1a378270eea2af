"""Pins of the oracle's windowed attention and paged cache: the mask written
out, central differences, the causal attention as the widest window, and the
paged forms against dense ones."""
import numpy as np
import pytest

import oracle as O


def rng(seed):
    return np.random.default_rng(seed)


def test_window_mask_written_out():
    m = O.window_mask(6, 2, 1).astype(int)
    assert m.tolist() == [[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0],
                          [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert np.array_equal(O.window_mask(5, 1, 0), np.eye(5, dtype=bool))
    assert np.array_equal(O.window_mask(5, 9, 3), np.tril(np.ones((5, 5), bool)))


@pytest.mark.parametrize("window,sinks,lengths", [(2, 1, None), (3, 0, [4, 0]), (9, 2, [5, 1])])
def test_window_backward_is_the_difference_quotient(window, sinks, lengths):
    r = rng(1)
    q, k, v, w = r.normal(size=(2, 5, 4, 3)), r.normal(size=(2, 5, 2, 3)), r.normal(size=(2, 5, 2, 3)), r.normal(size=(2, 5, 4, 3))
    grads = O.attn_window_backward(q, k, v, w, 0.7, window, sinks, lengths)
    for i, g in enumerate(grads):
        def f(x):
            a = [q, k, v]
            a[i] = x
            return float(np.sum(w * O.attn_window_forward(*a, 0.7, window, sinks, lengths)[0]))
        assert O.check_gradient(g, O.numerical_grad(f, [q, k, v][i]), 1e-6)


def test_the_widest_window_is_the_causal_attention():
    r = rng(2)
    q, k, v = r.normal(size=(1, 7, 4, 4)), r.normal(size=(1, 7, 2, 4)), r.normal(size=(1, 7, 2, 4))
    o, lse = O.attn_window_forward(q, k, v, 0.5, 7)
    ro, rl = O.causal_forward(q, k, v, 0.5)
    assert np.allclose(o, ro) and np.allclose(lse, rl)
    g, rg = O.attn_window_backward(q, k, v, o, 0.5, 100, 3), O.causal_backward(q, k, v, o, 0.5, 0.0, 0)
    assert all(np.allclose(a, b) for a, b in zip(g, rg))
    assert all(np.allclose(a, b) for a, b in zip(O.attn_window_backward(q, k, v, o, 0.5, 100, 3, o=ro), rg))


def paged(seed, B, lengths, page=3, Hkv=2, D=4, spare=4):
    r = rng(seed)
    each = (max(max(lengths), 1) + page - 1) // page
    n = B * each + spare
    order = r.permutation(n)
    return (r.normal(size=(n, page, Hkv, D)), r.normal(size=(n, page, Hkv, D)), order[:B * each].reshape(B, each), order[B * each:])


@pytest.mark.parametrize("window,sinks", [(None, 0), (3, 0), (2, 1)])
def test_paged_decode_is_the_last_row(window, sinks):
    """Written token by token, the cache's last query is the window's last."""
    r = rng(3)
    n = 8
    q, k, v = r.normal(size=(1, n, 4, 4)), r.normal(size=(1, n, 2, 4)), r.normal(size=(1, n, 2, 4))
    kp, vp, table, _ = paged(4, 1, [n])
    for t in range(n):
        kp, vp = O.kv_pages_write(k[:, t:t + 1], v[:, t:t + 1], kp, vp, table, [t])
    sums = np.zeros((1, 2, table.shape[1] * 3))
    o, sums = O.attn_decode_paged(q[:, -1], kp, vp, table, [n], 0.5, window, sinks, sums)
    ref, _ = O.attn_window_forward(q, k, v, 0.5, window or n, sinks)
    assert np.allclose(o, ref[:, -1])
    seen = O.window_mask(n, window or n, sinks)[-1]
    assert np.allclose(sums.sum(-1), 2.0) and np.all((sums[0, :, :n] > 0) == seen)


def test_absent_pages_and_empty_rows():
    kp, vp, table, _ = paged(5, 3, [7, 7, 7])
    table[0, 1], table[1, :] = -1, 99
    q = rng(6).normal(size=(3, 2, 4))
    o, sums = O.attn_decode_paged(q, kp, vp, table, [7, 7, 0], 0.5, None, 0, np.zeros((3, 2, 9)))
    assert np.all(o[1:] == 0) and np.all(sums[1:] == 0) and np.all((sums[0, 0] > 0) == [1, 1, 1, 0, 0, 0, 1, 0, 0])


def test_eviction_by_hand():
    kp, vp, table, fresh = paged(7, 1, [7], Hkv=1)
    w = np.array([[[0.1, 5.0, 3.0, 3.0, np.nan, 3.0, 0.0, 9.0, 9.0]]])
    k2, v2, kept, n, sums = O.kv_pages_evict(kp, vp, table, [7], w, 4, [fresh[:2]], sinks=1, recent=1)
    assert kept.tolist() == [[[0, 1, 2, 6]]] and n.tolist() == [4]        # of the equal ones the first
    assert sums[0, 0].tolist() == [0.1, 5.0, 3.0, 0.0, 0.0, 0.0]
    assert np.array_equal(k2[fresh[0], :, 0], [kp[table[0, 0], 0, 0], kp[table[0, 0], 1, 0], kp[table[0, 0], 2, 0]])
    assert np.array_equal(v2[fresh[1], 0, 0], vp[table[0, 2], 0, 0])
    _, _, kept, n, _ = O.kv_pages_evict(kp, vp, table, [3], w, 4, [fresh[:2]])
    assert kept.tolist() == [[[0, 1, 2, -1]]] and n.tolist() == [3]
