"""Pins of the oracle's per-head norm with rotation and of its linear
attention: central differences, the quadratic closed form, the split of a
sequence in two, and the single-token form."""
import numpy as np
import pytest

import oracle as O


def rng(seed):
    return np.random.default_rng(seed)


def weighted(f, w):
    return lambda x: float(np.sum(w * f(x)))


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("norm", [True, False])
def test_qk_norm_rope_backward_is_the_difference_quotient(interleaved, norm):
    r = rng(1)
    x, w, gamma = r.normal(size=(2, 3, 2, 8)), r.normal(size=(2, 3, 2, 8)), 1 + 0.1 * r.normal(size=8)
    theta = O.section_angles(r.integers(-50, 50, size=(2, 2, 3)), 6, 100.0, [2, 1])
    g = gamma if norm else None
    dx, dg = O.qk_norm_rope_backward(x, g, w, 1e-3, theta, 6, interleaved)
    f = weighted(lambda z: O.qk_norm_rope_forward(z, g, 1e-3, theta, 6, interleaved), w)
    assert O.check_gradient(dx, O.numerical_grad(f, x), 1e-6)
    if norm:
        f = weighted(lambda z: O.qk_norm_rope_forward(x, z, 1e-3, theta, 6, interleaved), w)
        assert O.check_gradient(dg, O.numerical_grad(f, gamma), 1e-6)


def test_section_angles_take_each_axis_for_its_pairs():
    pos = np.array([[[3, 4]], [[10, 20]]])                     # two axes, one sequence, two tokens
    th = O.section_angles(pos, 8, 16.0, [1, 3])
    inv = 16.0 ** (-2.0 * np.arange(4) / 8)
    assert np.allclose(th[0, 0], [3 * inv[0], 10 * inv[1], 10 * inv[2], 10 * inv[3]])
    assert np.allclose(th[0, 1], [4 * inv[0], 20 * inv[1], 20 * inv[2], 20 * inv[3]])


def lin_case(seed, B=2, T=5, Hq=4, Hkv=2, D=3):
    r = rng(seed)
    return (r.normal(size=(B, T, Hq, D)), r.normal(size=(B, T, Hkv, D)), r.normal(size=(B, T, Hkv, D)),
            -np.abs(r.normal(size=Hkv)), r.normal(size=(B, Hkv, D, D)))


def test_lin_attn_is_the_masked_product():
    q, k, v, ld, s0 = lin_case(2)
    o, s = O.lin_attn_forward(q, k, v, ld, 0.3, s0)
    T = q.shape[1]
    t = np.arange(T)
    for h in range(4):
        w = np.tril(np.exp(ld[h // 2] * (t[:, None] - t[None, :])))
        ref = 0.3 * ((w * (q[1, :, h] @ k[1, :, h // 2].T)) @ v[1, :, h // 2]
                     + np.exp(ld[h // 2] * (t + 1))[:, None] * (q[1, :, h] @ s0[1, h // 2]))
        assert np.allclose(o[1, :, h], ref)
    fall = np.exp(ld[0] * (T - 1 - t))[:, None]
    assert np.allclose(s[1, 0], np.exp(ld[0] * T) * s0[1, 0] + (fall * k[1, :, 0]).T @ v[1, :, 0])


@pytest.mark.parametrize("lengths", [None, [5, 2], [0, 3]])
def test_lin_attn_backward_is_the_difference_quotient(lengths):
    q, k, v, ld, s0 = lin_case(3)
    r = rng(4)
    w, ws = r.normal(size=q.shape), r.normal(size=s0.shape)
    dq, dk, dv, ds = O.lin_attn_backward(q, k, v, w, ld, 0.4, s0, ws, lengths)

    def f(q=q, k=k, v=v, s0=s0):
        o, s = O.lin_attn_forward(q, k, v, ld, 0.4, s0, lengths)
        return float(np.sum(w * o) + np.sum(ws * s))

    assert O.check_gradient(dq, O.numerical_grad(lambda x: f(q=x), q), 1e-6)
    assert O.check_gradient(dk, O.numerical_grad(lambda x: f(k=x), k), 1e-6)
    assert O.check_gradient(dv, O.numerical_grad(lambda x: f(v=x), v), 1e-6)
    assert O.check_gradient(ds, O.numerical_grad(lambda x: f(s0=x), s0), 1e-6)


def test_lin_attn_split_in_two_and_decode_agree():
    q, k, v, ld, s0 = lin_case(5)
    o, s = O.lin_attn_forward(q, k, v, ld, 0.4, s0)
    o1, s1 = O.lin_attn_forward(q[:, :3], k[:, :3], v[:, :3], ld, 0.4, s0)
    o2, s2 = O.lin_attn_forward(q[:, 3:], k[:, 3:], v[:, 3:], ld, 0.4, s1)
    assert np.allclose(o, np.concatenate([o1, o2], 1)) and np.allclose(s, s2)
    state = s0
    for t in range(q.shape[1]):
        ot, state = O.lin_attn_decode(q[:, t], k[:, t], v[:, t], state, ld, 0.4)
        assert np.allclose(ot, o[:, t])
    assert np.allclose(state, s)


def test_a_planted_mistake_is_seen():
    """The difference quotient tells a backward that forgets a decay apart."""
    q, k, v, ld, s0 = lin_case(6)
    w = rng(7).normal(size=q.shape)
    _, dk, _, _ = O.lin_attn_backward(q, k, v, w, np.zeros_like(ld), 0.4, s0)
    f = weighted(lambda x: O.lin_attn_forward(q, x, v, ld, 0.4, s0)[0], w)
    assert not O.check_gradient(dk, O.numerical_grad(f, k), 1e-3)
