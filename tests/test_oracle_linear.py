"""Pins of the fp64 linear-attention and norm-rotation oracle against closed forms."""

import numpy as np

import oracle


def _rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def test_no_decay_is_causal_attention_without_softmax():
    q, k, v = _rand(9, 2, 5, seed=1), _rand(9, 2, 5, seed=2), _rand(9, 2, 4, seed=3)
    o, hT = oracle.linear_recurrence(q, k, v, np.zeros((9, 2)), scale=0.5)
    p = np.tril(np.einsum("ihk,jhk->hij", q, k))
    assert np.allclose(o, 0.5 * np.einsum("hij,jhv->ihv", p, v))
    assert np.allclose(hT[0], np.einsum("jhv,jhk->hvk", v, k))


def test_decay_weights_and_initial_state():
    q, k, v = _rand(6, 1, 3, seed=4), _rand(6, 1, 3, seed=5), _rand(6, 1, 3, seed=6)
    g = -np.abs(_rand(6, 1, seed=7))
    h0 = _rand(1, 1, 3, 3, seed=8)
    o, hT = oracle.linear_recurrence(q, k, v, g, h0)
    G = np.cumsum(g[:, 0])
    w = np.tril(np.exp(G[:, None] - G[None, :]))
    ref = (w * (q[:, 0] @ k[:, 0].T)) @ v[:, 0] + np.exp(G)[:, None] * (q[:, 0] @ h0[0, 0].T)
    assert np.allclose(o[:, 0], ref)
    assert np.allclose(hT[0, 0], np.exp(G[-1]) * h0[0, 0]
                       + (v[:, 0] * np.exp(G[-1] - G)[:, None]).T @ k[:, 0])


def test_minus_infinity_drops_the_state():
    q, k, v = (_rand(5, 2, 4, seed=s) for s in (11, 12, 13))
    g = np.zeros((5, 2))
    g[3] = -np.inf
    o, hT = oracle.linear_recurrence(q, k, v, g, h0=_rand(1, 2, 4, 4, seed=14))
    o2, hT2 = oracle.linear_recurrence(q[3:], k[3:], v[3:], np.zeros((2, 2)))
    assert np.allclose(o[3:], o2) and np.allclose(hT, hT2)


def test_packing_head_groups_and_partial_advance():
    q, k, v = _rand(7, 2, 4, seed=21), _rand(7, 2, 4, seed=22), _rand(7, 6, 4, seed=23)
    g = -np.abs(_rand(6, seed=24))
    o, hT = oracle.linear_recurrence(q, k, v, g, cu_seqlens=[0, 3, 3, 7], n_advance=[2, 0, 4])
    for h in range(6):
        s = np.s_[h // 3:h // 3 + 1]
        for n, (a, b, adv) in enumerate([(0, 3, 2), (3, 3, 0), (3, 7, 4)]):
            one, _ = oracle.linear_recurrence(q[a:b, s], k[a:b, s], v[a:b, h:h + 1], g[h:h + 1])
            _, st = oracle.linear_recurrence(q[a:a + adv, s], k[a:a + adv, s],
                                             v[a:a + adv, h:h + 1], g[h:h + 1])
            assert np.allclose(o[a:b, h:h + 1], one) and np.allclose(hT[n, h], st[0, 0])


def test_rotation_by_quarter_turns_and_relative_positions():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    f = [np.pi / 2, np.pi]
    y = oracle.norm_rope(x, [1], f, eps=None)
    assert np.allclose(y[0, 0], [-3, -2, 1, -4, 5, 6, 7, 8])  # (1,3): quarter turn, (2,4): half
    y = oracle.norm_rope(x, [1], f, eps=None, interleaved=True)
    assert np.allclose(y[0, 0], [-2, 1, -3, -4, 5, 6, 7, 8])
    # q . k depends on the difference of positions alone
    q, k = _rand(1, 1, 8, seed=31), _rand(1, 1, 8, seed=32)
    f = [0.3, 0.02, 1.1, 0.7]
    dots = [float(np.sum(oracle.norm_rope(q, [p + 5], f, eps=None) *
                         oracle.norm_rope(k, [p], f, eps=None))) for p in (0, 17, 1000)]
    assert np.allclose(dots, dots[0])


def test_norm_weight_and_axes():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])  # mean square 25/4
    y = oracle.norm_rope(x, [0], [1.0], weight=[1, 2, 1, 1], eps=0.0)
    assert np.allclose(y[0, 0], [3 / 2.5, 8 / 2.5, 0, 0])
    x = _rand(3, 2, 8, seed=41)
    pos, axis, f = np.array([[1, 2, 3], [10, 20, 30]]), [1, 0], [0.5, 0.25]
    y = oracle.norm_rope(x, pos, f, eps=None, freq_axis=axis)
    for t in range(3):
        for i, (p, w) in enumerate([(pos[1, t], 0.5), (pos[0, t], 0.25)]):
            a, b = x[t, :, i], x[t, :, i + 2]
            assert np.allclose(y[t, :, i], a * np.cos(p * w) - b * np.sin(p * w))
            assert np.allclose(y[t, :, i + 2], a * np.sin(p * w) + b * np.cos(p * w))
