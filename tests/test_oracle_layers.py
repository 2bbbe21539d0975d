"""Pins of the fp64 oracle of the convolution, the scan and the verification."""

import numpy as np

import oracle


def _rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def test_conv_of_one_impulse_is_the_taps_backwards():
    x = np.zeros((6, 2))
    x[1] = [1.0, 2.0]
    w = np.array([[1.0, 2.0, 3.0], [4.0, 5.0, 6.0]])
    y, last = oracle.causal_conv(x, w, silu=False)
    assert np.array_equal(y[:, 0], [0, 3, 2, 1, 0, 0]) and np.array_equal(y[:, 1], [0, 12, 10, 8, 0, 0])
    assert np.array_equal(last[0], x[4:])
    y, _ = oracle.causal_conv(np.zeros((1, 2)), w, bias=[0.0, 2.0])
    assert np.allclose(y, [[0.0, 2.0 / (1 + np.exp(-2.0))]])


def test_conv_pieces_continue_and_short_sequences_keep_old_inputs():
    x, w = _rand(9, 3, seed=1), _rand(3, 4, seed=2)
    y, last = oracle.causal_conv(x, w)
    y1, s = oracle.causal_conv(x[:1], w)
    y2, s = oracle.causal_conv(x[1:3], w, state=s)
    y3, s = oracle.causal_conv(x[3:], w, state=s)
    assert np.allclose(np.concatenate([y1, y2, y3]), y) and np.array_equal(s, last)
    both, kept = oracle.causal_conv(x, w, cu_seqlens=[0, 2, 2, 9], n_advance=[1, 0, 7],
                                    state=_rand(3, 3, 3, seed=3))
    one, _ = oracle.causal_conv(x[2:], w, state=_rand(3, 3, 3, seed=3)[2:])
    assert np.allclose(both[2:], one) and np.array_equal(kept[0][2], x[0])
    assert np.array_equal(kept[1], _rand(3, 3, 3, seed=3)[1]) and np.array_equal(kept[2], x[6:])


def test_scan_with_constant_steps_is_a_weighted_sum():
    T, ch, S = 7, 4, 3
    x, B, C = _rand(T, ch, seed=1), _rand(T, 2, S, seed=2), _rand(T, 2, S, seed=3)
    A = -np.abs(_rand(ch, S, seed=4))
    y, hT = oracle.selective_scan(x, np.full((T, ch), 0.5), A, B, C, softplus=False)
    lag = np.arange(T)[:, None] - np.arange(T)[None, :]
    for c in range(ch):
        w = np.where(lag[..., None] >= 0, np.exp(0.5 * A[c] * np.maximum(lag, 0)[..., None]), 0.0)
        ref = np.einsum("ts,tjs,js,j->t", C[:, c // 2], w, B[:, c // 2], 0.5 * x[:, c])
        assert np.allclose(y[:, c], ref)
        assert np.allclose(hT[0, c], np.einsum("js,js,j->s", w[-1], B[:, c // 2], 0.5 * x[:, c]))


def test_scan_steps_skip_gate_and_partial_advance():
    x, dt, z = (_rand(6, 2, seed=s) for s in (1, 2, 3))
    B, C, A = _rand(6, 1, 2, seed=4), _rand(6, 1, 2, seed=5), -np.ones((2, 2))
    h0 = _rand(2, 2, 2, seed=6)
    y, hT = oracle.selective_scan(x, dt, A, B, C, h0, [0, 2, 6], [1.0, -1.0], z, [0.1, 0.2],
                                  n_advance=[0, 3])
    _, h3 = oracle.selective_scan(x[2:5], dt[2:5], A, B[2:5], C[2:5], h0[1:], dt_bias=[0.1, 0.2])
    assert np.allclose(hT[0], h0[0]) and np.allclose(hT[1], h3[0])
    plain, _ = oracle.selective_scan(x, dt, A, B, C, h0, [0, 2, 6], dt_bias=[0.1, 0.2])
    assert np.allclose(y, (plain + x * [1.0, -1.0]) * z / (1 + np.exp(-z)))
    y, _ = oracle.selective_scan(x, np.full((6, 2), -800.0), A, B, C, h0, [0, 2, 6])
    assert np.allclose(y[0], (C[0, 0] * h0[0]).sum(axis=1))  # steps of 0: the state stays


def test_verify_accepts_by_the_ratio_and_draws_from_what_is_left():
    p = np.array([[[0.5, 0.25, 0.25], [0.125, 0.125, 0.75]]])
    q = np.array([[[0.25, 0.5, 0.25]]])
    f = lambda d, u, s: oracle.verify_draft([[d]], q, p, [[u]], [s])  # noqa: E731
    t, a = f(1, 0.4, 0.0)                       # 0.4 x 0.5 < 0.25
    assert t.tolist() == [[1, 0]] and a.tolist() == [2]
    t, a = f(1, 0.5, 0.99)                      # equal is not below: only token 0 is left
    assert t.tolist() == [[0, -1]] and a.tolist() == [1]
    assert f(0, 0.999, 0.3)[0].tolist() == [[0, 2]]
    assert f(0, 0.999, 0.125)[0].tolist() == [[0, 1]]  # a border belongs to the next token
    assert f(-1, 0.0, 0.5)[0].tolist() == [[1, -1]]    # no draft: from p
    t, a = oracle.verify_draft([[0]], p[:, :1], p, [[1.0 - 2.0 ** -24]], [0.6])
    assert t.tolist() == [[0, 2]] and a.tolist() == [2]


def test_verified_tokens_follow_the_target():
    rng = np.random.default_rng(5)
    p, q = np.array([0.6, 0.1, 0.3]), np.array([0.2, 0.7, 0.1])
    n = 4000
    draft = rng.choice(3, size=(n, 1), p=q)
    t, _ = oracle.verify_draft(draft, np.broadcast_to(q, (n, 1, 3)), np.broadcast_to(p, (n, 2, 3)),
                               rng.random((n, 1)), rng.random(n))
    share = np.bincount(t[:, 0], minlength=3) / n
    # five standard deviations of a share over n draws
    assert np.all(np.abs(share - p) < 5 * np.sqrt(p * (1 - p) / n))
