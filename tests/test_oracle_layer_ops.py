"""Pins of the fp64 definitions in oracle/layer_ops.py: closed forms, brute force and finite
differences (CPU)."""
import numpy as np
import pytest

from oracle import layer_ops as O


def rec_inputs(rng, ntok, D):
    return [rng.standard_normal((ntok, D)) for _ in range(3)] + [rng.uniform(-2, 1, D), rng.uniform(-4, 1, D)]


def test_recurrence_closed_form():
    # constant gates: h_t = u (1 - alpha^(t+1)) / (1 - alpha) + alpha^(t+1) h0
    T, D = 9, 2
    x, a, b = np.full((T, D), 0.7), np.full((T, D), 0.3), np.full((T, D), -0.2)
    A_log, bias, h0 = np.array([0.1, -1.0]), np.array([-1.0, 0.5]), np.array([[0.4, -2.0]])
    alpha = np.exp(-np.exp(A_log) * np.log1p(np.exp(0.3 + bias)))
    u = np.sqrt(1 - alpha ** 2) / (1 + np.exp(0.2)) * 0.7
    r = O.recurrence(x, a, b, A_log, bias, [0, T], h0)
    k = np.arange(1, T + 1)[:, None]
    assert np.allclose(r["out"], u * (1 - alpha ** k) / (1 - alpha) + alpha ** k * h0, rtol=1e-12)
    assert np.array_equal(r["final"][0], r["out"][-1])


def test_recurrence_empty_sequences_keep_their_state():
    rng = np.random.default_rng(0)
    x, a, b, A, bias = rec_inputs(rng, 5, 3)
    h0 = rng.standard_normal((4, 3))
    r = O.recurrence(x, a, b, A, bias, [0, 0, 3, 3, 5], h0)
    assert np.array_equal(r["final"][0], h0[0]) and np.array_equal(r["final"][2], h0[2])
    alone = O.recurrence(x[3:], a[3:], b[3:], A, bias, [0, 2], h0[3:])
    assert np.array_equal(r["out"][3:], alone["out"])


def test_recurrence_gradients_against_differences():
    rng = np.random.default_rng(1)
    starts, D = [0, 4, 4, 9], 3
    args = rec_inputs(rng, 9, D)
    h0 = rng.standard_normal((3, D))
    dout, dfinal = rng.standard_normal((9, D)), rng.standard_normal((3, D))

    def loss(v):
        r = O.recurrence(*v[:5], starts, v[5])
        return (r["out"] * dout).sum() + (r["final"] * dfinal).sum()

    v = args + [h0]
    g = O.recurrence(*args, starts, h0, dout, dfinal)
    for i, name in enumerate(("dx", "da", "db", "dA_log", "ddt_bias", "dstate")):
        num = np.zeros_like(v[i])
        for j in np.ndindex(v[i].shape):
            w = [u.copy() for u in v]
            w[i][j] += 1e-5
            hi = loss(w)
            w[i][j] -= 2e-5
            num[j] = (hi - loss(w)) / 2e-5
        assert np.allclose(g[name], num, rtol=1e-6, atol=1e-8), name


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_pins(layout):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((7, 2, 10))
    f = O.frequencies(6)
    pos = np.array([0, 1, 2, 5, 1000, -3, 7])
    y = O.rotary(x, pos, f, 6, layout)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose(O.rotary(y, pos, f, 6, layout, inverse=True), x, atol=1e-12)
    # scores depend on distances alone
    k = rng.standard_normal((1, 2, 10))
    s = [(O.rotary(x[:1], [p], f, 6, layout) * O.rotary(k, [p - 4], f, 6, layout)).sum() for p in (4, 11, 900)]
    assert np.allclose(s, s[0], atol=1e-10)


def test_rotary_scalings():
    f = O.frequencies(64, 500000.0)
    assert np.allclose(O.frequencies(64, 500000.0, "linear", 4.0), f / 4)
    g = O.frequencies(64, 500000.0, "by_parts", 8.0, 1.0, 4.0, 8192)
    turns = 8192 * f / (2 * np.pi)
    assert np.array_equal(g[turns >= 4], f[turns >= 4]) and np.allclose(g[turns <= 1], f[turns <= 1] / 8)
    assert np.all((g <= f) & (g >= f / 8 * (1 - 1e-15)))


@pytest.mark.parametrize("act", ["none", "silu"])
def test_group_norm_gradients_against_differences(act):
    rng = np.random.default_rng(3)
    x, w, b = rng.standard_normal((2, 3, 8)), rng.standard_normal(8), rng.standard_normal(8)
    dy = rng.standard_normal(x.shape)
    loss = lambda v: (O.group_norm(v[0], v[1], v[2], 2, act, 1e-3)["out"] * dy).sum()  # noqa: E731
    v = [x, w, b]
    g = O.group_norm(x, w, b, 2, act, 1e-3, dy)
    for i, name in enumerate(("dx", "dweight", "dbias")):
        num = np.zeros_like(v[i])
        for j in np.ndindex(v[i].shape):
            u = [t.copy() for t in v]
            u[i][j] += 1e-5
            hi = loss(u)
            u[i][j] -= 2e-5
            num[j] = (hi - loss(u)) / 2e-5
        assert np.allclose(g[name], num, rtol=1e-6, atol=1e-8), name


def test_group_norm_closed_form():
    x = np.array([[[1.0, 3.0, -2.0, 2.0]]])
    r = O.group_norm(x, None, None, 2, "none", 0.0)
    assert np.allclose(r["out"], [[[-1, 1, -1, 1]]]) and np.allclose(r["mean"], [[2, 0]]) and np.allclose(r["rstd"], [[1, 0.5]])
