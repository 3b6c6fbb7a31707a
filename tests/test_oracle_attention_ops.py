"""The fp64 definitions of the attention layers' operators pinned: against loops written out pair by pair, and their
gradients against central differences."""
import math

import numpy as np
import pytest

from oracle import attention_ops as A


def brute(q, k, v, window, sinks, scale):
    Lq, Hq, d = q.shape
    Lk, Hk, _ = k.shape
    out, lse = np.zeros((Lq, Hq, d)), np.full((Hq, Lq), -np.inf)
    for i in range(Lq):
        p = Lk - Lq + i
        for h in range(Hq):
            keys = [j for j in range(Lk) if j <= p and (p - j < window or j < sinks)]
            if not keys:
                continue
            s = [scale * sum(q[i, h, c] * k[j, h // (Hq // Hk), c] for c in range(d)) for j in keys]
            top = max(s)
            w = [math.exp(x - top) for x in s]
            lse[h, i] = top + math.log(sum(w))
            for j, x in zip(keys, w):
                out[i, h] += x / sum(w) * v[j, h // (Hq // Hk)]
    return out, lse


@pytest.mark.parametrize("Lq,Lk,window,sinks", [(1, 1, 1, 0), (7, 7, 3, 0), (7, 7, 3, 2), (9, 9, 100, 0), (3, 8, 4, 1), (8, 3, 2, 1), (5, 5, 1, 9)])
def test_window_attention_is_the_sum_over_pairs(Lq, Lk, window, sinks):
    g = np.random.default_rng(Lq * 10 + Lk)
    q, k, v = g.normal(size=(Lq, 4, 3)), g.normal(size=(Lk, 2, 3)), g.normal(size=(Lk, 2, 3))
    r = A.window_attention(q, k, v, window, sinks, 0.7, "fp32")
    out, lse = brute(q, k, v, window, sinks, 0.7)
    assert np.allclose(r["out"], out, atol=1e-13) and np.allclose(r["lse"], lse, atol=1e-13)


def differences(f, x, dy, h=1e-6):
    """Central differences of sum(dy * f(x))."""
    out = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        out[i] = ((f(a) - f(b)) * dy).sum() / (2 * h)
    return out


@pytest.mark.parametrize("Lq,Lk,window,sinks", [(6, 6, 3, 1), (3, 6, 4, 0), (6, 4, 2, 1)])
def test_window_attention_gradients_are_the_differences(Lq, Lk, window, sinks):
    g = np.random.default_rng(5)
    q, k, v, dy = g.normal(size=(Lq, 2, 3)), g.normal(size=(Lk, 1, 3)), g.normal(size=(Lk, 1, 3)), g.normal(size=(Lq, 2, 3))
    r = A.window_attention(q, k, v, window, sinks, 0.6, "fp32", dy)
    f = lambda q, k, v: A.window_attention(q, k, v, window, sinks, 0.6, "fp32")["out"]  # noqa: E731
    assert np.allclose(r["dq"], differences(lambda x: f(x, k, v), q, dy), atol=1e-8)
    assert np.allclose(r["dk"], differences(lambda x: f(q, x, v), k, dy), atol=1e-8)
    assert np.allclose(r["dv"], differences(lambda x: f(q, k, x), v, dy), atol=1e-8)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(6, 6), (8, 4)])
def test_norm_rotary_and_its_gradients(d, rot, layout):
    g = np.random.default_rng(d)
    x, w, dy = g.normal(size=(1, 3, 2, d)), 1 + 0.1 * g.normal(size=d), g.normal(size=(1, 3, 2, d))
    pos, f = np.array([[0, 5, 77]]), A.frequencies(rot, 100.0)
    y = lambda x, w: A.norm_rotary(x, w, pos, f, rot, layout, 1e-3, 1.3)["y"]  # noqa: E731
    # a head by hand: the norm leaves mean square 1 (less eps), the turn keeps a pair's length
    z = x[0, 1, 0] / math.sqrt((x[0, 1, 0] ** 2).mean() + 1e-3) * w
    i, j = (0, rot // 2) if layout == "half" else (0, 1)
    a = 5 * f[0]
    assert np.allclose(y(x, w)[0, 1, 0, [i, j]], 1.3 * np.array([z[i] * math.cos(a) - z[j] * math.sin(a), z[j] * math.cos(a) + z[i] * math.sin(a)]))
    assert np.allclose(y(x, w)[0, 1, 0, rot:], z[rot:])
    r = A.norm_rotary(x, w, pos, f, rot, layout, 1e-3, 1.3, dy)
    assert np.allclose(r["dx"], differences(lambda t: y(t, w), x, dy), atol=1e-7)
    assert np.allclose(r["dw"], differences(lambda t: y(x, t), w, dy), atol=1e-7)


def test_cache_write_keeps_what_the_mask_can_show():
    """After a write of any split, every visible position of the next query is in its slot."""
    g = np.random.default_rng(2)
    for sinks, window, slack, sizes in ((2, 3, 0, [1, 1, 4, 9]), (0, 4, 2, [5, 5]), (3, 2, 1, [20]), (4, 1, 0, [2, 1, 1, 3])):
        x = g.normal(size=(sum(sizes), 1, 2))
        cache, t = np.zeros((1, 1, sinks + window + slack, 2)), 0
        for n in sizes:
            cache = A.cache_write(cache, [x[t:t + n]], [t], sinks)
            t += n
            for p in range(t):
                if t - 1 - p < window or p < sinks:
                    assert np.array_equal(cache[0, 0, A.slot_of(p, sinks, cache.shape[2])], x[p, 0]), (sinks, window, p)
