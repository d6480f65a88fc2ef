"""Pins of oracle/block.py on the CPU: finite differences, carries, closed forms."""
import numpy as np
import pytest

from oracle import block


def rng(seed):
    return np.random.default_rng(seed)


def slope(f, x, d, step=1e-6):
    return (f(x + step * d) - f(x - step * d)) / (2 * step)


@pytest.mark.parametrize("weight,skip", [(True, True), (False, False)])
def test_norm_gradients_against_differences(weight, skip):
    r = rng(1)
    h, dy, dh, w = r.standard_normal((5, 24)), r.standard_normal((5, 24)), r.standard_normal((5, 24)), 1 + 0.3 * r.standard_normal(24)
    w = w if weight else None
    dx, dw = block.rms_norm_bwd(h, w, dy, dh if skip else None, 1e-6)
    loss = lambda a, b: (block.rms_norm(a, b, 1e-6) * dy).sum() + ((a * dh).sum() if skip else 0.0)
    d = r.standard_normal(h.shape)
    assert abs(slope(lambda a: loss(a, w), h, d) - (dx * d).sum()) < 1e-6
    v = r.standard_normal(24)
    assert abs(slope(lambda b: loss(h, b), np.ones(24) if w is None else w, v) - (dw * v).sum()) < 1e-6


def test_norm_of_a_constant_row():
    assert np.allclose(block.rms_norm(np.full((1, 8), -3.0), None, 0.0), -1.0)


def test_blocks_and_product():
    r = rng(2)
    n = r.standard_normal((3, 300))
    assert np.array_equal(block.block_max(n)[1], [np.abs(n[1, :128]).max(), np.abs(n[1, 128:256]).max(), np.abs(n[1, 256:]).max()])
    a, w, sa, sw = r.standard_normal((3, 300)), r.standard_normal((140, 300)), r.random((3, 3)), r.random((2, 3))
    c = block.product(a, sa, w, sw)
    one = sum(sa[2, k // 128] * sw[1, k // 128] * a[2, k] * w[130, k] for k in range(300))
    assert c.shape == (3, 140) and abs(c[2, 130] - one) < 1e-12


@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("gate,igate", [(True, True), (False, False), (True, False)])
def test_recurrence_gradients_against_differences(unit, gate, igate):
    r = rng(3)
    T, D = 9, 4
    v = dict(x=r.standard_normal((T, D)), r=r.standard_normal((T, D)) if gate else -r.uniform(0.01, 1, (T, D)),
             i=r.standard_normal((T, D)) if igate else None, c=r.uniform(0.1, 1, D) if gate else None, h0=r.standard_normal(D))
    dy, dht = r.standard_normal((T, D)), r.standard_normal(D)

    def loss(**kw):
        y, ht = block.lru_fwd(unit=unit, **{**v, **kw})
        return (y * dy).sum() + (ht * dht).sum()
    got = dict(zip(("x", "r", "i", "c", "h0"), block.lru_bwd(dy=dy, dht=dht, unit=unit, **v)))
    for n, g in got.items():
        assert (g is None) == (v[n] is None)
        if g is not None:
            d = r.standard_normal(g.shape)
            assert abs(slope(lambda a: loss(**{n: a}), v[n], d) - (g * d).sum()) < 1e-6, n


def test_recurrence_carries_and_closed_form():
    r = rng(4)
    x, g, h0 = r.standard_normal((12, 3)), -r.uniform(0, 2, (12, 3)), r.standard_normal(3)
    y, ht = block.lru_fwd(x, g, None, None, h0, False)
    y1, h1 = block.lru_fwd(x[:5], g[:5], None, None, h0, False)
    y2, h2 = block.lru_fwd(x[5:], g[5:], None, None, h1, False)
    assert np.allclose(np.concatenate([y1, y2]), y, atol=1e-14) and np.allclose(h2, ht, atol=1e-14)
    s = g.cumsum(0)
    t = 8
    want = np.exp(s[t]) * h0 + sum(np.exp(s[t] - s[k]) * x[k] for k in range(t + 1))
    assert np.allclose(y[t], want, atol=1e-12)
    # with unit inputs of variance one the state keeps that variance
    _, a, m, _ = block.lru_gates(x, g, None, None, True)
    assert np.allclose(a * a + m * m, 1.0)


def test_reset_and_open_gate():
    x = np.array([[1.0], [2.0], [4.0]])
    g = np.array([[0.0], [-np.inf], [0.0]])
    y, _ = block.lru_fwd(x, g, None, None, np.array([10.0]), False)
    assert np.array_equal(y[:, 0], [11.0, 2.0, 6.0])
    y, _ = block.lru_fwd(x, g, None, None, np.array([10.0]), True)
    assert np.array_equal(y[:, 0], [10.0, 2.0, 2.0])
