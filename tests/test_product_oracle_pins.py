"""The 64-bit definitions of the expert products, pinned to values worked out by
hand and to differences of the forward formulas."""
import math

import numpy as np
import pytest

import oracle.product_oracle as po


def test_product_by_hand():
    x = np.array([[1.0, 2.0], [3.0, -1.0], [9.0, 9.0]])
    w = np.array([[[1.0, 0.0], [1.0, 1.0]], [[0.0, 2.0], [-1.0, 0.0]]])
    z, y = po.product(x, w, [0, 1, 2], bias=np.array([[10.0, 0.0], [0.0, 1.0]]), residual=np.ones((3, 2)))
    assert np.array_equal(z[:2], [[11, 3], [-2, -2]]) and np.array_equal(y[:2], z[:2] + 1) and np.isnan(y[2]).all()
    dx, dw, db, _ = po.product_backward(np.array([[1.0, 1.0], [2.0, 0.0], [7.0, 7.0]]), x, w, [0, 1, 2])
    assert np.array_equal(dx[:2], [[2, 1], [0, 4]]) and np.array_equal(db, [[1, 1], [2, 0]])
    assert np.array_equal(dw, [[[1, 2], [1, 2]], [[6, -2], [0, 0]]])


def test_activations_by_hand():
    one = np.array([1.0, 0.0, -1.0])
    assert np.allclose(po.act(one, "silu"), [1 / (1 + math.exp(-1)), 0, -1 / (1 + math.e)], rtol=1e-15)
    phi = 0.5 * math.erfc(-1 / math.sqrt(2))
    assert np.allclose(po.act(one, "gelu"), [phi, 0, -(1 - phi)], rtol=1e-15)
    assert po.slope(np.zeros(1), "silu")[0] == 0.5 and po.slope(np.zeros(1), "gelu")[0] == 0.5


def test_gelu_far_below_zero_by_hand():
    z = np.array([-10.0, -6.0])
    phi = np.array([7.619853024160527e-24, 9.865876450376946e-10])      # tables of the normal distribution function
    assert np.allclose(po.act(z, "gelu"), z * phi, rtol=1e-12, atol=0)
    bell = np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    assert np.allclose(po.slope(z, "gelu"), phi + z * bell, rtol=1e-12, atol=0)


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gradients_against_differences(name):
    rng = np.random.default_rng(5)
    S, H, I, E, off = 7, 6, 5, 3, [0, 4, 4, 6]
    x, dy = rng.standard_normal((S, H)), rng.standard_normal((S, H))
    wgu, wd = rng.standard_normal((E, 2 * I, H)), rng.standard_normal((E, H, I))
    z = po.ffn(x, wgu, wd, off, name)[0]
    got = po.ffn_backward(dy, x, wgu, wd, z, off, name)
    loss = lambda: float((po.ffn(x, wgu, wd, off, name)[2] * dy)[:6].sum())
    eps = 1e-5
    for a, g in [(x, got[0]), (wgu, got[1]), (wd, got[2])]:
        for at in rng.permutation(a.size)[:25]:
            i = np.unravel_index(at, a.shape)
            if a is x and i[0] >= 6:
                continue
            keep = a[i]
            a[i] = keep + eps
            up = loss()
            a[i] = keep - eps
            down = loss()
            a[i] = keep
            assert abs((up - down) / (2 * eps) - g[i]) < 1e-7 * (1 + abs(g[i]) + abs(up))
    b = rng.standard_normal((E, 2 * I))
    r = rng.standard_normal((S, 2 * I))
    pre = po.product(x, wgu, off, b, name)[0]
    dx, dw, db, _ = po.product_backward(r, x, wgu, off, name, pre)
    loss = lambda: float((po.product(x, wgu, off, b, name)[1] * r)[:6].sum())
    for a, g in [(x, dx), (wgu, dw), (b, db)]:
        for at in rng.permutation(a.size)[:20]:
            i = np.unravel_index(at, a.shape)
            if a is x and i[0] >= 6:
                continue
            keep = a[i]
            a[i] = keep + eps
            up = loss()
            a[i] = keep - eps
            down = loss()
            a[i] = keep
            assert abs((up - down) / (2 * eps) - g[i]) < 1e-7 * (1 + abs(g[i]) + abs(up))
    assert not got[1][1].any() and not dw[1].any() and not db[1].any()     # an expert without rows


def test_scales_by_hand():
    z = np.zeros((1, 2 * 136))
    z[0, 5], z[0, 130], z[0, 136 + 127] = -4.48, 0.0, 448
    s = po.scales(z)
    assert s.shape == (1, 4) and np.array_equal(s[0], [4.48 / 448, 2.0 ** -100, 1.0, 2.0 ** -100])
    wide = po.spread_scales(s, 136)
    assert wide.shape == z.shape and wide[0, 127] == s[0, 0] and wide[0, 128] == s[0, 1] and wide[0, 136 + 128] == s[0, 3]
