"""The 64-bit definitions of the operators around the layer, pinned on the CPU:
hand-worked values, and every gradient against central differences of its own
forward definition."""
import numpy as np
import pytest

import oracle.ops_oracle as oo


def test_rmsnorm_by_hand():
    r, y = oo.rmsnorm(np.array([[3.0, -1.0]]), np.array([2.0, 10.0]), 0.0, residual=np.array([[0.0, 5.0]]))
    assert r.tolist() == [[3.0, 4.0]]
    # sqrt((9 + 16) / 2) = 5 / sqrt(2)
    np.testing.assert_allclose(y, [[6 * np.sqrt(2) / 5, 8 * np.sqrt(2)]], rtol=1e-15)
    assert oo.e4m3_scales(np.array([[-448.0, 1.0, 0.0, 0.0]]), 2).tolist() == [[1.0, 2.0 ** -100]]
    assert oo.e4m3_scales(np.array([[-448.0, 1.0, 896.0]]), 0).tolist() == [[2.0]]


def test_sort_by_hand():
    offsets, inv, perm = oo.sort_slots(np.array([[2, 0], [-1, 2], [0, 3]]), 3)
    assert offsets.tolist() == [0, 2, 2, 4]          # expert 3 is outside [0, 3)
    assert perm.tolist() == [1, 4, 0, 3]
    assert inv.tolist() == [2, 0, -1, 3, 1, -1]


def differences(f, a, h=1e-6):
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        up, down = a.copy(), a.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


@pytest.mark.parametrize("T,H,eps", [(1, 8, 1e-5), (3, 5, 0.1)])
def test_rmsnorm_gradient_against_differences(T, H, eps):
    rng = np.random.default_rng(1)
    r, g, dy, dres = rng.normal(size=(T, H)), rng.normal(size=H), rng.normal(size=(T, H)), rng.normal(size=(T, H))
    dx, dg = oo.rmsnorm_backward(dy, r, g, eps, dres)
    # the loss reaches r by y and by the residual stream
    np.testing.assert_allclose(dx, differences(lambda a: np.sum(oo.rmsnorm(a, g, eps)[1] * dy) + np.sum(a * dres), r),
                               atol=1e-8)
    np.testing.assert_allclose(dg, differences(lambda a: np.sum(oo.rmsnorm(r, a, eps)[1] * dy), g), atol=1e-8)


def test_unpermute_gradient_against_differences():
    rng = np.random.default_rng(2)
    T, k, E, H = 4, 3, 5, 6
    ids = rng.integers(-1, E, size=(T, k))
    _, inv, perm = oo.sort_slots(ids, E)
    rows, w, dy = rng.normal(size=(T * k, H)), rng.normal(size=(T, k)), rng.normal(size=(T, H))
    drows, dw = oo.unpermute_backward(dy, rows, inv, w, T, k)
    loss = lambda a, b: np.sum(oo.unpermute(a, inv, b, T, k) * dy)
    np.testing.assert_allclose(drows, differences(lambda a: loss(a, w), rows), atol=1e-8)
    np.testing.assert_allclose(dw, differences(lambda b: loss(rows, b), w), atol=1e-8)
    # permute is linear: <xs, dxs> = <x, dx>
    x, dxs = rng.normal(size=(T, H)), rng.normal(size=(T * k, H))
    xs = np.zeros((T * k, H))
    xs[:len(perm)] = x[perm // k]
    dx = oo.unpermute(dxs, inv, None, T, k)
    np.testing.assert_allclose(np.sum(xs[:len(perm)] * dxs[:len(perm)]), np.sum(x * dx))


def test_router_gradient_against_differences():
    rng = np.random.default_rng(3)
    T, E, k, H = 5, 6, 3, 7
    x, wr, dw, add = rng.normal(size=(T, H)), rng.normal(size=(E, H)), rng.normal(size=(T, k)), rng.normal(size=(T, H))
    ids = np.argsort(-(x @ wr.T), axis=1)[:, :k]

    def weights(x, wr):
        l = np.take_along_axis(x @ wr.T, ids, axis=1)
        z = np.exp(l - l.max(axis=1, keepdims=True))
        return z / z.sum(axis=1, keepdims=True)

    dx, dwr = oo.router_backward(x, wr, ids, weights(x, wr), dw, add)
    np.testing.assert_allclose(dx, differences(lambda a: np.sum(weights(a, wr) * dw) + np.sum(a * add), x), atol=1e-8)
    np.testing.assert_allclose(dwr, differences(lambda a: np.sum(weights(x, a) * dw), wr), atol=1e-8)
    # a dropped slot takes no part
    ids2, w2 = np.concatenate([ids, -np.ones((T, 1), int)], axis=1), np.concatenate([weights(x, wr), np.ones((T, 1))], axis=1)
    dw2 = np.concatenate([dw, np.full((T, 1), 9.0)], axis=1)
    again = oo.router_backward(x, wr, ids2, w2, dw2, add)
    np.testing.assert_array_equal(again[0], dx)
    np.testing.assert_array_equal(again[1], dwr)


def test_router_gradient_of_slots_masked_after_the_router():
    """Slots that lose their expert after the softmax, the others keeping their weights: the gradient is that of the
    router's own ids with dw 0 in the masked slots, and not that of the masked ids, which forgets the masked slots'
    logits in the softmax (it is right where the kept weights are a softmax of their own)."""
    rng = np.random.default_rng(5)
    T, E, k, H = 6, 7, 3, 5
    x, wr, dw = rng.normal(size=(T, H)), rng.normal(size=(E, H)), rng.normal(size=(T, k))
    ids = np.argsort(-(x @ wr.T), axis=1)[:, :k]
    kept = rng.random((T, k)) < 0.6
    kept[0], kept[1] = False, True

    def weights(x, wr, among):
        l = np.where(among, np.take_along_axis(x @ wr.T, ids, axis=1), -np.inf)
        z = np.exp(l - np.take_along_axis(x @ wr.T, ids, axis=1).max(axis=1, keepdims=True))
        return z / np.maximum(z.sum(axis=1, keepdims=True), 1e-300)

    every = np.ones((T, k), bool)
    loss = lambda a, b: np.sum(np.where(kept, weights(a, b, every) * dw, 0.0))
    want = differences(lambda a: loss(a, wr), x), differences(lambda b: loss(x, b), wr)
    got = oo.router_backward(x, wr, ids, weights(x, wr, every), np.where(kept, dw, 0.0))
    for a, b in zip(got, want):
        np.testing.assert_allclose(a, b, atol=1e-8)
    masked = np.where(kept, ids, -1)
    short = oo.router_backward(x, wr, masked, weights(x, wr, every), dw)
    assert np.max(np.abs(short[0] - want[0])) > 1e-2

    # a softmax over the kept slots alone: the masked ids are the right ones
    loss = lambda a, b: np.sum(np.where(kept, weights(a, b, kept) * dw, 0.0))
    want = differences(lambda a: loss(a, wr), x), differences(lambda b: loss(x, b), wr)
    got = oo.router_backward(x, wr, masked, weights(x, wr, kept), dw)
    for a, b in zip(got, want):
        np.testing.assert_allclose(a, b, atol=1e-8)
