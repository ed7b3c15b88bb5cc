"""The fp64 oracles of rotary and the norm against hand-worked values and differences."""
import numpy as np

from oracle import layer as Y


def test_rotary_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    quarter = [np.pi / 2, np.pi]
    assert np.allclose(Y.rotary(x, [1], quarter, True), [[[-2, 1, -3, -4, 5]]])
    assert np.allclose(Y.rotary(x, [1], quarter, False), [[[-3, -2, 1, -4, 5]]])
    assert np.allclose(Y.rotary(x, [2], quarter, False, mscale=0.5), [[[-0.5, 1, -1.5, 2, 5]]])


def test_rotary_keeps_relative_positions_and_turns_back():
    r = np.random.default_rng(0)
    q, k, f = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8)), [1.0, 0.3, 0.05]
    for inter in (True, False):
        dots = [(Y.rotary(q, [p + 7], f, inter) * Y.rotary(k, [p], f, inter)).sum() for p in (0, 5, 100000)]
        assert np.allclose(dots, dots[0])
        assert np.allclose(Y.rotary(Y.rotary(q, [9], f, inter), [9], f, inter, back=True), q)
        d = r.normal(size=q.shape)  # the gradient is the transpose
        assert np.isclose((Y.rotary(q, [3], f, inter) * d).sum(), (q * Y.rotary(d, [3], f, inter, back=True)).sum())
    assert Y.positions([0, 2, 2, 5], [10, 20, 30]).tolist() == [10, 11, 30, 31, 32]


def test_norm_by_hand():
    y, rstd = Y.rmsnorm([[3.0, 4.0]], np.array([1.0, 2.0]), eps=0.0, unit=1.0)
    size = np.sqrt(12.5)
    assert np.allclose(rstd, 1 / size) and np.allclose(y, [[6 / size, 12 / size]])
    assert np.allclose(Y.scales(np.array([[1.0, -4.48, 2.0], [0, 0, 0]]), 0), [0.01, 2.0 ** -100 / 448])
    assert np.allclose(Y.scales(np.array([[1.0, -4.48, 2.0]]), 2), [[0.01, 2 / 448]])


def test_norm_gradients_are_differences():
    r = np.random.default_rng(1)
    s, w, dy, ds = r.normal(size=(3, 5)), r.normal(size=5), r.normal(size=(3, 5)), r.normal(size=(3, 5))
    dx, dw = Y.rmsnorm_backward(s, dy, w, 1e-3, 1.0, ds)
    loss = lambda s_, w_: (Y.rmsnorm(s_, w_, 1e-3, 1.0)[0] * dy).sum() + (s_ * ds).sum()  # noqa: E731
    a, b = r.normal(size=s.shape), r.normal(size=5)
    assert np.isclose((loss(s + 1e-5 * a, w) - loss(s - 1e-5 * a, w)) / 2e-5, (dx * a).sum(), rtol=1e-6)
    assert np.isclose((loss(s, w + 1e-5 * b) - loss(s, w - 1e-5 * b)) / 2e-5, (dw * b).sum(), rtol=1e-6)
