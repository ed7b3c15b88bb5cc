"""Pins of the attention oracle: cases worked out by hand, laws, central differences."""
import math

import numpy as np
import pytest

from oracle import attention as A


def rng_case(lens, HQ, HK, D, seed=0):
    r = np.random.default_rng(seed)
    T = sum(lens)
    return (r.standard_normal((T, HQ, D)), r.standard_normal((T, HK, D)), r.standard_normal((T, HK, D)),
            np.concatenate([[0], np.cumsum(lens)]).tolist(), r)


def test_by_hand():
    q, k = np.ones((3, 1, 1)), np.array([0.0, math.log(2), math.log(3)]).reshape(3, 1, 1)
    v = np.array([1.0, 4.0, 10.0]).reshape(3, 1, 1)
    o, lse = A.forward(q, k, v, [0, 3], scale=1.0)
    assert np.allclose(o.ravel(), [1.0, 9 / 3, 39 / 6]) and np.allclose(np.exp(lse.ravel()), [1, 3, 6])
    o, _ = A.forward(q, k, v, [0, 3], window=1, scale=1.0)
    assert np.allclose(o.ravel(), [1, 4, 10])
    o, _ = A.forward(q, k, v, [0, 3], window=1, sinks=1, scale=1.0)
    assert np.allclose(o.ravel(), [1, 3, 31 / 4])


def test_visible():
    see = A.visible([0, 4, 9], range(10), 3, 2)
    assert [np.nonzero(x)[0].tolist() for x in see] == [[0], [0, 1, 2, 3, 4], [0, 1, 7, 8, 9]]
    assert A.visible([9], range(10), 0, 2).all() and not A.visible([-1], range(10), 0, 0).any()


def test_packs_groups_and_growing_windows():
    q, k, v, cu, _ = rng_case([5, 0, 9, 1], 4, 2, 8)
    o, lse = A.forward(q, k, v, cu, window=3, sinks=1)
    for a, b in zip(cu[:-1], cu[1:]):
        for h in range(4):
            one = A.forward(q[a:b, h:h + 1], k[a:b, h // 2:h // 2 + 1], v[a:b, h // 2:h // 2 + 1], [0, b - a], 3, 1)
            assert np.array_equal(o[a:b, h:h + 1], one[0]) and np.array_equal(lse[a:b, h:h + 1], one[1])
    assert np.array_equal(A.forward(q, k, v, cu)[0], A.forward(q, k, v, cu, window=9)[0])
    # equal scores: means of the values that are seen
    o, lse = A.forward(0 * q, k, v, cu, window=2)
    assert np.allclose(o[3, 0], v[2:4, 0].mean(0)) and np.allclose(np.exp(lse[3]), 2)


@pytest.mark.parametrize("window, sinks", [(0, 0), (3, 0), (2, 2)])
def test_gradients_against_differences(window, sinks):
    q, k, v, cu, r = rng_case([6, 1, 4], 4, 2, 3, seed=window)
    dO = r.standard_normal(q.shape)
    g = A.backward(q, k, v, cu, dO, window, sinks)
    loss = lambda: (A.forward(q, k, v, cu, window, sinks)[0] * dO).sum()  # noqa: E731
    for x, d in ((q, g["dq"]), (k, g["dk"]), (v, g["dv"])):
        for i in np.ndindex(x.shape):
            keep, h = x[i], 1e-5
            x[i] = keep + h
            up = loss()
            x[i] = keep - h
            down = loss()
            x[i] = keep
            assert abs((up - down) / (2 * h) - d[i]) < 1e-8


def test_paged_is_the_forward_and_steps_are_its_rows():
    lens, size = [7, 12, 3], 4
    q, k, v, cu, r = rng_case(lens, 4, 2, 8, seed=3)
    want, want_lse = A.forward(q, k, v, cu, 5, 1)
    table = r.permutation(np.arange(1, 10)).reshape(3, 3)
    kc, vc = (r.standard_normal((10, size, 2, 8)) for _ in range(2))
    first = [3, 4, 0]  # tokens of the first call; then the rest, the last one by a step
    starts, lasts = np.array(cu[:-1]), np.array(cu[1:])
    for a, b in ((np.zeros(3, int), np.array(first)), (np.array(first), np.array(lens) - 1)):
        rows = np.concatenate([np.arange(s + x, s + y) for s, x, y in zip(starts, a, b)])
        c = np.concatenate([[0], np.cumsum(b - a)]).tolist()
        _, kc, vc = A.append(k[rows], v[rows], kc, vc, table, a, c)
        o, lse = A.forward_paged(q[rows], kc, vc, table, c, a, 5, 1)
        assert np.allclose(o, want[rows], atol=1e-12) and np.allclose(lse, want_lse[rows])
    rows = lasts - 1
    _, kc, vc = A.append(k[rows], v[rows], kc, vc, table, np.array(lens) - 1, [0, 1, 2, 3])
    o, _ = A.step(q[rows], kc, vc, table, np.array(lens) - 1, 5, 1)
    assert np.allclose(o, want[rows], atol=1e-12)
    # without its pages a sequence's earlier tokens are not seen
    table[1, 0] = 0
    o, _ = A.step(q[rows], kc, vc, table, np.array(lens) - 1)
    alone, _, _ = A.head(q[rows[1], :1], k[starts[1] + 4:lasts[1], 0], v[starts[1] + 4:lasts[1], 0], np.ones((1, 8), bool), 8 ** -0.5)
    assert np.allclose(o[1, :1], alone)
    o, lse = A.step(q[rows], kc, vc, table, np.array([-1, 2, -5]))
    assert not o.any() and np.isneginf(lse).all()


def test_append_turns_by_the_place_in_the_cache():
    q, k, v, cu, r = rng_case([2, 3], 2, 1, 4, seed=5)
    f = np.array([1.0, 0.1])
    kc = np.zeros((4, 2, 1, 4))
    qt, kc, vc = A.append(k, v, kc, kc, np.array([[1, 9], [3, 2]]), [1, -1], cu, q, f)
    z = lambda x: x[..., :2] + 1j * x[..., 2:]  # noqa: E731
    turn = lambda x, p: z(x) * np.exp(1j * p * f)  # noqa: E731
    assert np.allclose(z(kc[1, 1]), turn(k[0], 1)) and np.array_equal(vc[1, 1], v[0])  # the second's page is none
    assert np.allclose(z(kc[3, 0]), turn(k[3], 0)) and np.allclose(z(kc[3, 1]), turn(k[4], 1))
    assert not kc[0].any() and not kc[2].any() and not kc[1, 0].any()
    assert np.allclose(z(qt[1]), turn(q[1], 2)) and np.allclose(z(qt[2]), turn(q[2], -1))
