"""The fp64 oracle of the linear attention against hand-worked values, its closed form and differences."""
import numpy as np
import pytest

from oracle import linear as L


def _inputs(seed=0, lens=(3, 0, 5), H=2, HV=4, D=4):
    r = np.random.default_rng(seed)
    T = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    return dict(q=r.normal(size=(T, H, D)), k=r.normal(size=(T, H, D)), v=r.normal(size=(T, HV, D)),
                log_decay=-r.uniform(0.01, 1.0, HV), cu=cu, h0=r.normal(size=(len(lens), HV, D, D)))


def test_two_tokens_by_hand():
    one = np.ones((2, 1, 1))
    o, hT = L.forward(2 * one, 3 * one, np.array([5.0, 7.0]).reshape(2, 1, 1), [np.log(0.5)], [0, 2],
                      h0=np.array([[[[4.0]]]]), scale=1.0)
    # S_1 = 2 + 15 = 17, S_2 = 8.5 + 21 = 29.5
    assert np.allclose(o.ravel(), [34.0, 59.0]) and np.allclose(hT.ravel(), 29.5)


def test_closed_form():
    x = _inputs()
    o, hT = L.forward(**x)
    D, cu = 4, x["cu"]
    for n in range(3):
        for hv in range(4):
            h, g = hv // 2, x["log_decay"][hv]
            for t in range(cu[n], cu[n + 1]):
                S = np.exp(g * (t - cu[n] + 1)) * x["h0"][n, hv]
                for j in range(cu[n], t + 1):
                    S = S + np.exp(g * (t - j)) * np.outer(x["v"][j, hv], x["k"][j, h])
                assert np.allclose(o[t, hv], D ** -0.5 * S @ x["q"][t, h])
    assert np.array_equal(hT[1], x["h0"][1])  # no tokens: the state passes through


def test_gradients_are_differences():
    x = _inputs(1)
    r = np.random.default_rng(2)
    dO, dhT = r.normal(size=x["v"].shape), r.normal(size=x["h0"].shape)
    g = L.backward(**x, dO=dO, dhT=dhT)

    def loss(y):
        o, hT = L.forward(**y)
        return (o * dO).sum() + (hT * dhT).sum()

    for name in ("q", "k", "v", "h0"):
        d = r.normal(size=x[name].shape)
        up, down = (loss(dict(x, **{name: x[name] + s * 1e-5 * d})) for s in (1, -1))
        assert np.isclose((up - down) / 2e-5, (g["d" + name] * d).sum(), rtol=1e-6), name


@pytest.mark.parametrize("decay", [-np.inf, 0.0, -0.3])
def test_steps_are_the_forward(decay):
    x = _inputs(3, lens=(6,), H=1, HV=1)
    x["log_decay"] = np.array([decay])
    o, hT = L.forward(**x)
    pool = np.zeros((3, 1, 4, 4))
    pool[2] = x["h0"][0]
    for t in range(6):
        ot, pool = L.step(x["q"][t:t + 1], x["k"][t:t + 1], x["v"][t:t + 1], x["log_decay"], pool, [2])
        assert np.allclose(ot[0], o[t])
    assert np.allclose(pool[2], hT[0]) and not pool[:2].any()
