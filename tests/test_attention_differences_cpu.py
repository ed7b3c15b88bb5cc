"""The check of gradients against differences on the CPU: it passes the oracle's gradients, and no gradients with a mistake."""
import numpy as np
import pytest

from oracle import attention as A
from tests.attention_differences import bf16, check

CASES = [  # lens, HQ, HK, D, window, sinks
    ([25, 15], 4, 2, 64, 0, 0), ([40], 4, 1, 128, 9, 0), ([30, 10], 2, 1, 256, 0, 0), ([60], 3, 1, 64, 12, 3), ([150], 2, 2, 64, 20, 30),
]


def make(lens, HQ, HK, D, seed=0):
    r = np.random.default_rng(seed + D)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    return [bf16(r.standard_normal((cu[-1], h, D))) for h in (HQ, HK, HK, HQ)] + [cu]


@pytest.mark.parametrize("lens, HQ, HK, D, window, sinks", CASES)
def test_mistakes_show(lens, HQ, HK, D, window, sinks):
    q, k, v, dO, cu = make(lens, HQ, HK, D)
    forward = lambda *x: bf16(A.forward(*x, cu, window, sinks)[0])  # noqa: E731
    grads = A.backward(q, k, v, cu, dO, window, sinks)
    assert check(forward, grads, q, k, v, dO, cu, window, sinks) <= 1
    wrong = [dict(grads, **{n: grads[n] * f}) for n in grads for f in (0.5, -1, 1.5)]
    wrong.append(dict(grads, **{n: np.roll(grads[n], 1, 0) for n in ("dk",)}))
    if HQ > HK:  # one query head of a key head left out
        few = dO * (np.arange(HQ) % (HQ // HK) > 0)[:, None]
        wrong.append(dict(A.backward(q, k, v, cu, few, window, sinks), dq=grads["dq"]))
    if window:
        wrong.append(A.backward(q, k, v, cu, dO))
    if sinks:
        wrong.append(A.backward(q, k, v, cu, dO, window))
    for g in wrong:
        assert check(forward, g, q, k, v, dO, cu, window, sinks) > 1
