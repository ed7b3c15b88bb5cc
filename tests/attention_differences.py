"""Gradients of the softmax attention against differences of its forward, along directions in which a wrong gradient shows: the
gradients themselves (a wrong size or sign, or a share too many) and the oracle's (a share that is missing).

For q, k and v in turn the input moves by +h d and -h d, d the direction in units of its own root mean square, and the loss
sum(o dO) is summed in 64 bits from outputs in bf16. With `moved` the whole way between the two rounded inputs, the difference of the
losses is gradient . moved, up to
- roundings: an output carries its own, at most u |o|, and its weights', at most u w |v| each, of any sign and independent: the loss is
  off by a deviation of at most u / sqrt(3) |dO sqrt(o^2 + w^2 v^2)|, two losses by sqrt(2) of that; six of those are allowed;
- the third derivative: with scores that move by at most 1/8 each way it is below (1/4)^2 5 / 6 = 0.05 of the sum of the shares of the
  difference, and shares of both signs may leave half of that sum: 0.1 of the difference.
A gradient of half the size or the wrong sign is off by 0.5 and 2."""
import numpy as np
import torch

from oracle import attention as A


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float64)).bfloat16().double().numpy()


def noise(q, k, v, dO, cu, window, sinks):
    """deviation of the loss by the roundings of its outputs"""
    HQ, D = q.shape[1:]
    G, total = HQ // k.shape[1], 0.0
    for a, b in zip(cu[:-1], cu[1:]):
        seen = A.visible(np.arange(b - a), np.arange(b - a), window, sinks)
        for h in range(HQ):
            z = v[a:b, h // G]
            o, _, w = A.head(q[a:b, h], k[a:b, h // G], z, seen, D ** -0.5)
            total += (dO[a:b, h] ** 2 * (o ** 2 + w ** 2 @ z ** 2)).sum()
    return 2.0 ** -8 * (total / 3) ** 0.5


def moves(name, d, q, k, cu, window, sinks):
    """largest change of a score along d"""
    D, G, most = q.shape[2], q.shape[1] // k.shape[1], 0.0
    for a, b in zip(cu[:-1], cu[1:]):
        seen = A.visible(np.arange(b - a), np.arange(b - a), window, sinks)
        for h in range(q.shape[1] if name != "dv" and b > a else 0):
            x, y = (d[a:b, h], k[a:b, h // G]) if name == "dq" else (q[a:b, h], d[a:b, h // G])
            most = max(most, float(np.where(seen, np.abs(x @ y.T), 0).max()) * D ** -0.5)
    return most


def check(forward, grads, q, k, v, dO, cu, window=0, sinks=0):
    """forward(q, k, v) -> o; all arrays fp64 that bf16 holds; grads: dict dq, dk, dv. Returns the worst error over its bound."""
    worst = 0.0
    sigma = noise(q, k, v, dO, cu, window, sinks)
    exact = A.backward(q, k, v, cu, dO, window, sinks)
    for i, name in enumerate(("dq", "dk", "dv")):
        for along in (grads, exact):
            d = along[name] / np.sqrt((along[name] ** 2).mean())
            h = 1.0 if name == "dv" else 0.125 / moves(name, d, q, k, cu, window, sinks)
            ends = [[bf16(x + s * h * d) if j == i else x for j, x in enumerate((q, k, v))] for s in (1, -1)]
            loss = [float((forward(*x) * dO).sum()) for x in ends]
            want = float((grads[name] * (ends[0][i] - ends[1][i])).sum())
            bound = 6 * 2 ** 0.5 * sigma + 0.1 * abs(loss[0] - loss[1])
            print(name, "difference", loss[0] - loss[1], "gradient", want, "bound", bound, flush=True)
            worst = max(worst, abs(loss[0] - loss[1] - want) / bound)
    return worst
