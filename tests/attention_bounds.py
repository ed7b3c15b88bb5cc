"""How far the attention kernels' outputs may be from 64 bits, element by element, from the roundings that they make.

u is half a step of the tensors' type. Scores are sums of D exact products in fp32, at most D 2^-24 of the sum of their
magnitudes off; a weight's relative error e is twice that of the largest score (its own and the sum's or lse's) and 2^-18 for
exponentials, sums and quotients. Weights and the scores' gradients are rounded once to the type where they are multiplied, an
output once more; fp16 has steps of 2^-24 at its least, so half of that is added for each of them. A weight below fp32's least
normal number may be zero: 2^-126 is added to each, and to a score's gradient that times what the weight meets."""
import numpy as np

from oracle import attention as A

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
LEAST = {"bf16": 0.0, "fp16": 2.0 ** -25}
ZERO = 2.0 ** -126


def score_error(q, k, seen, scale):
    """largest error of a score of one head"""
    if not seen.any():
        return 0.0
    k = np.where(seen.any(0)[:, None], k, 0.0)
    return q.shape[1] * 2.0 ** -24 * scale * float(np.where(seen, np.abs(q) @ np.abs(k).T, 0).max())


def head_bounds(q, k, v, seen, scale, dtype, dO=None):
    """Bounds of o, lse and, with dO, of (dq, dk, dv) of one head's share, before what these round to at the end."""
    u, least = U[dtype], LEAST[dtype]
    some = seen.any(0)[:, None]
    k, v = np.where(some, k, 0.0), np.where(some, v, 0.0)
    o, lse, w = A.head(q, k, v, seen, scale)
    err = score_error(q, k, seen, scale)
    e = 2 * err + 2.0 ** -18
    bo = (u + e) * (w @ np.abs(v)) + (least + ZERO) * (seen @ np.abs(v)) + u * np.abs(o) + least
    blse = err + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
    if dO is None:
        return bo, blse
    D = q.shape[1]
    dp = np.abs(dO) @ np.abs(v).T
    ddelta = (np.abs(dO) * bo).sum(1, keepdims=True) + D * 2.0 ** -24 * (np.abs(dO) * np.abs(o)).sum(1, keepdims=True)
    ds = scale * w * (dO @ v.T - (dO * o).sum(1, keepdims=True))
    bds = scale * w * (ddelta + D * 2.0 ** -24 * dp) * (1 + u) + (u + e) * np.abs(ds) + (least + ZERO * scale * (dp + np.abs(ddelta) + (np.abs(dO) * np.abs(o)).sum(1, keepdims=True))) * seen
    bw = (u + e) * w + (least + ZERO) * seen
    sums = 2.0 ** -20  # long sums in fp32
    bq = bds @ np.abs(k) + sums * (np.abs(ds) @ np.abs(k))
    bk = bds.T @ np.abs(q) + sums * (np.abs(ds).T @ np.abs(q))
    bv = bw.T @ np.abs(dO) + sums * (w.T @ np.abs(dO))
    return bo, blse, bq, bk, bv


def pack_bounds(q, k, v, cu, window, sinks, dtype, dO=None, scale=None):
    """Bounds of o, lse, dq, dk, dv of a pack (gradients with dO)."""
    HQ, D = q.shape[1:]
    G = HQ // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out = dict(o=np.zeros(q.shape), lse=np.zeros(q.shape[:2]), dq=np.zeros(q.shape), dk=np.zeros(k.shape), dv=np.zeros(v.shape))
    for a, b in zip(cu[:-1], cu[1:]):
        seen = A.visible(np.arange(b - a), np.arange(b - a), window, sinks)
        for h in range(HQ):
            r = head_bounds(q[a:b, h], k[a:b, h // G], v[a:b, h // G], seen, scale, dtype, None if dO is None else dO[a:b, h])
            out["o"][a:b, h], out["lse"][a:b, h] = r[:2]
            if dO is not None:
                out["dq"][a:b, h] = r[2]
                out["dk"][a:b, h // G] += r[3]
                out["dv"][a:b, h // G] += r[4]
    return out


def check(name, got, want, bound, dtype=None):
    """|got - want| <= bound, plus with a type the rounding to it."""
    got = got.detach().to("cpu").double().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine) and np.array_equal(got[~fine], want[~fine]), name
    err = np.abs(got[fine] - want[fine])
    bound = bound[fine] + (0.0 if dtype is None else U[dtype] * np.abs(want[fine]) + LEAST[dtype])
    assert (err <= bound).all(), (name, float(err.max()), float((err / np.maximum(bound, 1e-300)).max()))
