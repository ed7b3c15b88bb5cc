"""Causal softmax attention with a window and sinks, its gradients, and the paged key-value cache in fp64
on the CPU, from their definitions. numpy arrays: q, dO [T, HQ, D], k, v [T, HK, D], cu a list of
boundaries, caches [pages, page_size, HK, D], table [N, columns], offsets [N]. The query at position t
sees keys j <= t with window == 0, j > t - window or j < sinks."""
import numpy as np

from oracle import layer


def visible(t, j, window, sinks):
    """[len(t), len(j)]"""
    t, j = np.asarray(t)[:, None], np.asarray(j)[None]
    return (j <= t) & ((window == 0) | (j > t - window) | (j < sinks))


def head(q, k, v, seen, scale):
    """One head: q [L, D], k, v [keys, D], seen [L, keys] -> (o, lse, weights); rows that see nothing: 0, -inf, 0."""
    # keys that no row sees may hold anything
    some = seen.any(0)[:, None]
    k, v = np.where(some, k, 0.0), np.where(some, v, 0.0)
    s = np.where(seen, scale * (q @ k.T), -np.inf)
    top = s.max(1, initial=-np.inf, keepdims=True)
    p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    total = p.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.log(total[:, 0]) + np.where(np.isfinite(top), top, 0.0)[:, 0]
    w = p / np.where(total > 0, total, 1.0)
    return w @ v, lse, w


def _scale(scale, D):
    return D ** -0.5 if scale is None else scale


def forward(q, k, v, cu, window=0, sinks=0, scale=None):
    """(o [T, HQ, D], lse [T, HQ])"""
    HQ, D = q.shape[1:]
    G = HQ // k.shape[1]
    o, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    for a, b in zip(cu[:-1], cu[1:]):
        seen = visible(np.arange(b - a), np.arange(b - a), window, sinks)
        for h in range(HQ):
            o[a:b, h], lse[a:b, h], _ = head(q[a:b, h], k[a:b, h // G], v[a:b, h // G], seen, _scale(scale, D))
    return o, lse


def backward(q, k, v, cu, dO, window=0, sinks=0, scale=None):
    """dict dq [T, HQ, D], dk, dv [T, HK, D]"""
    HQ, D = q.shape[1:]
    G, scale = HQ // k.shape[1], _scale(scale, D)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for a, b in zip(cu[:-1], cu[1:]):
        seen = visible(np.arange(b - a), np.arange(b - a), window, sinks)
        for h in range(HQ):
            g = h // G
            o, _, w = head(q[a:b, h], k[a:b, g], v[a:b, g], seen, scale)
            ds = scale * w * (dO[a:b, h] @ v[a:b, g].T - (dO[a:b, h] * o).sum(1, keepdims=True))
            dq[a:b, h] = ds @ k[a:b, g]
            dk[a:b, g] += ds.T @ q[a:b, h]
            dv[a:b, g] += w.T @ dO[a:b, h]
    return dict(dq=dq, dk=dk, dv=dv)


def place(table_row, page_size, pages, j):
    """(page, row) of position j, or None where it has none"""
    if j < 0 or j // page_size >= len(table_row):
        return None
    page = int(table_row[j // page_size])
    return (page, j % page_size) if 0 < page < pages else None


def forward_paged(q, k_cache, v_cache, table, cu, offsets, window=0, sinks=0, scale=None):
    """(o, lse) of a call whose tokens are in the cache already"""
    HQ, D = q.shape[1:]
    pages, size, HK = k_cache.shape[:3]
    o, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        t = int(offsets[n]) + np.arange(b - a)
        j = np.arange(max(int(offsets[n]) + b - a, 0))
        at = [place(table[n], size, pages, x) for x in j]
        has = np.array([x is not None for x in at], bool)
        k, v = np.zeros((len(j), HK, D)), np.zeros((len(j), HK, D))
        for x, y in enumerate(at):
            if y is not None:
                k[x], v[x] = k_cache[y], v_cache[y]
        seen = visible(t, j, window, sinks) & has[None]
        for h in range(HQ):
            g = h // (HQ // HK)
            o[a:b, h], lse[a:b, h], _ = head(q[a:b, h], k[:, g], v[:, g], seen, _scale(scale, D))
    return o, lse


def step(q, k_cache, v_cache, table, offsets, window=0, sinks=0, scale=None):
    """(o [N, HQ, D], lse): one token a sequence"""
    return forward_paged(q, k_cache, v_cache, table, list(range(len(q) + 1)), offsets, window, sinks, scale)


def append(k, v, k_cache, v_cache, table, offsets, cu, q=None, inv_freq=(), interleaved=False, mscale=1.0):
    """(q turned or None, k_cache, v_cache afterwards)"""
    pages, size = k_cache.shape[:2]
    pos = layer.positions(cu, offsets)
    turn = lambda x: x if len(inv_freq) == 0 else layer.rotary(x, pos, inv_freq, interleaved, mscale)  # noqa: E731
    k, k_cache, v_cache = turn(k), np.array(k_cache, np.float64), np.array(v_cache, np.float64)
    for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        for t in range(a, b):
            at = place(table[n], size, pages, int(offsets[n]) + t - a)
            if at is not None:
                k_cache[at], v_cache[at] = k[t], v[t]
    return None if q is None else turn(q), k_cache, v_cache
