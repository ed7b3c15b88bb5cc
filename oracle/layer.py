"""Rotary positions and the root-mean-square norm in fp64 on the CPU, from their definitions."""
import numpy as np

E4M3_MAX = 448.0


def rotary(x, positions, inv_freq, interleaved, mscale=1.0, back=False):
    """x [T, heads, D], positions [T], inv_freq [R / 2]: pairs turned by position * inv_freq."""
    y = np.array(x, np.float64)
    half = len(inv_freq)
    a = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = mscale * np.cos(a)[:, None], mscale * np.sin(a)[:, None] * (-1 if back else 1)
    i, j = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
    return y


def positions(cu, offsets=None):
    """A token's place in its sequence, plus the sequence's offset."""
    return np.concatenate([np.arange(b - a) + (0 if offsets is None else offsets[n])
                           for n, (a, b) in enumerate(zip(cu[:-1], cu[1:]))] or [np.zeros(0)])


def rmsnorm(s, weight=None, eps=1e-6, unit=0.0):
    """(y, rstd) of rows s"""
    s = np.asarray(s, np.float64)
    rstd = 1.0 / np.sqrt((s * s).mean(1) + eps)
    return s * rstd[:, None] * (1.0 if weight is None else weight + unit), rstd


def rmsnorm_backward(s, dy, weight=None, eps=1e-6, unit=0.0, ds=None):
    """(dx, dweight)"""
    n, rstd = rmsnorm(s, None, eps)
    dn = dy * (1.0 if weight is None else weight + unit)
    dx = rstd[:, None] * (dn - n * (dn * n).mean(1, keepdims=True))
    return dx + (0.0 if ds is None else ds), (dy * n).sum(0)


def scales(y, group):
    """e4m3 scales of y in groups of columns (0: whole rows): [rows] or [rows, groups]"""
    top = np.abs(y)
    if group:
        top = np.pad(top, ((0, 0), (0, -top.shape[1] % group))).reshape(len(top), -1, group)
    return np.maximum(top.max(-1), 2.0 ** -100) / E4M3_MAX
