"""Linear attention with a decay for each head in fp64 on the CPU, token by token from its recurrence
S_t = lam S_{t-1} + v_t k_t^T, o_t = scale S_t q_t, with a hand-written adjoint. numpy arrays:
q, k [T, H, D], v, dO [T, HV, D], log_decay [HV], states [N, HV, V, K], cu a list of boundaries."""
import numpy as np


def _spread(x, HV):
    return np.repeat(x, HV // x.shape[1], axis=1)


def _lam(log_decay):
    return np.exp(np.asarray(log_decay, np.float64))[:, None, None]


def forward(q, k, v, log_decay, cu, h0=None, scale=None):
    """(o [T, HV, D], hT [N, HV, V, K])"""
    HV, D = v.shape[1:]
    scale = D ** -0.5 if scale is None else scale
    lam, qs, ks = _lam(log_decay), _spread(q, HV), _spread(k, HV)
    o, hT = np.zeros(v.shape), np.zeros((len(cu) - 1, HV, D, D))
    for n in range(len(cu) - 1):
        S = np.zeros((HV, D, D)) if h0 is None else np.array(h0[n], np.float64)
        for t in range(cu[n], cu[n + 1]):
            S = lam * S + v[t][:, :, None] * ks[t][:, None, :]
            o[t] = scale * (S @ qs[t][:, :, None])[..., 0]
        hT[n] = S
    return o, hT


def backward(q, k, v, log_decay, cu, dO, h0=None, dhT=None, scale=None):
    """dict dq, dk [T, H, D], dv [T, HV, D], dh0 [N, HV, V, K]"""
    T, H, D = q.shape
    HV = v.shape[1]
    scale = D ** -0.5 if scale is None else scale
    lam, qs, ks = _lam(log_decay), _spread(q, HV), _spread(k, HV)
    dq, dk, dv = np.zeros((T, HV, D)), np.zeros((T, HV, D)), np.zeros(v.shape)
    dh0 = np.zeros((len(cu) - 1, HV, D, D))
    for n in range(len(cu) - 1):
        S = np.zeros((HV, D, D)) if h0 is None else np.array(h0[n], np.float64)
        for t in range(cu[n], cu[n + 1]):
            S = lam * S + v[t][:, :, None] * ks[t][:, None, :]
            dq[t] = scale * (dO[t][:, None, :] @ S)[:, 0]
        G = np.zeros((HV, D, D)) if dhT is None else np.array(dhT[n], np.float64)
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            G = G + scale * dO[t][:, :, None] * qs[t][:, None, :]
            dv[t] = (G @ ks[t][:, :, None])[..., 0]
            dk[t] = (v[t][:, None, :] @ G)[:, 0]
            G = lam * G
        dh0[n] = G
    fold = lambda x: x.reshape(T, H, HV // H, D).sum(2)  # noqa: E731
    return dict(dq=fold(dq), dk=fold(dk), dv=dv, dh0=dh0)


def step(q, k, v, log_decay, pool, idx, scale=None):
    """(o [N, HV, D], the pool afterwards): rows whose index is <= 0 or past the pool give zeros."""
    HV, D = v.shape[1:]
    scale = D ** -0.5 if scale is None else scale
    lam, qs, ks = _lam(log_decay), _spread(q, HV), _spread(k, HV)
    pool, o = np.array(pool, np.float64), np.zeros(v.shape)
    for n, i in enumerate(idx):
        if 0 < i < pool.shape[0]:
            pool[i] = lam * pool[i] + v[n][:, :, None] * ks[n][:, None, :]
            o[n] = scale * (pool[i] @ qs[n][:, :, None])[..., 0]
    return o, pool
