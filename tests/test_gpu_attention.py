"""The softmax attention on the GPU, over packs and their gradients, against the fp64 oracle. Tolerances: see attention_bounds."""
import sys

import numpy as np
import pytest
import torch

from oracle import attention as A
from tests.attention_bounds import check, pack_bounds
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def rows(T, H, D, dt, gen, pad=0):
    """[T, H, D]: a tensor of its own, or with pad a slice of wider rows"""
    x = torch.randn(T, H * D + pad, generator=gen).to(dt).cuda()
    return x[:, :H * D].unflatten(1, (H, D)) if pad else x.view(T, H, D)


def make(lens, HQ, HK, D, dtype, seed=0, pad=0):
    gen = torch.Generator().manual_seed(seed)
    dt, T = TYPES[dtype], sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    return (rows(T, HQ, D, dt, gen, pad), rows(T, HK, D, dt, gen, pad), rows(T, HK, D, dt, gen, 2 * pad), rows(T, HQ, D, dt, gen),
            cu, torch.tensor(cu, dtype=torch.int32, device="cuda"))


CASES = [  # lens, HQ, HK, D, dtype, window, sinks, padding of the rows
    ([1], 1, 1, 64, "bf16", 0, 0, 0), ([1], 2, 1, 256, "fp16", 0, 0, 8), ([0, 2, 0, 3, 0], 3, 1, 128, "bf16", 0, 0, 8),
    ([63, 64, 65, 1, 127, 128, 129], 4, 2, 64, "bf16", 0, 0, 16), ([300], 5, 1, 128, "fp16", 0, 0, 0),
    ([200, 31], 8, 2, 256, "bf16", 0, 0, 8), ([190], 16, 1, 128, "bf16", 0, 0, 0), ([70, 5], 64, 1, 64, "fp16", 0, 0, 0),
    ([40], 128, 1, 64, "bf16", 0, 0, 0), ([150, 90], 7, 7, 128, "bf16", 1, 0, 0), ([400, 33], 4, 2, 128, "bf16", 50, 4, 0),
    ([500], 2, 1, 64, "fp16", 64, 1, 0), ([260, 300], 6, 2, 256, "bf16", 100, 130, 8), ([700], 4, 1, 64, "bf16", 7, 200, 0),
    ([333, 12, 90], 3, 3, 128, "fp16", 1000, 5, 0), ([129] * 9, 2, 2, 64, "bf16", 128, 128, 0), ([257], 24, 8, 64, "bf16", 33, 3, 0),
]


@pytest.mark.parametrize("lens, HQ, HK, D, dtype, window, sinks, pad", CASES)
def test_forward_and_gradients(lens, HQ, HK, D, dtype, window, sinks, pad):
    say(lens, HQ, HK, D, dtype, window, sinks, pad)
    q, k, v, dO, cu, dcu = make(lens, HQ, HK, D, dtype, seed=D + len(lens), pad=pad)
    host = torch.tensor(cu, dtype=torch.int32)
    o, lse = gdn.attn_fwd(q, k, v, dcu, window=window, sinks=sinks, cu_seqlens_host=host, want_lse=True)
    args = [f64(x) for x in (q, k, v)]
    want, want_lse = A.forward(*args, cu, window, sinks)
    bound = pack_bounds(*args, cu, window, sinks, dtype, f64(dO))
    check("o", o, want, bound["o"])
    check("lse", lse, want_lse, bound["lse"])
    g = gdn.attn_bwd(q, k, v, dcu, o, lse, dO, window=window, sinks=sinks)
    ref = A.backward(*args, cu, f64(dO), window, sinks)
    for n in ("dq", "dk", "dv"):
        check(n, g[n], ref[n], bound[n], dtype)
    # the same bits again, without the host's boundaries, and without lse
    again, none = gdn.attn_fwd(q, k, v, dcu, window=window, sinks=sinks)
    assert none is None and torch.equal(o, again)
    g2 = gdn.attn_bwd(q, k, v, dcu, o, lse, dO, window=window, sinks=sinks, cu_seqlens_host=host)
    assert all(torch.equal(g[n], g2[n]) for n in g)


def plain(q, k, v, cu, window, sinks, scale, dO):
    """Forward and gradients in fp64 on the GPU, a head of a sequence at a time."""
    q, k, v, dO = (x.double() for x in (q, k, v, dO))
    HQ, HK = q.shape[1], k.shape[1]
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a, b in zip(cu[:-1], cu[1:]):
        i = torch.arange(b - a, device=q.device)
        off = (i[None] > i[:, None]) | ((i[:, None] - i[None] >= window) & (i[None] >= sinks) if window else False)
        for h in range(HQ):
            g = h // (HQ // HK)
            x, y, z, d = q[a:b, h], k[a:b, g], v[a:b, g], dO[a:b, h]
            s = (scale * (x @ y.T)).masked_fill_(off, -float("inf"))
            lse[a:b, h] = torch.logsumexp(s, 1)
            w = torch.exp(s - lse[a:b, h, None])
            o[a:b, h] = w @ z
            ds = scale * w * (d @ z.T - (d * o[a:b, h]).sum(1, keepdim=True))
            dq[a:b, h] = ds @ y
            dk[a:b, g] += ds.T @ x
            dv[a:b, g] += w.T @ d
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)


@pytest.mark.parametrize("lens, HQ, HK, D, dtype, window, sinks", [
    ([4100, 700], 8, 2, 128, "bf16", 0, 0), ([6000], 4, 1, 256, "bf16", 0, 0), ([9000, 1], 2, 2, 64, "fp16", 0, 0),
    ([8200], 4, 1, 128, "bf16", 300, 5), ([5000, 3000], 3, 1, 64, "bf16", 64, 260), ([4096], 2, 1, 256, "fp16", 1000, 1),
])
def test_long(lens, HQ, HK, D, dtype, window, sinks):
    """Long sequences: parts of the keys, of the rows and of the sinks' rows, by relative 2-norms: the roundings to the type of a
    weight or score gradient and of the output, at most u each and both of any sign, are below 2 u of a tensor's norm; dq, dk have
    delta's too, from the rounded o: 3 u."""
    say(lens, HQ, HK, D, dtype, window, sinks)
    q, k, v, dO, cu, dcu = make(lens, HQ, HK, D, dtype, seed=3)
    o, lse = gdn.attn_fwd(q, k, v, dcu, window=window, sinks=sinks, want_lse=True)
    g = gdn.attn_bwd(q, k, v, dcu, o, lse, dO, window=window, sinks=sinks)
    ref = plain(q, k, v, cu, window, sinks, D ** -0.5, dO)
    u = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[dtype]
    for n, x in dict(g, o=o).items():
        assert float((x.double() - ref[n]).norm()) <= (3 if n in ("dq", "dk") else 2) * u * float(ref[n].norm()), n
    assert float((lse.double() - ref["lse"]).abs().max()) < 2.0 ** -12


def test_rows_behind_the_last_sequence_stay():
    q, k, v, dO, _, _ = make([300], 4, 2, 128, "bf16", seed=1)
    cu = torch.tensor([0, 100, 201], dtype=torch.int32, device="cuda")
    p = gdn.GdnAttnProblem(2, 300, 4, 2, 128, 0, 60, 3, 0.0, cu.data_ptr(), None, 0, 0, 0)
    import ctypes
    out = {n: torch.full_like(t, 7.0) for n, t in dict(o=q, dq=q, dk=k, dv=v).items()}
    lse = torch.full((300, 4), 7.0, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(max(gdn._lib.gdn_attn_fwd_workspace_size(ctypes.byref(p)), gdn._lib.gdn_attn_bwd_workspace_size(ctypes.byref(p))),
                     dtype=torch.uint8, device="cuda")
    ptr = lambda *t: [x.data_ptr() for x in t]  # noqa: E731
    gdn._check(gdn._lib.gdn_attn_fwd(ctypes.byref(p), *ptr(q, k, v, out["o"], lse, ws), ws.numel(), s), "fwd")
    gdn._check(gdn._lib.gdn_attn_bwd(ctypes.byref(p), *ptr(q, k, v, out["o"], lse, dO, out["dq"], out["dk"], out["dv"], ws),
                                     ws.numel(), s), "bwd")
    for n, t in dict(out, lse=lse).items():
        assert bool((t[201:] == 7.0).all()), n
        assert not bool((t[:201] == 7.0).all()), n
    short, _ = gdn.attn_fwd(q[:201], k[:201], v[:201], cu, window=60, sinks=3)
    args = [f64(x[:201]) for x in (q, k, v)]
    bound = pack_bounds(*args, [0, 100, 201], 60, 3, "bf16")
    want, _ = A.forward(*args, [0, 100, 201], 60, 3)
    check("o", out["o"][:201], want, bound["o"])
    check("o", short, want, bound["o"])


def test_no_tokens():
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    o, lse = gdn.attn_fwd(e, e[:, :2], e[:, :2], cu, want_lse=True)
    assert o.shape == e.shape and lse.shape == (0, 4)
    g = gdn.attn_bwd(e, e[:, :2], e[:, :2], cu, o, lse, e)
    assert g["dk"].shape == (0, 2, 64)


def test_scale_and_large_scores():
    """Scores of some hundreds: the weights are nearly those of one key."""
    q, k, v, dO, cu, dcu = make([200], 2, 1, 64, "bf16", seed=9)
    q = q * 16
    o, lse = gdn.attn_fwd(q, k, v, dcu, scale=0.5, want_lse=True)
    args = [f64(x) for x in (q, k, v)]
    want, want_lse = A.forward(*args, cu, scale=0.5)
    bound = pack_bounds(*args, cu, 0, 0, "bf16", f64(dO), scale=0.5)
    check("o", o, want, bound["o"])
    check("lse", lse, want_lse, bound["lse"])
    g = gdn.attn_bwd(q, k, v, dcu, o, lse, dO, scale=0.5)
    ref = A.backward(*args, cu, f64(dO), scale=0.5)
    for n in ("dq", "dk", "dv"):
        check(n, g[n], ref[n], bound[n], "bf16")


def test_nan_stays_in_its_sequence():
    q, k, v, dO, cu, dcu = make([90, 100, 80], 4, 2, 64, "bf16", seed=2)
    o, lse = gdn.attn_fwd(q, k, v, dcu, want_lse=True)
    g = gdn.attn_bwd(q, k, v, dcu, o, lse, dO)
    for i in range(3):
        y = [t.clone() for t in (q, k, v)]
        y[i][120] = float("nan")
        o2, lse2 = gdn.attn_fwd(*y, dcu, want_lse=True)
        g2 = gdn.attn_bwd(*y, dcu, o2, lse2, dO)
        for a, b in ((o, o2), (lse, lse2), *((g[n], g2[n]) for n in g)):
            assert torch.equal(a[:90], b[:90]) and torch.equal(a[190:], b[190:])
        assert bool(o2[120].isnan().any())
