"""The rotary and norm entry points on the CPU: every bad argument is refused before anything is
enqueued, and the host's frequency table. No call here reaches a launch; the addresses are never read."""
import ctypes
import math
import os

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "chunked_gated_delta_04_amd", "libgdn.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libgdn.so not built")

FAKE, ODD = 0x10000, 0x10001
OK, NULL, SHAPE, UNSUPPORTED, SEQLENS, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 6, 8


@pytest.fixture(scope="module")
def G():
    from chunked_gated_delta_04_amd import gdn
    return gdn


def rotary(G, back=False, host=None, ptr=None, **over):
    p = G.GdnRotaryProblem()
    a = dict(T=10, HQ=4, HK=2, D=64, R=32, interleaved=0, dtype=0, N=2, cu_seqlens=FAKE)
    for n, x in dict(a, **over).items():
        setattr(p, n, x)
    if host is not None:
        keep = (ctypes.c_int32 * len(host))(*host)
        p.cu_seqlens_host = ctypes.cast(keep, ctypes.c_void_p)
    t = dict(f=FAKE, q=FAKE, k=FAKE, qo=FAKE, ko=FAKE)
    t.update(ptr or {})
    f = G._lib.gdn_rotary_bwd if back else G._lib.gdn_rotary
    return f(ctypes.byref(p), t["f"], t["q"], t["k"], t["qo"], t["ko"], None)


@pytest.mark.parametrize("back", [False, True])
def test_rotary_refuses(G, back):
    assert (G._lib.gdn_rotary_bwd if back else G._lib.gdn_rotary)(None, FAKE, FAKE, FAKE, FAKE, FAKE, None) == NULL
    for bad in (dict(T=-1), dict(HQ=0), dict(HK=-1), dict(D=0), dict(N=-1), dict(N=0), dict(q_stride=255),
                dict(k_stride=127), dict(q_out_stride=-256), dict(k_out_stride=1 << 31), dict(HQ=1 << 24),
                dict(T=(1 << 25) + 1)):
        assert rotary(G, back, **bad) == SHAPE, bad
    for bad in (dict(R=0), dict(R=31), dict(R=66), dict(R=-2), dict(D=1026), dict(interleaved=2), dict(dtype=3),
                dict(dtype=-1)):
        assert rotary(G, back, **bad) == UNSUPPORTED, bad
    for host in ((0, 5, 9), (1, 5, 10), (0, 11, 10)):
        assert rotary(G, back, host=host) == SEQLENS, host
    for x in ("f", "q", "k", "qo", "ko"):
        assert rotary(G, back, ptr={x: None}) == NULL, x
    assert rotary(G, back, cu_seqlens=None) == NULL
    for x in ("q", "k", "qo", "ko"):
        assert rotary(G, back, ptr={x: ODD}) == ALIGN, x
    assert rotary(G, back, T=0, N=0, ptr=dict(q=None, k=None, qo=None, ko=None, f=None)) == OK


def norm(G, back=False, ptr=None, n=1 << 40, **over):
    p = G.GdnRmsnormProblem()
    for name, x in dict(dict(rows=10, D=64, dtype=0, unit_offset=0, group=0, eps=1e-6), **over).items():
        setattr(p, name, x)
    t = dict(x=FAKE, r=FAKE, w=FAKE, so=FAKE, y=FAKE, y8=FAKE, sc=FAKE, rstd=FAKE, dy=FAKE, ds=None, dx=FAKE, dw=FAKE,
             ws=FAKE)
    t.update(ptr or {})
    if back:
        return G._lib.gdn_rmsnorm_bwd(ctypes.byref(p), *[t[i] for i in "x w rstd dy ds dx dw ws".split()], n, None)
    return G._lib.gdn_rmsnorm_fwd(ctypes.byref(p), *[t[i] for i in "x r w so y y8 sc rstd".split()], None)


@pytest.mark.parametrize("back", [False, True])
def test_norm_refuses(G, back):
    for bad in (dict(rows=-1), dict(D=0), dict(D=-5), dict(x_stride=63), dict(x_stride=-64), dict(residual_stride=1),
                dict(x_stride=1 << 31), dict(rows=1 << 24, D=8192), dict(rows=(1 << 31) - 1, D=5120)):
        assert norm(G, back, **bad) == SHAPE, bad
    for bad in (dict(D=16385), dict(dtype=3), dict(dtype=-1), dict(group=64), dict(group=-1), dict(unit_offset=2)):
        assert norm(G, back, **bad) == UNSUPPORTED, bad
    if back:
        for x in ("x", "rstd", "dy", "dx"):
            assert norm(G, back, ptr={x: None}) == NULL, x
        for x in ("x", "w", "rstd", "dy", "ds", "dx", "dw", "ws"):
            assert norm(G, back, ptr={x: ODD}) == ALIGN, x
        assert norm(G, back, ptr=dict(ws=None)) == WORKSPACE
        p = G.GdnRmsnormProblem()
        p.rows, p.D = 10, 64
        need = G.gdn_rmsnorm_bwd_workspace_size(p)
        assert need > 0 and norm(G, back, n=need - 1) == WORKSPACE
        p.D = 20000
        assert G.gdn_rmsnorm_bwd_workspace_size(p) == 0
    else:
        for x in (dict(x=None), dict(so=None), dict(y=None, y8=None), dict(sc=None)):
            assert norm(G, back, ptr=x) == NULL, x
        for x in ("x", "r", "w", "so", "y", "sc", "rstd"):
            assert norm(G, back, ptr={x: ODD}) == ALIGN, x
        assert norm(G, rows=0, ptr=dict(x=None, r=None, y=None, y8=None)) == OK


def test_inverse_frequencies(G):
    R, base = 64, 10000.0
    j = np.arange(R // 2)
    f = base ** (-2.0 * j / R)
    get = lambda *a, **k: (lambda t: (t[0].numpy().astype(np.float64), t[1]))(G.rotary_inv_freq(*a, **k))  # noqa: E731
    near = lambda a, b: np.allclose(a, b, rtol=2.0 ** -23, atol=0)  # noqa: E731
    x, m = get(R, base)
    assert near(x, f) and m == 1.0
    x, m = get(R, base, "linear", factor=4.0)
    assert near(x, f / 4) and m == 1.0
    x, m = get(R, base, "ntk", factor=4.0)
    assert near(x[0], 1.0) and near(x[-1], f[-1] / 4) and m == 1.0
    x, m = get(R, base, "yarn", factor=8.0, original=4096)
    turns = 4096 * f / (2 * math.pi)
    assert near(x[turns >= 40], f[turns >= 40]) and near(x[turns <= 0.8], f[turns <= 0.8] / 8)
    assert (np.diff(x) < 0).all() and abs(m - (1 + 0.1 * math.log(8))) < 1e-6
    assert near(get(R, base, "yarn", factor=1.0, original=4096)[0], f)


@pytest.mark.parametrize("status, args", [
    (SHAPE, (3, 1e4, 0, 1, 1)), (SHAPE, (0, 1e4, 0, 1, 1)), (SHAPE, (64, 1.0, 0, 1, 1)), (SHAPE, (64, float("nan"), 0, 1, 1)),
    (SHAPE, (64, 1e4, 1, 0.5, 1)), (SHAPE, (64, 1e4, 2, float("inf"), 1)), (SHAPE, (2, 1e4, 2, 2, 1)),
    (SHAPE, (64, 1e4, 3, 2, 0)), (SHAPE, (2048, 1e4, 0, 1, 1)), (UNSUPPORTED, (64, 1e4, 4, 1, 1)), (UNSUPPORTED, (64, 1e4, -1, 1, 1)),
])
def test_inverse_frequencies_refuse(G, status, args):
    out, m = (ctypes.c_float * 512)(), ctypes.c_float()
    assert G._lib.gdn_rotary_inv_freq(*args, ctypes.cast(out, ctypes.c_void_p), ctypes.byref(m)) == status
    assert not any(out)
    assert G._lib.gdn_rotary_inv_freq(64, 1e4, 0, 1, 1, None, ctypes.byref(m)) == NULL


def test_the_binding_refuses_host_tensors(G):
    import torch
    x = torch.zeros(4, 2, 64)
    for f in (lambda: G.rotary(x, x, torch.zeros(32), positions=torch.zeros(4, dtype=torch.int32)),
              lambda: G.rotary_bwd(x, x, torch.zeros(32), positions=torch.zeros(4, dtype=torch.int32)),
              lambda: G.rmsnorm_fwd(x[:, 0]), lambda: G.rmsnorm_bwd(x[:, 0], x[:, 0], None, torch.zeros(4))):
        with pytest.raises(ValueError, match="on the GPU"):
            f()
