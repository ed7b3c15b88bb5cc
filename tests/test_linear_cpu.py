"""The linear attention's C entry points on the CPU: every bad argument is refused before anything is
enqueued, and the size queries. No call here reaches a launch; the addresses are never read."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "chunked_gated_delta_04_amd", "libgdn.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libgdn.so not built")

FAKE, OFF = 0x10000, 0x10008
OK, NULL, SHAPE, UNSUPPORTED, SEQLENS, INDEX, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 5, 6, 8


@pytest.fixture(scope="module")
def G():
    from chunked_gated_delta_04_amd import gdn
    return gdn


def ints(*x):
    return (ctypes.c_int32 * len(x))(*x)


def problem(G, N=2, T=130, H=2, HV=4, K=128, V=128, cu=FAKE, host=(0, 70, 130), **strides):
    p = G.GdnLinearProblem()
    p.N, p.T, p.H, p.HV, p.K, p.V, p.cu_seqlens = N, T, H, HV, K, V, cu
    if host is not None:
        p._keep = ints(*host)
        p.cu_seqlens_host = ctypes.cast(p._keep, ctypes.c_void_p)
    for name, x in strides.items():
        setattr(p, name, x)
    return p


def call(G, name, p, order, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, h0=None, o=FAKE, hT=None, saved=None, ws=FAKE, n=1 << 40,
             pool=FAKE, slots=8, idx=FAKE, init=None, host=None, dO=FAKE, dhT=None, dq=FAKE, dk=FAKE,
             dv=FAKE, dh0=None, stream=None)
    a.update(over)
    if a["host"] is not None:
        a["host"] = ctypes.cast(ints(*a["host"]), ctypes.c_void_p)
    return getattr(G._lib, name)(ctypes.byref(p) if p is not None else None, *[a[x] for x in order.split()])


def fwd(G, p, **over):
    return call(G, "gdn_linear_fwd", p, "q k v g h0 o hT saved ws n stream", **over)


def paged(G, p, **over):
    return call(G, "gdn_linear_fwd_paged", p, "q k v g pool slots idx init host o saved ws n stream", **over)


def bwd(G, p, **over):
    return call(G, "gdn_linear_bwd", p, "q k v g saved dO dhT dq dk dv dh0 ws n stream",
                **dict(dict(saved=FAKE), **over))


def step(G, p, **over):
    return call(G, "gdn_linear_step", p, "q k v g pool slots idx host o stream", **over)


@pytest.mark.parametrize("f", [fwd, paged, bwd, step])
def test_problem_is_checked(G, f):
    T = 130 if f is not step else 2
    ok = dict(T=T, host=(0, 70, 130) if f is not step else None)
    assert f(G, None) == NULL
    for bad in (dict(N=-1), dict(T=-1), dict(H=0), dict(HV=0), dict(K=0), dict(V=-1)):
        assert f(G, problem(G, **dict(ok, **bad))) == SHAPE, bad
    for bad in (dict(K=64), dict(V=64), dict(K=32, V=32), dict(K=256, V=256), dict(H=3), dict(H=8)):
        assert f(G, problem(G, **dict(ok, **bad))) == UNSUPPORTED, bad
    for bad in (dict(q_stride=255), dict(q_stride=248), dict(k_stride=260), dict(v_stride=504),
                dict(v_stride=1 << 23), dict(q_stride=-256), dict(k_stride=1 << 40)):
        assert f(G, problem(G, **dict(ok, **bad))) == SHAPE, bad


@pytest.mark.parametrize("f", [fwd, paged, bwd])
def test_pack_is_checked(G, f):
    assert f(G, problem(G, N=0, T=5, host=None)) == SHAPE
    for host in ((1, 70, 130), (0, 70, 129), (0, 131, 130), (0, -1, 130)):
        assert f(G, problem(G, host=host)) == SEQLENS, host
    assert f(G, problem(G, cu=None)) == NULL
    assert f(G, problem(G, N=1 << 21, HV=64, H=64, host=None)) == SHAPE  # more workgroups than a launch takes


def test_pointers_are_checked(G):
    p = problem(G)
    for f, names in ((fwd, "q k v g o"), (paged, "q k v g o pool idx"), (bwd, "q k v g saved dO dq dk dv")):
        for x in names.split():
            assert f(G, p, **{x: None}) == NULL, (f.__name__, x)
    for f, names in ((fwd, "q k v h0 o hT saved ws"), (paged, "q k v o pool saved ws"),
                     (bwd, "q k v saved dO dhT dq dk dv dh0 ws")):
        for x in names.split():
            assert f(G, p, **{x: OFF}) == ALIGN, (f.__name__, x)
    s = problem(G, T=2, host=None)
    for x in "q k v g o pool idx".split():
        assert step(G, s, **{x: None}) == NULL, x
    for x in "q k v o pool".split():
        assert step(G, s, **{x: OFF}) == ALIGN, x
    assert step(G, problem(G, T=3, host=None)) == SHAPE  # one token per row
    assert step(G, s, slots=-1) == SHAPE and paged(G, p, slots=-1) == SHAPE


def test_indices_are_checked(G):
    p, s = problem(G), problem(G, T=2, host=None)
    for f, x in ((paged, p), (step, s)):
        for host in ((1, 8), (3, 3), (1, 1 << 30)):
            assert f(G, x, host=host) == INDEX, (f.__name__, host)


def test_empty_calls(G):
    empty = problem(G, N=0, T=0, host=(0,))
    assert fwd(G, empty, q=None, k=None, v=None, g=None, o=None, ws=None, n=0) == OK
    assert bwd(G, empty, q=None, k=None, v=None, g=None, saved=None, dO=None, dq=None, dk=None, dv=None) == OK
    assert step(G, problem(G, N=0, T=0, host=None), q=None, k=None, v=None, g=None, o=None, pool=None, idx=None) == OK


def test_sizes(G):
    for bad in (dict(K=96, V=96), dict(N=-1), dict(host=(0, 70, 131))):
        p = problem(G, **bad)
        assert G.gdn_linear_saved_size(p) == G.gdn_linear_fwd_workspace_size(p) == G.gdn_linear_bwd_workspace_size(p) == 0
    # states of every sequence at least; they do not depend on the boundaries
    a, b = (problem(G, N=3, T=9000, host=h) for h in ((0, 0, 1, 9000), None))
    assert G.gdn_linear_saved_size(a) == G.gdn_linear_saved_size(b) >= 3 * 4 * 128 * 128 * 4
    assert G.gdn_linear_bwd_workspace_size(a) == G.gdn_linear_bwd_workspace_size(b)
    need = G.gdn_linear_bwd_workspace_size(a)
    assert need > 0 and bwd(G, a, n=need - 1) == WORKSPACE and bwd(G, a, ws=None) == WORKSPACE
    need = G.gdn_linear_fwd_workspace_size(a)
    if need:
        assert fwd(G, a, n=need - 1) == WORKSPACE and fwd(G, a, ws=None) == WORKSPACE


def test_the_binding_refuses_host_tensors(G):
    import torch
    q = torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    g, cu = torch.zeros(1), torch.tensor([0, 4], dtype=torch.int32)
    pool, idx = torch.zeros(5, 1, 64, 64), torch.arange(4, dtype=torch.int32)
    for f in (lambda: G.linear_fwd(q, q, q, g, cu), lambda: G.linear_step(q, q, q, g, pool, idx),
              lambda: G.linear_fwd_paged(q, q, q, g, cu, pool, idx[:1]),
              lambda: G.linear_bwd(q, q, q, g, cu, pool, q)):
        with pytest.raises(ValueError, match="on the GPU"):
            f()
