"""The attention and cache entry points on the CPU: every bad argument is refused before anything is enqueued, and the workspace
sizes. No call here reaches a launch; the addresses are never read."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "chunked_gated_delta_04_amd", "libgdn.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libgdn.so not built")

FAKE, ODD, HALF = 0x10000, 0x10001, 0x10008
OK, NULL, SHAPE, UNSUPPORTED, SEQLENS, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 6, 8
NAMES = ("fwd", "paged", "step", "bwd")


@pytest.fixture(scope="module")
def G():
    from chunked_gated_delta_04_amd import gdn
    return gdn


def problem(G, host=None, **over):
    p = G.GdnAttnProblem()
    for n, x in dict(dict(N=2, T=10, HQ=4, HK=2, D=64, cu_seqlens=FAKE), **over).items():
        setattr(p, n, x)
    if host is not None:
        p._keep = (ctypes.c_int32 * len(host))(*host)
        p.cu_seqlens_host = ctypes.cast(p._keep, ctypes.c_void_p)
    return p


def cache(G, **over):
    c = G.GdnKvCache()
    for n, x in dict(dict(k=FAKE, v=FAKE, pages=9, page_size=16, columns=4, page_stride=16 * 2 * 64, token_stride=128,
                          head_stride=64, page_table=FAKE, offsets=FAKE), **over).items():
        setattr(c, n, x)
    return c


def call(G, name, ptr=None, n=1 << 40, pool=None, **over):
    if name == "step":
        over = dict(dict(T=over.get("N", 2)), **over)
    p, c = problem(G, **over), cache(G, **(pool or {}))
    t = dict(dict.fromkeys("q k v o lse dO dq dk dv ws".split(), FAKE), **(ptr or {}))
    f = getattr(G._lib, dict(fwd="gdn_attn_fwd", paged="gdn_attn_fwd_paged", step="gdn_attn_step", bwd="gdn_attn_bwd")[name])
    names = dict(fwd="q k v o lse ws", bwd="q k v o lse dO dq dk dv ws").get(name, "q o lse ws").split()
    head = [ctypes.byref(p)] + ([ctypes.byref(c)] if name in ("paged", "step") else [])
    return f(*head, *[t[x] for x in names], n, None)


@pytest.mark.parametrize("name", NAMES)
def test_refuses(G, name):
    for bad in (dict(N=-1, T=10), dict(T=-1), dict(HQ=0), dict(HK=0), dict(D=0), dict(window=-1), dict(sinks=-1), dict(N=0, T=10),
                dict(q_stride=255), dict(q_stride=260), dict(q_stride=1 << 23), dict(HQ=1 << 17, HK=1 << 11), dict(window=(1 << 30) + 1),
                dict(sinks=(1 << 30) + 1), dict(T=(1 << 30) + 1, HQ=1, HK=1), dict(T=1 << 29, HQ=4)):
        assert call(G, name, **bad) == SHAPE, bad
    for bad in (dict(D=32), dict(D=96), dict(D=512), dict(HQ=5), dict(HQ=129, HK=1), dict(dtype=2), dict(dtype=-1), dict(dtype=3)):
        assert call(G, name, **bad) == UNSUPPORTED, bad
    needed = dict(fwd="q k v o", paged="q o", step="q o", bwd="q k v o lse dO dq dk dv")[name].split()
    for x in needed:
        assert call(G, name, ptr={x: None}) == NULL, x
        assert call(G, name, ptr={x: ODD}) == ALIGN, x
        assert x == "lse" or call(G, name, ptr={x: HALF}) == ALIGN, x
    if name != "step":
        assert call(G, name, cu_seqlens=None) == NULL
        for host in ((0, 5, 9), (1, 5, 10), (0, 11, 10)):
            assert call(G, name, host=host) == SEQLENS, host
    else:
        assert call(G, name, N=2, T=3) == SHAPE
    assert call(G, name, N=0, T=0, ptr=dict.fromkeys("q k v o lse dO dq dk dv ws".split())) == OK
    if name in ("fwd", "bwd"):
        for bad in (dict(k_stride=127), dict(v_stride=132), dict(k_stride=1 << 23)):
            assert call(G, name, **bad) == SHAPE, bad


@pytest.mark.parametrize("name", ("paged", "step"))
def test_refuses_caches(G, name):
    for bad in (dict(pages=-1), dict(page_size=0), dict(page_size=-4), dict(columns=-1), dict(table_stride=-1),
                dict(token_stride=63), dict(head_stride=68), dict(page_stride=0), dict(token_stride=132), dict(page_stride=1 << 41)):
        assert call(G, name, pool=bad) == SHAPE, bad
    for bad in (dict(k=None), dict(v=None), dict(page_table=None), dict(offsets=None)):
        assert call(G, name, pool=bad) == NULL, bad
    for bad in (dict(k=HALF), dict(v=HALF), dict(page_table=ODD), dict(offsets=ODD)):
        assert call(G, name, pool=bad) == ALIGN, bad
    f = G._lib.gdn_attn_step if name == "step" else G._lib.gdn_attn_fwd_paged
    assert f(ctypes.byref(problem(G, T=2)), None, FAKE, FAKE, None, None, 0, None) == NULL
    assert f(None, ctypes.byref(cache(G)), FAKE, FAKE, None, None, 0, None) == NULL


def test_workspaces(G):
    """Sizes from the extents; a short or missing workspace is refused."""
    lib, ref = G._lib, ctypes.byref
    long = problem(G, T=20000)
    assert lib.gdn_attn_bwd_workspace_size(ref(long)) > 2 * 20000 * 4 * 4
    for name, need in (("bwd", lib.gdn_attn_bwd_workspace_size(ref(problem(G)))),):
        assert call(G, name, n=need - 1) == WORKSPACE and call(G, name, ptr=dict(ws=None)) == WORKSPACE
        assert call(G, name, ptr=dict(ws=HALF)) == ALIGN
    big = cache(G, columns=4096)
    need = lib.gdn_attn_step_workspace_size(ref(problem(G, T=2)), ref(big))
    assert need > 0 and call(G, "step", n=need - 1, pool=dict(columns=4096)) == WORKSPACE
    need = lib.gdn_attn_fwd_paged_workspace_size(ref(problem(G)), ref(big))
    assert need > 0 and call(G, "paged", n=need - 1, pool=dict(columns=4096)) == WORKSPACE
    assert lib.gdn_attn_step_workspace_size(ref(problem(G, T=2, window=50)), ref(big)) < lib.gdn_attn_step_workspace_size(
        ref(problem(G, T=2)), ref(big))
    # the same with and without the host's boundaries
    for q in ("fwd", "bwd"):
        f = getattr(lib, f"gdn_attn_{q}_workspace_size")
        assert f(ref(problem(G, T=5000))) == f(ref(problem(G, T=5000, host=(0, 1, 5000))))
    for bad in (problem(G, D=32), problem(G, T=-1)):
        assert lib.gdn_attn_fwd_workspace_size(ref(bad)) == lib.gdn_attn_bwd_workspace_size(ref(bad)) == 0
        assert lib.gdn_attn_step_workspace_size(ref(bad), ref(big)) == 0
    assert lib.gdn_attn_step_workspace_size(ref(problem(G, T=3)), ref(big)) == 0
    # sinks of many sequences: at most some times the gradients themselves
    many = problem(G, N=5000, T=100000, window=16, sinks=4)
    assert lib.gdn_attn_bwd_workspace_size(ref(many)) < 40 * 100000 * 2 * 64 * 4


def append(G, ptr=None, pool=None, host=None, **over):
    p = G.GdnKvAppendProblem()
    for n, x in dict(dict(N=2, T=10, HQ=4, HK=2, D=64, R=32, cu_seqlens=FAKE), **over).items():
        setattr(p, n, x)
    if host is not None:
        p._keep = (ctypes.c_int32 * len(host))(*host)
        p.cu_seqlens_host = ctypes.cast(p._keep, ctypes.c_void_p)
    t = dict(dict.fromkeys("f q k v qo".split(), FAKE), **(ptr or {}))
    return G._lib.gdn_kv_append(ctypes.byref(p), ctypes.byref(cache(G, **(pool or {}))), *[t[x] for x in "f q k v qo".split()], None)


def test_append_refuses(G):
    for bad in (dict(N=-1), dict(T=-1), dict(HQ=-1), dict(HK=0), dict(D=0), dict(N=0), dict(q_stride=255), dict(k_stride=127),
                dict(v_stride=-128), dict(q_out_stride=1 << 31), dict(HQ=1 << 24), dict(cu_seqlens=None), dict(T=(1 << 30) + 1)):
        assert append(G, **bad) == SHAPE, bad
    for bad in (dict(R=-2), dict(R=31), dict(R=66), dict(D=1026), dict(interleaved=2), dict(dtype=2), dict(dtype=-1)):
        assert append(G, **bad) == UNSUPPORTED, bad
    for host in ((0, 5, 9), (1, 5, 10), (0, 11, 10)):
        assert append(G, host=host) == SEQLENS, host
    for x in "f q k v qo".split():
        assert append(G, ptr={x: None}) == NULL, x
        assert append(G, ptr={x: ODD}) == ALIGN, x
    for bad in (dict(k=None), dict(v=None), dict(page_table=None), dict(offsets=None)):
        assert append(G, pool=bad) == NULL, bad
    for bad in (dict(k=ODD), dict(v=ODD), dict(page_table=0x10002), dict(offsets=0x10002)):
        assert append(G, pool=bad) == ALIGN, bad
    for bad in (dict(page_size=0), dict(pages=-1), dict(columns=-1), dict(token_stride=1), dict(table_stride=-4)):
        assert append(G, pool=bad) == SHAPE, bad
    p = G.GdnKvAppendProblem()
    assert G._lib.gdn_kv_append(None, ctypes.byref(cache(G)), FAKE, FAKE, FAKE, FAKE, FAKE, None) == NULL
    p.HK, p.D = 1, 64
    assert G._lib.gdn_kv_append(ctypes.byref(p), None, FAKE, FAKE, FAKE, FAKE, FAKE, None) == NULL
    assert append(G, N=0, T=0, ptr=dict.fromkeys("f q k v qo".split())) == OK


def test_the_binding_refuses_host_tensors(G):
    import torch
    x, i = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    for f in (lambda: G.attn_fwd(x, x, x, i), lambda: G.attn_bwd(x, x, x, i, x, x[..., 0].float(), x),
              lambda: G.attn_fwd_paged(x, c, c, i[None], i, i), lambda: G.attn_step(x, c, c, i[:, None], i),
              lambda: G.kv_append(x, x, c, c, i[:, None], i)):
        with pytest.raises(ValueError, match="on the GPU"):
            f()
