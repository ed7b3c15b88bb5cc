"""Caches in the orders of memory that the binding takes, shared pages, what it refuses, and rows of outputs that no sequence holds."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn


def bf(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("pages, size, HK", [(9, 16, 1), (3, 1, 2), (9, 1, 1), (2, 16, 1)])
def test_an_extent_of_one_has_no_stride(pages, size, HK):
    """The same memory with another stride where the extent is 1, as transposing and slicing leave it, in k's cache or in v's."""
    D, N = 64, 2
    kc, vc, k, q = bf(pages, size, HK, D), bf(pages, size, HK, D, seed=1), bf(N, HK, D, seed=2), bf(N, 2 * HK, D, seed=3)
    table, past = ints(1, 1, 1, 1).view(2, 2), ints(0, 0 if size == 1 else 7)

    def odd(c):
        s = [99991 if n == 1 else x for n, x in zip(c.shape, c.stride())]
        return torch.as_strided(c, c.shape, s)

    want = gdn.attn_step(q, kc, vc, table, past)[0]
    for a, b in ((odd(kc), vc), (kc, odd(vc)), (odd(kc), odd(vc))):
        assert torch.equal(gdn.attn_step(q, a, b, table, past)[0], want)
    x, y = kc.clone(), vc.clone()
    gdn.kv_append(k[:1], k[:1], x, y, table[:1], past[:1])
    u, w = kc.clone(), vc.clone()
    gdn.kv_append(k[:1], k[:1], u, odd(w), table[:1], past[:1])
    assert torch.equal(u, x) and torch.equal(w, y) and not torch.equal(x, kc)


def test_what_is_no_cache_or_token():
    """A cache or tokens of another number of extents: the binding's own errors."""
    q, k, kc, t, off = bf(1, 4, 64), bf(1, 2, 64), bf(5, 16, 2, 64), ints(1, 2)[None], ints(0)
    for bad in (kc[0, 0], kc[0, 0, 0], kc[None], kc.flatten()):
        for f in (lambda: gdn.attn_step(q, bad, bad, t, off), lambda: gdn.attn_fwd_paged(q, bad, bad, t, ints(0, 1), off),
                  lambda: gdn.kv_append(k, k, bad, bad, t, off)):
            with pytest.raises(ValueError, match="k_cache must be"):
                f()


def behind(T, cu, D, paged, window=0, sinks=0):
    """outputs of a call whose last sequence ends before T, and of one without the rows behind"""
    import ctypes
    HQ, HK, size = 4, 2, 16
    q, k, v = bf(T, HQ, D), bf(T, HK, D, seed=1), bf(T, HK, D, seed=2)
    N, dcu = len(cu) - 1, ints(*cu)
    o, lse = torch.full_like(q, 7.0), torch.full((T, HQ), 7.0, device="cuda")
    p = gdn.GdnAttnProblem(N, T, HQ, HK, D, 0, window, sinks, 0.0, dcu.data_ptr(), None, 0, 0, 0)
    args = [ctypes.byref(p)]
    if paged:
        cols = 300
        table = (torch.arange(N * cols, dtype=torch.int32).view(N, cols) + 1).cuda()
        kc, vc = bf(N * cols + 1, size, HK, D, seed=1), bf(N * cols + 1, size, HK, D, seed=2)
        past = ints(*[700 + n for n in range(N)])
        c = gdn._cache(kc, vc, table, past, N, HK, D, q.dtype, q.device)
        args.append(ctypes.byref(c))
        name, ptrs = "gdn_attn_fwd_paged", [q]
        want = gdn.attn_fwd_paged(q[:cu[-1]], kc, vc, table, dcu, past, window=window, sinks=sinks, want_lse=True)
    else:
        name, ptrs = "gdn_attn_fwd", [q, k, v]
        want = gdn.attn_fwd(q[:cu[-1]], k[:cu[-1]], v[:cu[-1]], dcu, window=window, sinks=sinks, want_lse=True)
    n = getattr(gdn._lib, name + "_workspace_size")(*args)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda").fill_(255)
    gdn._check(getattr(gdn._lib, name)(*args, *[x.data_ptr() for x in ptrs], o.data_ptr(), lse.data_ptr(), ws.data_ptr(), n,
                                       torch.cuda.current_stream().cuda_stream), name)
    return o, lse, want, n


@pytest.mark.parametrize("D, window, sinks", [(64, 0, 0), (128, 900, 3), (256, 0, 0)])
@pytest.mark.parametrize("paged", [False, True])
def test_rows_behind_the_last_sequence_stay_where_keys_are_split(D, paged, window, sinks):
    """Against the call without those rows, whose parts of the keys may be others: a rounding of o and 2^-12 of lse."""
    T, cu = 2500, [0, 900, 900, 2111]
    o, lse, want, n = behind(T, cu, D, paged, window, sinks)
    assert n > 0  # split
    assert bool((o[cu[-1]:] == 7).all()) and bool((lse[cu[-1]:] == 7).all())
    a, b = o[:cu[-1]].double(), want[0].double()
    assert float((a - b).norm()) <= 2.0 ** -8 * 2 * float(b.norm())
    assert float((lse[:cu[-1]] - want[1]).abs().max()) < 2.0 ** -12


def test_sequences_share_pages():
    """A page in several rows of the table, and twice in one: what copies of it give."""
    D, size, HK = 64, 16, 2
    kc, vc, q = bf(12, size, HK, D), bf(12, size, HK, D, seed=1), bf(60, 6, D, seed=2)
    shared = ints(5, 2, 9, 1, 5, 2, 7, 9, 5, 5, 5, 5).view(3, 4)
    own = torch.arange(1, 13, device="cuda").int().view(3, 4)
    k2, v2 = (torch.cat([c[:1], c[shared.flatten().long()]]) for c in (kc, vc))
    for mask in (dict(), dict(window=20, sinks=3)):
        past = ints(63, 40, 17)
        a, b = (gdn.attn_step(q[:3], *c, past, want_lse=True, **mask) for c in ((kc, vc, shared), (k2, v2, own)))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        cu, past = ints(0, 20, 40, 60), ints(44, 20, 0)
        a, b = (gdn.attn_fwd_paged(q, *c, cu, past, want_lse=True, **mask) for c in ((kc, vc, shared), (k2, v2, own)))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
