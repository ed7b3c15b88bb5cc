"""The attention and the cache as programs call them: in a captured graph, on other streams, two calls at once, on memory given
back while a stream is busy, over caches and packs past 32 bits, with many sequences, and chained with rotary positions and
the norm in a layer's forward and backward."""
import sys

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import layer as Y
from tests.attention_bounds import check, pack_bounds
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn

HQ, HK, D, SIZE = 8, 2, 128, 16


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def bf(*shape, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=gen, device="cuda").bfloat16()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def calls(T=700, seed=0):
    """name -> (function without arguments, what it changes in place)"""
    q, k, v, dO = bf(T, HQ, D, seed=seed), bf(T, HK, D, seed=seed + 1), bf(T, HK, D, seed=seed + 2), bf(T, HQ, D, seed=seed + 3)
    cu = ints(0, 130, T)
    kc, vc = bf(120, SIZE, HK, D, seed=seed + 4), bf(120, SIZE, HK, D, seed=seed + 5)
    table = torch.randperm(119, generator=torch.Generator().manual_seed(seed))[:110].int().add(1).view(2, 55).cuda()
    past, long, short = ints(200, 40), ints(800, 611), ints(3, -1)
    f = gdn.rotary_inv_freq(64, device="cuda")[0]
    o, lse = gdn.attn_fwd(q, k, v, cu, window=300, sinks=4, want_lse=True)
    one = dict(q=q[:2], k_cache=kc, v_cache=vc, page_table=table)
    return dict(
        append=lambda **s: (gdn.kv_append(k, v, kc, vc, table, past, cu_seqlens=cu, q=q, inv_freq=f, **s), kc, vc),
        append_tokens=lambda **s: (gdn.kv_append(k[:2], v[:2], kc, vc, table, past, **s), kc, vc),
        step=lambda **s: gdn.attn_step(offsets=long, want_lse=True, **one, **s),
        step_short=lambda **s: gdn.attn_step(offsets=short, window=3, sinks=1, **one, **s),
        paged=lambda **s: gdn.attn_fwd_paged(q, kc, vc, table, cu, past, want_lse=True, **s),
        fwd=lambda **s: gdn.attn_fwd(q, k, v, cu, window=300, sinks=4, want_lse=True, **s),
        bwd=lambda **s: tuple(gdn.attn_bwd(q, k, v, cu, o, lse, dO, window=300, sinks=4, **s).values()),
        bwd_whole=lambda **s: tuple(gdn.attn_bwd(q, k, v, cu, o, lse, dO, **s).values()))


NAMES = ["append", "append_tokens", "step", "step_short", "paged", "fwd", "bwd", "bwd_whole"]


def same(a, b):
    return all((x is None and y is None) or torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def kept(r):
    return [None if x is None else x.clone() for x in r]


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    call = calls()[name]
    want = kept(call())
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    for i in range(4):
        for x in got:
            if x is not None and i < 2 and not name.startswith("append"):
                x.fill_(3)
        g.replay()
        _ = bf(300, 300, seed=i) @ bf(300, 300)  # the program's own work between replays
        torch.cuda.synchronize()
        assert same(got, want), i


@pytest.mark.parametrize("name", NAMES)
def test_other_streams_and_two_at_once(name):
    a, b = calls(seed=1)[name], calls(seed=50)[name]
    want = [kept(a()), kept(b())]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [x(stream=s) for x, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        assert all(same(x, y) for x, y in zip(got, want))
    with torch.cuda.stream(streams[0]):
        got = a()
    torch.cuda.synchronize()
    assert same(got, want[0])
    got = b(stream=streams[1].cuda_stream)  # a raw handle
    torch.cuda.synchronize()
    assert same(got, want[1])


@pytest.mark.parametrize("name", ["fwd", "bwd", "paged", "step", "append"])
def test_memory_follows_the_stream(name):
    """Inputs that the caller lets go of while the given stream is busy are not handed out before it is through."""
    def inputs():
        q, k, v, dO, cu = bf(700, HQ, D), bf(700, HK, D, seed=1), bf(700, HK, D, seed=2), bf(700, HQ, D, seed=3), ints(0, 700)
        kc, vc, table = bf(60, SIZE, HK, D, seed=4), bf(60, SIZE, HK, D, seed=5), torch.arange(1, 50, device="cuda").int()[None]
        if name == "fwd":
            return gdn.attn_fwd, dict(q=q, k=k, v=v, cu_seqlens=cu)
        if name == "bwd":
            o, lse = gdn.attn_fwd(q, k, v, cu, want_lse=True)
            return gdn.attn_bwd, dict(q=q, k=k, v=v, cu_seqlens=cu, o=o, lse=lse, dO=dO)
        pages = dict(k_cache=kc, v_cache=vc, page_table=table)
        if name == "paged":
            return gdn.attn_fwd_paged, dict(q=q, cu_seqlens=cu, offsets=ints(20), **pages)
        if name == "step":
            return gdn.attn_step, dict(q=q[:1].clone(), offsets=ints(719), **pages)
        return gdn.kv_append, dict(k=k, v=v, q=q, cu_seqlens=cu, offsets=ints(20), inv_freq=gdn.rotary_inv_freq(64, device="cuda")[0],
                                   **pages)

    def values(r):
        return [r] if isinstance(r, torch.Tensor) else list(r.values()) if isinstance(r, dict) else [x for x in r if x is not None]

    call, kw = inputs()
    want = kept(values(call(**kw)))
    s = torch.cuda.Stream()
    call, kw = inputs()
    keep = [kw.get("k_cache"), kw.get("v_cache")] if name == "append" else []
    torch.cuda.synchronize()
    sizes = {t.numel() * t.element_size() for t in kw.values()}
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    got = values(call(**kw, stream=s))
    del kw
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]
    torch.cuda.synchronize()
    assert same(got, want)
    del junk, keep


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements, pages near its end."""
    pages = (1 << 32) // (SIZE * HK * D) + 40
    kc, vc = (torch.empty(pages, SIZE, HK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    T, last = 100, pages - 10
    table = torch.arange(last, last + 8, device="cuda").int()[None]
    q, k, v = bf(T, HQ, D), bf(T, HK, D, seed=1), bf(T, HK, D, seed=2)
    kc[last:], vc[last:] = float("nan"), float("nan")
    gdn.kv_append(k, v, kc, vc, table, ints(0), cu_seqlens=ints(0, T))
    assert torch.equal(kc[last:last + 8].flatten(0, 1)[:T], k) and torch.equal(vc[last:last + 8].flatten(0, 1)[:T], v)
    o, _ = gdn.attn_fwd_paged(q, kc, vc, table, ints(0, T), ints(0))
    want, _ = gdn.attn_fwd(q, k, v, ints(0, T))
    bound = pack_bounds(f64(q), f64(k), f64(v), [0, T], 0, 0, "bf16")["o"]
    exact, _ = A.forward(f64(q), f64(k), f64(v), [0, T])
    check("paged", o, exact, bound)
    check("pack", want, exact, bound)
    one, _ = gdn.attn_step(q[-1:], kc, vc, table, ints(T - 1))
    check("step", one, exact[-1:], bound[-1:])


def test_rows_past_32_bits():
    """Token rows at a stride whose offsets pass 2^31 elements."""
    T, wide = 600, 1 << 22
    x = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")
    q, k, v = (x[:, i * 4096:i * 4096 + h * D].unflatten(1, (h, D)) for i, h in enumerate((HQ, HK, HK)))
    q.copy_(bf(T, HQ, D)), k.copy_(bf(T, HK, D, seed=1)), v.copy_(bf(T, HK, D, seed=2))
    dO, cu = bf(T, HQ, D, seed=3), ints(0, 50, T)
    dense = [t.contiguous() for t in (q, k, v)]
    a, la = gdn.attn_fwd(q, k, v, cu, want_lse=True)
    b, lb = gdn.attn_fwd(*dense, cu, want_lse=True)
    assert torch.equal(a, b) and torch.equal(la, lb)
    ga, gb = gdn.attn_bwd(q, k, v, cu, a, la, dO), gdn.attn_bwd(*dense, cu, b, lb, dO)
    assert all(torch.equal(ga[n], gb[n]) for n in ga)


@pytest.mark.parametrize("n, window, sinks", [(65, 0, 0), (100, 20, 2), (300, 5, 130)])
def test_many_sequences(n, window, sinks):
    """More than a wave has lanes: the tiles are then found by the boundaries."""
    say(n, window, sinks)
    r = np.random.default_rng(n)
    lens = r.integers(0, 40, n).tolist()
    lens[3], lens[-1] = 200, 0
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    T = cu[-1]
    q, k, v, dO = bf(T, 4, 64), bf(T, 2, 64, seed=1), bf(T, 2, 64, seed=2), bf(T, 4, 64, seed=3)
    o, lse = gdn.attn_fwd(q, k, v, ints(*cu), window=window, sinks=sinks, want_lse=True)
    g = gdn.attn_bwd(q, k, v, ints(*cu), o, lse, dO, window=window, sinks=sinks)
    args = [f64(x) for x in (q, k, v)]
    bound = pack_bounds(*args, cu, window, sinks, "bf16", f64(dO))
    want, want_lse = A.forward(*args, cu, window, sinks)
    ref = A.backward(*args, cu, f64(dO), window, sinks)
    check("o", o, want, bound["o"])
    check("lse", lse, want_lse, bound["lse"])
    for name in g:
        check(name, g[name], ref[name], bound[name], "bf16")


def test_far_and_negative_offsets():
    """Positions past the table and below zero, to the ends of 32 bits."""
    far, low = [(1 << 31) - 300, 1 << 30, 900], [-(1 << 31), -(1 << 30), -60]
    q, k, v = bf(150, 4, 64), bf(150, 2, 64, seed=1), bf(150, 2, 64, seed=2)
    kc, vc = bf(60, SIZE, 2, 64, seed=3), bf(60, SIZE, 2, 64, seed=4)
    table = torch.arange(1, 31, device="cuda").int().expand(3, 30).contiguous()  # 480 positions
    cu, one = ints(0, 50, 100, 150), dict(page_table=table, want_lse=True)
    for mask in (dict(), dict(window=100, sinks=3)):
        was = kc.clone(), vc.clone()
        for past in (far, low):
            gdn.kv_append(k, v, kc, vc, table, ints(*past), cu_seqlens=cu)
            gdn.kv_append(k[:3], v[:3], kc, vc, table, ints(*past))
        assert torch.equal(kc, was[0]) and torch.equal(vc, was[1])
        rows = torch.cat([q[:50]] * 3)
        o, lse = gdn.attn_fwd_paged(rows, kc, vc, cu_seqlens=cu, offsets=ints(*far), **one, **mask)
        for n in (0, 1):
            assert torch.equal(o[50 * n:50 * n + 50], o[100:]) and torch.equal(lse[50 * n:50 * n + 50], lse[100:])
        assert bool(lse.isfinite().all())
        s, ls = gdn.attn_step(torch.cat([q[:1]] * 3), kc, vc, offsets=ints(*far), **one, **mask)
        assert torch.equal(s[0], s[2]) and torch.equal(s[1], s[2]) and torch.equal(ls[0], ls[2]) and bool(ls.isfinite().all())
        o, lse = gdn.attn_fwd_paged(rows, kc, vc, cu_seqlens=cu, offsets=ints(*low), **one, **mask)
        s, ls = gdn.attn_step(q[:3], kc, vc, offsets=ints(*low), **one, **mask)
        assert not o.any() and not s.any() and bool((lse == -torch.inf).all()) and bool((ls == -torch.inf).all())


@pytest.mark.parametrize("size", [16, 17])
@pytest.mark.parametrize("D, window, sinks", [(64, 100, 3), (128, 33, 0), (256, 7, 70)])
def test_pages_behind_the_window_hold_anything(size, D, window, sinks):
    past, lens, cu = [900, 40], [30, 300], ints(0, 30, 330)
    q, cols = bf(330, 4, D), -(-930 // size)
    kc, vc = bf(2 * cols + 1, size, 2, D, seed=1), bf(2 * cols + 1, size, 2, D, seed=2)
    table = (torch.randperm(2 * cols, generator=torch.Generator().manual_seed(size)) + 1).int().view(2, cols).cuda()
    args = dict(page_table=table, cu_seqlens=cu, offsets=ints(*past), window=window, sinks=sinks, want_lse=True)
    want = gdn.attn_fwd_paged(q, kc, vc, **args)
    one = dict(page_table=table, offsets=ints(930, 340), window=window, sinks=sinks, want_lse=True)
    step = gdn.attn_step(q[:2], kc, vc, **one)
    kn, vn = torch.full_like(kc, torch.nan), torch.full_like(vc, torch.inf)
    for n, (p, t) in enumerate(zip(past, lens)):
        j = torch.tensor([j for j in range(p + t + 1) if j < sinks or j > p - window], device="cuda")
        at = table[n, j // size].long(), j % size
        kn[at], vn[at] = kc[at], vc[at]
    assert same(gdn.attn_fwd_paged(q, kn, vn, **args), want)
    assert same(gdn.attn_step(q[:2], kn, vn, **one), step)


def test_sinks_beyond_every_sequence():
    """All keys are sinks: what no window gives, also where the sequences' tiles are far fewer than sinks would be."""
    r = np.random.default_rng(1)
    lens = r.integers(0, 6, 1000).tolist()
    lens[500], lens[20] = 700, 131
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    T = cu[-1]
    q, k, v, dO = bf(T, 2, 64), bf(T, 1, 64, seed=1), bf(T, 1, 64, seed=2), bf(T, 2, 64, seed=3)
    mask = dict(window=3, sinks=1 << 30)
    o, lse = gdn.attn_fwd(q, k, v, ints(*cu), want_lse=True, **mask)
    g = gdn.attn_bwd(q, k, v, ints(*cu), o, lse, dO, **mask)
    args = [f64(x) for x in (q, k, v)]
    bound = pack_bounds(*args, cu, 0, 0, "bf16", f64(dO))
    ref = A.backward(*args, cu, f64(dO))
    check("o", o, A.forward(*args, cu)[0], bound["o"])
    for name in g:
        check(name, g[name], ref[name], bound[name], "bf16")


@pytest.mark.parametrize("HQ, HK, D, window", [(4, 2, 64, 0), (4, 1, 128, 9), (2, 1, 256, 0)])
def test_gradients_against_differences(HQ, HK, D, window):
    """The kernels' gradients against differences of the kernels' own forward, along random directions: the loss sum(o dO) is
    summed in 64 bits from bf16 outputs. An output is off by at most 2 u of its largest value's size (a weight's and its own
    rounding), of any sign, so a difference over 2 h is off by about 2 u |dO| sqrt(rows) / h; h is a step that moves scores
    by about 1/8, where the third derivative's share, h^2 / 6 of the gradient's size, is below that."""
    T, u, h = 40, 2.0 ** -8, 0.125
    q, k, v, dO = bf(T, HQ, D), bf(T, HK, D, seed=1), bf(T, HK, D, seed=2), bf(T, HQ, D, seed=3)
    cu = ints(0, 25, T)
    o, lse = gdn.attn_fwd(q, k, v, cu, window=window, want_lse=True)
    g = gdn.attn_bwd(q, k, v, cu, o, lse, dO, window=window)

    def loss(x):
        return float((gdn.attn_fwd(*x, cu, window=window)[0].double() * dO.double()).sum())

    for i, name in enumerate(("dq", "dk", "dv")):
        d = bf(*(q, k, v)[i].shape, seed=7 + i)
        up, down = ([t if j != i else (t.float() + s * h * d.float()).bfloat16() for j, t in enumerate((q, k, v))] for s in (1, -1))
        moved = (up[i].double() - down[i].double()) / (2 * h)  # what the rounded inputs moved by
        want = float((g[name].double() * moved).sum())
        size = float((g[name].double().norm() * moved.norm()))
        noise = 2 * u * float(dO.double().norm()) * float(o.abs().max()) / (2 * h) * 2
        assert abs((loss(up) - loss(down)) / (2 * h) - want) <= noise + size * (h ** 2 / 6 + 2 * u), name


def test_layer_forward_and_backward():
    """rotary -> attention -> norm over heads, and back: each operator's backward fed by the next one's, against the oracles'
    chain from the tensors that each operator was given. Relative 2-norms, a rounding below 2^-8 of a tensor's norm: the norm's
    dx carries one, the attention's weights or score gradients, delta and output three more, the turn back a fifth."""
    gen = torch.Generator().manual_seed(5)
    cu = [0, 65, 105]
    r = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()  # noqa: E731
    q, k, v, w, dy = r(105, 4, 64), r(105, 2, 64), r(105, 2, 64), r(64), r(420, 64)
    f, m = gdn.rotary_inv_freq(32, scaling="yarn", factor=4.0, original=64, device="cuda")
    turn = dict(cu_seqlens=ints(*cu), mscale=m)
    mask = dict(window=30, sinks=2)
    qr, kr = gdn.rotary(q, k, f, **turn)
    o, lse = gdn.attn_fwd(qr, kr, v, ints(*cu), want_lse=True, **mask)
    n = gdn.rmsnorm_fwd(o.view(-1, 64), w, want_rstd=True)
    gn = gdn.rmsnorm_bwd(dy, o.view(-1, 64), w, n["rstd"])
    g = gdn.attn_bwd(qr, kr, v, ints(*cu), o, lse, gn["dx"].view(o.shape), **mask)
    dq, dk = gdn.rotary_bwd(g["dq"], g["dk"], f, **turn)
    dx, _ = Y.rmsnorm_backward(f64(o).reshape(-1, 64), f64(dy), f64(w))
    ref = A.backward(f64(qr), f64(kr), f64(v), cu, dx.reshape(o.shape), **mask)
    pos = Y.positions(cu)
    near = lambda a, b, c: np.linalg.norm(f64(a).ravel() - b.ravel()) <= c * 2.0 ** -8 * np.linalg.norm(b)  # noqa: E731
    assert near(g["dv"], ref["dv"], 3)
    for a, name in ((dq, "dq"), (dk, "dk")):
        assert near(a, Y.rotary(ref[name], pos, f64(f), False, m, back=True), 5)


def test_the_binding_refuses():
    q, k, cu = bf(10, 4, 64), bf(10, 2, 64), ints(0, 10)
    kc = bf(5, SIZE, 2, 64)
    t, off = ints(1, 2)[None], ints(0)
    ok = lambda **over: gdn.attn_step(**dict(dict(q=q[:1], k_cache=kc, v_cache=kc.clone(), page_table=t, offsets=off), **over))  # noqa: E731
    ok()
    for bad in (dict(k_cache=kc.half()), dict(v_cache=kc.float())):
        with pytest.raises(TypeError):
            ok(**bad)
    for bad in (dict(k_cache=kc[..., :32]), dict(k_cache=kc[:, :, :1]), dict(v_cache=kc[:4]), dict(v_cache=kc.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(page_table=t[0]), dict(page_table=t.long()), dict(page_table=t.expand(2, 2)), dict(page_table=t.cpu()),
                dict(offsets=ints(0, 1)), dict(k_cache=kc.cpu())):
        with pytest.raises((ValueError, TypeError)):
            ok(**bad)
    with pytest.raises(gdn.GdnError, match="UNSUPPORTED"):
        gdn.attn_fwd(bf(10, 3, 64), k, k, cu)
    with pytest.raises(gdn.GdnError, match="SEQLENS"):
        gdn.attn_fwd(q, k, k, cu, cu_seqlens_host=torch.tensor([0, 9], dtype=torch.int32))
    for f in (lambda: gdn.attn_fwd(q, k, k[:5], cu), lambda: gdn.attn_fwd(q, k, bf(10, 4, 64), cu), lambda: gdn.attn_fwd(q, k, k, cu.long()),
              lambda: gdn.attn_fwd(q.float(), k.float(), k.float(), cu), lambda: gdn.attn_fwd(q, k.half(), k.half(), cu),
              lambda: gdn.attn_bwd(q, k, k, cu, q, torch.zeros(10, 4), q), lambda: gdn.attn_fwd(q, k, k, cu, stream=object()),
              lambda: gdn.kv_append(k, k, kc, kc, t, off, q=q[:5], cu_seqlens=cu),
              lambda: gdn.kv_append(k, k[:3], kc, kc, t, off, cu_seqlens=cu),
              lambda: gdn.kv_append(k, k, kc, kc, t, off, q=q, q_out=q[:, :2], cu_seqlens=cu)):
        with pytest.raises((ValueError, TypeError)):
            f()
