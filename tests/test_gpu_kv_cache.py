"""The paged key-value cache on the GPU: appending, one token's attention and prompts' attention over it, against the fp64 oracle.
Tolerances of the attention: see attention_bounds; of the turned rows as rotary's (half a step of the type, 2^-20 of the pair's
size for sine, cosine and products)."""
import sys

import numpy as np
import pytest
import torch

from oracle import attention as A
from tests.attention_bounds import LEAST, U, check, head_bounds
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache_of(pages, size, HK, D, dt, gen, order):
    """k and v caches [pages, size, HK, D] in three orders of memory"""
    if order == "both":  # k and v of a page side by side
        x = torch.randn(pages, 2, size, HK, D, generator=gen).to(dt).cuda()
        return x[:, 0], x[:, 1]
    if order == "heads":  # [pages, HK, size, D]
        return tuple(torch.randn(pages, HK, size, D, generator=gen).to(dt).cuda().transpose(1, 2) for _ in range(2))
    return tuple(torch.randn(pages, size, HK, D, generator=gen).to(dt).cuda() for _ in range(2))


def table_of(totals, size, gen, spare=2, drop=()):
    """(table, pages) for sequences of these many tokens, pages in no order; drop: (sequence, column) without a page"""
    need = [-(-max(t, 0) // size) for t in totals]
    order = torch.randperm(sum(need) + spare, generator=gen) + 1
    table = torch.zeros(len(totals), max(max(need), 1), dtype=torch.int32)
    at = 0
    for n, m in enumerate(need):
        table[n, :m] = order[at:at + m]
        at += m
    for n, c in drop:
        table[n, c] = [0, -3, 10 ** 6][(n + c) % 3]
    return table, sum(need) + spare + 1


def paged_bounds(q, kc, vc, table, cu, offsets, window, sinks, dtype):
    HQ, D = q.shape[1:]
    pages, size, HK = kc.shape[:3]
    bo, bl = np.zeros(q.shape), np.zeros(q.shape[:2])
    for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        j = np.arange(max(int(offsets[n]) + b - a, 0))
        at = [A.place(table[n], size, pages, x) for x in j]
        has = np.array([x is not None for x in at], bool)
        k, v = np.zeros((len(j), HK, D)), np.zeros((len(j), HK, D))
        for x, y in enumerate(at):
            if y is not None:
                k[x], v[x] = kc[y], vc[y]
        seen = A.visible(int(offsets[n]) + np.arange(b - a), j, window, sinks) & has[None]
        for h in range(HQ):
            g = h // (HQ // HK)
            bo[a:b, h], bl[a:b, h] = head_bounds(q[a:b, h], k[:, g], v[:, g], seen, D ** -0.5, dtype)
    return bo, bl


APPEND = [  # lens (None: one token each), offsets, HQ, HK, D, R, size, dtype, inter, order, padding
    (None, [0], 1, 1, 64, 64, 16, "bf16", False, "plain", 0), (None, [5, -1, 100, 31], 4, 2, 128, 32, 16, "fp16", True, "both", 8),
    ([3, 0, 70, 1], [0, 4, 1000, 15], 16, 2, 256, 64, 48, "bf16", False, "heads", 16), ([40], [7], 0, 3, 128, 0, 1, "bf16", False, "plain", 0),
    ([9, 9], [-4, 2], 3, 1, 80, 74, 17, "fp16", False, "plain", 3), ([130, 5], [1, 2], 2, 2, 66, 66, 528, "bf16", True, "heads", 1),
    ([300], [90000], 8, 8, 64, 64, 64, "bf16", False, "both", 0), ([5] * 40, list(range(40)), 1, 1, 32, 16, 4, "bf16", False, "plain", 8),
]


@pytest.mark.parametrize("lens, offsets, HQ, HK, D, R, size, dtype, inter, order, pad", APPEND)
def test_append(lens, offsets, HQ, HK, D, R, size, dtype, inter, order, pad):
    say(lens, offsets[:4], HQ, HK, D, R, size, dtype, inter, order, pad)
    gen = torch.Generator().manual_seed(D + size)
    dt = TYPES[dtype]
    ns = lens or [1] * len(offsets)
    T, cu = sum(ns), np.concatenate([[0], np.cumsum(ns)]).tolist()

    def rows(H):
        x = torch.randn(T, H * D + pad, generator=gen).to(dt).cuda()
        return x[:, :H * D].unflatten(1, (H, D))

    q, k, v = rows(HQ) if HQ else None, rows(HK), rows(HK)
    # the last page of the last sequence is none, and so is what the table has no column for
    totals = [o + n for o, n in zip(offsets, ns)]
    table, pages = table_of(totals, size, gen)
    far = [int(table.shape[1]) - 1]
    table[-1, far] = 0
    kc, vc = cache_of(pages, size, HK, D, dt, gen, order)
    keep = (f64(kc), f64(vc), [x.clone() for x in (k, v)], q.clone() if HQ else None)
    f = gdn.rotary_inv_freq(R, device="cuda")[0] if R else None
    kw = dict(cu_seqlens=ints(cu)) if lens else {}
    out = gdn.kv_append(k, v, kc, vc, table.cuda(), ints(offsets), q=q, inv_freq=f, interleaved=inter, mscale=1.25 if R else 1.0, **kw)
    freq = f64(f) if R else ()
    want = A.append(f64(k), f64(v), keep[0], keep[1], table.numpy(), offsets, cu, f64(q) if HQ else None, freq, inter, 1.25)
    assert torch.equal(k, keep[2][0]) and torch.equal(v, keep[2][1])  # inputs stay
    assert np.array_equal(f64(vc), want[2])
    # rows that were not written keep their bits; turned ones are within a rounding
    written = (want[2] != keep[1]).any((2, 3))
    got = f64(kc)
    assert np.array_equal(got[~written], keep[0][~written])
    bound = lambda x, r: U[dtype] * np.abs(r) + 2.0 ** -20 * 2.5 * 6 + LEAST[dtype]  # noqa: E731  (|x| < 6)
    assert (np.abs(got - want[1]) <= bound(k, want[1])).all()
    if not HQ:
        assert out is None
        return
    assert torch.equal(q, keep[3]) and (np.abs(f64(out) - want[0]) <= bound(q, want[0])).all()
    # in place, and the second call leaves the same cache
    before = kc.clone()
    same = gdn.kv_append(k, v, kc, vc, table.cuda(), ints(offsets), q=q, inv_freq=f, interleaved=inter, mscale=1.25 if R else 1.0, q_out=q, **kw)
    assert same is q and torch.equal(q, out) and torch.equal(kc, before)


def test_append_is_rotary_and_a_copy():
    """The rows in the cache have the bits that rotary gives."""
    gen = torch.Generator().manual_seed(4)
    T, HQ, HK, D = 50, 4, 2, 128
    x = torch.randn(T, (HQ + 2 * HK) * D, generator=gen).bfloat16().cuda()
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([HQ * D, HK * D, HK * D], 1))
    f, m = gdn.rotary_inv_freq(64, scaling="yarn", factor=4.0, original=512, device="cuda")
    kc, vc = (torch.zeros(9, 16, HK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    past = ints([30])
    out = gdn.kv_append(k, v, kc, vc, ints([[3, 1, 5, 2, 8]]), past, cu_seqlens=ints([0, T]), q=q, inv_freq=f, mscale=m)
    qr, kr = gdn.rotary(q, k, f, cu_seqlens=ints([0, T]), offsets=past, mscale=m)
    pos = torch.arange(30, 80)
    pages = torch.tensor([3, 1, 5, 2, 8])[pos // 16]
    assert torch.equal(out, qr) and torch.equal(kc[pages, pos % 16], kr) and torch.equal(vc[pages, pos % 16], v)
    assert int((vc != 0).any(-1).any(-1).sum()) == T


STEP = [  # tokens of each row's sequence with the new one (0: idle), HQ, HK, D, size, dtype, window, sinks, order
    ([1], 1, 1, 64, 16, "bf16", 0, 0, "plain"), ([1, 0, 2, 33], 4, 2, 128, 16, "fp16", 0, 0, "both"),
    ([31, 32, 33, 64, 65, 511, 512, 513], 8, 2, 256, 17, "bf16", 0, 0, "heads"), ([1500, 3], 16, 1, 64, 64, "bf16", 0, 0, "plain"),
    ([700, 0, 90], 40, 2, 64, 1, "bf16", 0, 0, "plain"), ([1200], 128, 1, 64, 528, "fp16", 0, 0, "heads"),
    ([2000, 100, 1], 6, 2, 128, 48, "bf16", 100, 4, "plain"), ([900, 901], 3, 3, 256, 32, "fp16", 1, 0, "both"),
    ([600] * 5, 24, 8, 64, 20, "bf16", 77, 300, "plain"), ([5000], 2, 1, 128, 16, "bf16", 4000, 1, "heads"),
    ([40] * 300, 2, 2, 64, 16, "bf16", 0, 0, "plain"),
]


@pytest.mark.parametrize("totals, HQ, HK, D, size, dtype, window, sinks, order", STEP)
def test_step(totals, HQ, HK, D, size, dtype, window, sinks, order):
    say(totals[:4], HQ, HK, D, size, dtype, window, sinks, order)
    gen = torch.Generator().manual_seed(D + size)
    N = len(totals)
    table, pages = table_of(totals, size, gen)
    kc, vc = cache_of(pages, size, HK, D, TYPES[dtype], gen, order)
    x = torch.randn(N, HQ * D + 8, generator=gen).to(TYPES[dtype]).cuda()
    q = x[:, :HQ * D].unflatten(1, (HQ, D))
    offsets = [t - 1 for t in totals]
    args = (f64(q), f64(kc), f64(vc), table.numpy())
    want = A.step(*args, offsets, window, sinks)
    bound = paged_bounds(*args, list(range(N + 1)), offsets, window, sinks, dtype)
    # what no row sees may hold anything: NaN in the null page and wherever no token is
    used = np.zeros((pages, size), bool)
    for n, t in enumerate(totals):
        for j in range(t):
            if window == 0 or j > t - 1 - window or j < sinks:
                used[table[n, j // size], j % size] = True
    for c in (kc, vc):
        c[torch.from_numpy(~used).cuda()] = float("nan")
    wide = torch.full((N, table.shape[1] + 3), 10 ** 8, dtype=torch.int32)  # a slice of a wider table
    wide[:, :table.shape[1]] = table
    for t in (table.cuda(), wide.cuda()[:, :table.shape[1]], wide.cuda()):
        o, lse = gdn.attn_step(q, kc, vc, t, ints(offsets), window=window, sinks=sinks, want_lse=True)
        check("o", o, want[0], bound[0])
        check("lse", lse, want[1], bound[1])
    assert torch.equal(o, gdn.attn_step(q, kc, vc, wide.cuda(), ints(offsets), window=window, sinks=sinks)[0])


PAGED = [  # new tokens, offsets, HQ, HK, D, size, dtype, window, sinks, order
    ([1], [0], 1, 1, 64, 16, "bf16", 0, 0, "plain"), ([1, 3, 0, 5], [4, 0, 9, 100], 4, 2, 128, 16, "fp16", 0, 0, "both"),
    ([64, 65, 200], [0, 63, 1], 8, 2, 256, 48, "bf16", 0, 0, "heads"), ([20, 7], [600, 0], 16, 1, 64, 17, "bf16", 0, 0, "plain"),
    ([30, 100], [-10, -200], 2, 1, 64, 16, "bf16", 0, 0, "plain"), ([130], [700], 6, 2, 128, 64, "bf16", 90, 5, "plain"),
    ([50, 60], [500, 0], 5, 5, 256, 1, "fp16", 8, 70, "plain"), ([300], [2000], 3, 1, 64, 528, "bf16", 1024, 3, "heads"),
    ([2] * 70, [33] * 70, 4, 4, 64, 32, "bf16", 0, 0, "plain"),
]


@pytest.mark.parametrize("lens, offsets, HQ, HK, D, size, dtype, window, sinks, order", PAGED)
@pytest.mark.parametrize("holes", [False, True])
def test_paged(lens, offsets, HQ, HK, D, size, dtype, window, sinks, order, holes):
    say(lens[:4], offsets[:4], HQ, HK, D, size, dtype, window, sinks, order, holes)
    gen = torch.Generator().manual_seed(D + size)
    T, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)]).tolist()
    totals = [o + n for o, n in zip(offsets, lens)]
    table, pages = table_of(totals, size, gen, drop=[(0, 0), (len(lens) - 1, max(0, -(-totals[-1] // size)) // 2)] if holes else ())
    kc, vc = cache_of(pages, size, HK, D, TYPES[dtype], gen, order)
    q = torch.randn(T, HQ, D, generator=gen).to(TYPES[dtype]).cuda()
    args = (f64(q), f64(kc), f64(vc), table.numpy())
    want = A.forward_paged(*args, cu, offsets, window, sinks)
    bound = paged_bounds(*args, cu, offsets, window, sinks, dtype)
    used = np.zeros((pages, size), bool)
    for n, t in enumerate(totals):
        for j in range(max(t, 0)):
            at = A.place(table[n].numpy(), size, pages, j)
            if at is not None:
                used[at] = True
    for c in (kc, vc):
        c[torch.from_numpy(~used).cuda()] = float("nan")
    o, lse = gdn.attn_fwd_paged(q, kc, vc, table.cuda(), ints(cu), ints(offsets), window=window, sinks=sinks, want_lse=True)
    check("o", o, want[0], bound[0])
    check("lse", lse, want[1], bound[1])


def test_one_text_in_pieces_is_the_whole_pack():
    """Append and attend a prompt in two pieces and token by token: the rows that one forward over the whole text gives."""
    gen = torch.Generator().manual_seed(8)
    lens, HQ, HK, D, size = [150, 90], 8, 2, 128, 16
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    q, k, v = (torch.randn(sum(lens), h, D, generator=gen).bfloat16().cuda() for h in (HQ, HK, HK))
    f, m = gdn.rotary_inv_freq(64, device="cuda")
    for window, sinks in ((0, 0), (40, 3)):
        qr, kr = gdn.rotary(q, k, f, cu_seqlens=ints(cu))
        whole, _ = gdn.attn_fwd(qr, kr, v, ints(cu), window=window, sinks=sinks)
        bound = None
        table, pages = table_of(lens, size, gen)
        kc, vc = cache_of(pages, size, HK, D, torch.bfloat16, gen, "plain")
        cuts = [[0, 60, 140, *range(141, 151)], [0, 33, 80, *range(81, 91)]]
        from tests.attention_bounds import pack_bounds
        args = [f64(x) for x in (qr, kr, v)]
        bound = pack_bounds(*args, cu, window, sinks, "bf16")["o"]
        want, _ = A.forward(*args, cu, window, sinks)
        check("whole", whole, want, bound)
        for i in range(len(cuts[0]) - 1):
            a, b = [c[i] for c in cuts], [c[i + 1] for c in cuts]
            at = torch.cat([torch.arange(s + x, s + y) for s, x, y in zip(cu, a, b)]).cuda()
            n = [y - x for x, y in zip(a, b)]
            past, table_d = ints(a), table.cuda()
            if max(n) == 1:
                turned = gdn.kv_append(k[at], v[at], kc, vc, table_d, past, q=q[at], inv_freq=f)
                o, _ = gdn.attn_step(turned, kc, vc, table_d, past, window=window, sinks=sinks)
            else:
                c = ints(np.concatenate([[0], np.cumsum(n)]).tolist())
                turned = gdn.kv_append(k[at], v[at], kc, vc, table_d, past, q=q[at], inv_freq=f, cu_seqlens=c)
                o, _ = gdn.attn_fwd_paged(turned, kc, vc, table_d, c, past, window=window, sinks=sinks)
            rows = at.cpu().numpy()
            check("piece", o, want[rows], bound[rows])
