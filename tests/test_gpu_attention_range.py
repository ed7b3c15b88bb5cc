"""The softmax attention in fp16 where its numbers leave the middle of that type's range: small, large and unlike cotangents, and
weights far below a row's largest one. Against fp64 on the GPU.

u = 2^-11 is half a step of fp16 and 2^-25 half of its least one. A tensor is held by 2-norms, as in test_long of the attention: two
roundings of any sign, a weight's or score gradient's and the output's own, are below 2 u of its norm, dq and dk have delta's too: 3 u.
An output below fp16's normal numbers is off by at most 2^-25 besides, each element of it. The score gradients and the weights have
full precision over fp16's normal numbers, down to 2^-21 of the largest of a step, and lie by at most 2^-32 of that off below:
n keys or rows of equal size together n 2^-32, which is below u / 2^9 for the lengths here."""
import sys

import numpy as np
import pytest
import torch

from oracle import attention as A
from tests.attention_bounds import score_error
from tests.gpu_helpers import f64
from tests.test_gpu_attention import plain

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn

U, LEAST = 2.0 ** -11, 2.0 ** -25
FACTOR = dict(o=2, dv=2, dq=3, dk=3)


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def make(lens, HQ, HK, D, seed):
    gen = torch.Generator().manual_seed(seed)
    T, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)]).tolist()
    r = lambda h: torch.randn(T, h, D, generator=gen).cuda()  # noqa: E731
    return r(HQ), r(HK), r(HK), r(HQ), cu, torch.tensor(cu, dtype=torch.int32, device="cuda")


def gradients(q, k, v, dO, cu, dcu, window=0, sinks=0):
    """(the kernels' outputs, the reference's)"""
    o, lse = gdn.attn_fwd(q, k, v, dcu, window=window, sinks=sinks, want_lse=True)
    got = dict(gdn.attn_bwd(q, k, v, dcu, o, lse, dO, window=window, sinks=sinks), o=o)
    return got, plain(q, k, v, cu, window, sinks, q.shape[2] ** -0.5, dO)


def near(name, got, want, factor=None):
    off = float((got.double() - want).norm())
    bound = (factor or FACTOR[name]) * U * float(want.norm()) + LEAST * want.numel() ** 0.5
    say(name, off / float(want.norm()), bound / float(want.norm()))
    assert off <= bound, name  # also where it is NaN


CASES = [  # lens, HQ, HK, D, window, sinks
    ([2100, 300], 4, 2, 64, 0, 0), ([2100], 4, 1, 128, 0, 0), ([1500, 7], 2, 2, 256, 0, 0), ([2500], 4, 2, 128, 300, 5),
    ([3000, 2], 2, 1, 64, 200, 70), ([2000], 2, 1, 256, 500, 3), ([40] * 70, 3, 1, 64, 0, 0),
]


@pytest.mark.parametrize("size", [1.0, 0.1, 0.01, 0.001])
@pytest.mark.parametrize("lens, HQ, HK, D, window, sinks", CASES)
def test_small_cotangents(lens, HQ, HK, D, window, sinks, size):
    say(lens[:4], HQ, HK, D, window, sinks, size)
    q, k, v, dO, cu, dcu = make(lens, HQ, HK, D, D)
    q, k, v, dO = q.half(), k.half(), v.half(), (dO * size).half()
    got, want = gradients(q, k, v, dO, cu, dcu, window, sinks)
    for n in ("dq", "dk", "dv"):
        near(n, got[n], want[n])


@pytest.mark.parametrize("D, window, sinks", [(64, 0, 0), (128, 0, 0), (256, 0, 0), (128, 50, 3)])
def test_large_cotangents(D, window, sinks):
    """Score gradients past fp16's largest number whose products with q and k are not."""
    say(D, window, sinks)
    q, k, v, dO, cu, dcu = make([200, 31], 4, 2, D, D)
    q, k, v, dO = (q * 2.0 ** -9).half(), (k * 2.0 ** -9).half(), (v * 64).half(), (dO * 2.0 ** 13).half()
    got, want = gradients(q, k, v, dO, cu, dcu, window, sinks)
    # the weight of a row's own key is near 1 / (row + 1): the scores are near 0
    own = v.double().repeat_interleave(2, 1) - want["o"]
    ds = (own * dO.double()).sum(-1)[:30] * D ** -0.5 / torch.arange(1, 31, device="cuda")[:, None]
    assert float(ds.abs().max()) > 70000
    for n in ("dq", "dk"):
        near(n, got[n], want[n])


SIZES = [10, 1e-4, 1, 1e-3, 100, 1e-2, 1e-4, 10, 1e-3]


@pytest.mark.parametrize("HQ, HK, D, window, sinks", [(2, 1, 64, 0, 0), (2, 2, 128, 0, 0), (2, 1, 256, 0, 0), (2, 1, 64, 200, 4), (4, 1, 128, 150, 3),
                                                      (2, 1, 256, 100, 0)])
def test_unlike_cotangents(HQ, HK, D, window, sinks):
    """A cotangent whose size changes by up to 2^20 from one 128 tokens to the next: each 128 tokens' gradients have their own
    precision, small ones beside large ones too."""
    say(HQ, HK, D, window, sinks)
    q, k, v, dO, cu, dcu = make([128 * len(SIZES)], HQ, HK, D, D + HQ)
    size = torch.tensor(SIZES, device="cuda").repeat_interleave(128)[:, None, None]
    q, k, v, dO = q.half(), k.half(), v.half(), (dO * size).half()
    got, want = gradients(q, k, v, dO, cu, dcu, window, sinks)
    for n in ("dq", "dk"):
        for i in range(0, len(q), 128):
            near(n, got[n][i:i + 128], want[n][i:i + 128])


def with_sink(lens, HQ, HK, D, seed, gap=15.0):
    """The first key of each sequence takes nearly all weight, e^gap of another's, and has no value: the others' weights, some
    2^-22, are the outputs."""
    q, k, v, dO, cu, dcu = make(lens, HQ, HK, D, seed)
    q, k = q * 0.3, k * 0.3
    q[..., 0], k[..., 0] = 8, 0
    k[cu[:-1]] = 0
    k[cu[:-1], :, 0] = gap / 8 * D ** 0.5
    v = v * 16
    v[cu[:-1]] = 0
    return q.half(), k.half(), v.half(), (dO * 64).half(), cu, dcu


@pytest.mark.parametrize("lens, HQ, HK, D, window, sinks", [([1500, 200], 4, 2, 64, 0, 0), ([1500], 2, 1, 128, 0, 0), ([1200], 2, 2, 256, 0, 0),
                                                            ([1500], 4, 1, 128, 300, 1), ([2000, 900], 2, 1, 64, 700, 5)])
def test_small_weights_in_dv(lens, HQ, HK, D, window, sinks):
    say(lens, HQ, HK, D, window, sinks)
    q, k, v, dO, cu, dcu = with_sink(lens, HQ, HK, D, D)
    got, want = gradients(q, k, v, dO, cu, dcu, window, sinks)
    others = torch.ones(len(v), dtype=torch.bool)
    others[cu[:-1]] = False
    near("dv", got["dv"][others], want["dv"][others])


@pytest.mark.parametrize("lens, HQ, HK, D, window, sinks", [([1500, 200], 4, 2, 64, 0, 0), ([1500], 2, 1, 128, 0, 0), ([1200], 2, 2, 256, 0, 0),
                                                            ([1500], 4, 1, 128, 300, 1), ([3000], 1, 1, 64, 0, 0)])
def test_small_weights(lens, HQ, HK, D, window, sinks):
    """o element by element: a weight and its product with v are off by u + e (e: its score's and the exponentials', as in
    attention_bounds) and, below fp16's normal numbers, by 2^-25 where the row's largest weight is 2^7 at least; then o's own
    rounding."""
    say(lens, HQ, HK, D, window, sinks)
    q, k, v, dO, cu, dcu = with_sink(lens, HQ, HK, D, D + 1)
    got, want = gradients(q, k, v, dO, cu, dcu, window, sinks)
    close(got["o"], want["o"], bounds(f64(q), f64(k), f64(v), cu, window, sinks, cu))
    for n in ("o", "dq", "dk"):
        near(n, got[n], want[n])


def bounds(q, k, v, cu, window, sinks, kcu, past=None):
    out = np.zeros(q.shape)
    for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        first, last = kcu[n], kcu[n + 1]
        seen = A.visible((0 if past is None else past[n]) + np.arange(b - a), np.arange(last - first), window, sinks)
        for h in range(q.shape[1]):
            g, D = h // (q.shape[1] // k.shape[1]), q.shape[2]
            x, y, z = q[a:b, h], k[first:last, g], v[first:last, g]
            o, _, w = A.head(x, y, z, seen, D ** -0.5)
            e = 2 * score_error(x, y, seen, D ** -0.5) + 2.0 ** -18
            out[a:b, h] = (U + e) * (w @ np.abs(z)) + 2.0 ** -32 * (seen @ np.abs(z)) + U * np.abs(o) + LEAST
    return out


def close(got, want, bound):
    got, want = f64(got), f64(want)
    assert np.isfinite(got).all() and (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


@pytest.mark.parametrize("totals, HQ, HK, D, window, sinks", [([1500, 30, 700], 4, 2, 64, 0, 0), ([6000], 2, 1, 128, 0, 0), ([900, 901], 16, 2, 256, 0, 0),
                                                              ([1500, 2000], 4, 1, 128, 300, 1)])
def test_small_weights_in_a_cache(totals, HQ, HK, D, window, sinks):
    """One token's step and a prompt's last tokens over a cache."""
    say(totals, HQ, HK, D, window, sinks)
    q, k, v, _, cu, dcu = with_sink(totals, HQ, HK, D, D + 2)
    size, N = 16, len(totals)
    cols = [-(-t // size) for t in totals]
    table = torch.zeros(N, max(cols), dtype=torch.int32)
    for n, c in enumerate(cols):
        table[n, :c] = torch.arange(c) + 1 + sum(cols[:n])
    kc, vc = (torch.zeros(sum(cols) + 1, size, HK, D, dtype=torch.float16, device="cuda") for _ in range(2))
    zero = torch.zeros(N, dtype=torch.int32, device="cuda")
    gdn.kv_append(k, v, kc, vc, table.cuda(), zero, cu_seqlens=dcu)
    exact = A.forward(f64(q), f64(k), f64(v), cu, window, sinks)[0]
    for new in (1, 20):
        rows = np.concatenate([np.arange(b - new, b) for b in cu[1:]])
        past = [t - new for t in totals]
        args = (q[torch.from_numpy(rows).cuda()], kc, vc, table.cuda())
        p = torch.tensor(past, dtype=torch.int32, device="cuda")
        few = (np.arange(N + 1) * new).tolist()
        bound = bounds(f64(args[0]), f64(k), f64(v), few, window, sinks, cu, past)
        if new == 1:
            close(gdn.attn_step(*args, p, window=window, sinks=sinks)[0], torch.from_numpy(exact[rows]), bound)
        close(gdn.attn_fwd_paged(*args, torch.tensor(few, dtype=torch.int32, device="cuda"), p, window=window, sinks=sinks)[0],
              torch.from_numpy(exact[rows]), bound)
