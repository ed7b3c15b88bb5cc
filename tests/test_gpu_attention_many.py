"""The softmax attention and its cache with very many sequences, many tokens with one place, and fp16 gradients replayed
with other data. Tolerances: relative 2-norms, as in test_long of the attention."""
import sys

import pytest
import torch

from tests.test_gpu_attention import plain

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn


def test_millions_of_empty_sequences():
    """Tiles of keys with sinks and all tiles of keys together are more workgroups of 512 threads than one launch counts."""
    N, T, L, D = 4193600, 100000, 250, 128
    mask = dict(window=1, sinks=200)
    print(N, T, D, mask, file=sys.stderr, flush=True)
    assert ((T // 256 + N) + (T // 128 + N)) <= 1 << 23 and 2 * (T // 128 + N) * 512 > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, dO = (torch.randn(T, 1, D, generator=gen, device="cuda").bfloat16() for _ in range(4))
    lens = torch.zeros(N, dtype=torch.int64)
    full = torch.randperm(N, generator=torch.Generator().manual_seed(2))[:T // L].sort().values
    lens[full] = L
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).int()
    o, lse = gdn.attn_fwd(q, k, v, cu.cuda(), want_lse=True, **mask)
    g = gdn.attn_bwd(q, k, v, cu.cuda(), o, lse, dO, **mask)
    for n in (0, 1, T // L // 2, T // L - 2, T // L - 1):
        at = slice(n * L, n * L + L)
        ref = plain(q[at], k[at], v[at], [0, L], 1, 200, D ** -0.5, dO[at])
        for name, x in dict(g, o=o).items():
            far = float((x[at].double() - ref[name]).norm() / ref[name].norm())
            assert far <= (3 if name in ("dq", "dk") else 2) * 2.0 ** -8, (n, name, far)


@pytest.mark.parametrize("D, R", [(128, 0), (80, 74), (64, 64)])
def test_tokens_with_one_place(D, R):
    """Each element of the row is one of the tokens' (with R those that do not turn), and no other row changes."""
    N, size = 300, 16
    x = torch.arange(1, N + 1, device="cuda").bfloat16()[:, None, None].expand(N, 2, D).contiguous()
    kc, vc = (torch.zeros(4, size, 2, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, past = (torch.full(s, n, dtype=torch.int32, device="cuda") for s, n in (((N, 2), 2), ((N,), 21)))
    f = gdn.rotary_inv_freq(R, device="cuda")[0] if R else None
    gdn.kv_append(x, -x, kc, vc, table, past, inv_freq=f)
    row = (kc[2, 5, :, R:], -vc[2, 5])
    assert all(bool(torch.isin(r, x[:, 0, 0]).all()) for r in row)
    if R:
        assert bool(kc[2, 5, :, :R].isfinite().all())
    kc[2, 5], vc[2, 5] = 0, 0
    assert not kc.any() and not vc.any()


def test_appends_of_thousands_of_sequences():
    """Places of tokens among many boundaries, empty sequences and idle ones between: each row by its own indices."""
    gen = torch.Generator().manual_seed(3)
    N, size, HK, D = 9001, 8, 1, 64
    lens = torch.randint(0, 4, (N,), generator=gen) * (torch.rand(N, generator=gen) < 0.6)
    lens[-1] = 0
    past = torch.randint(-2, 20, (N,), generator=gen)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    T = int(cu[-1])
    table = torch.randperm(3 * N, generator=gen).view(N, 3) + 1
    k, v = (torch.randn(T, HK, D, generator=gen).bfloat16() for _ in range(2))
    kc, vc = (torch.zeros(3 * N + 1, size, HK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gdn.kv_append(k.cuda(), v.cuda(), kc, vc, table.int().cuda(), past.int().cuda(), cu_seqlens=cu.int().cuda())
    seq = torch.repeat_interleave(torch.arange(N), lens)
    pos = past[seq] + torch.arange(T) - cu[seq]
    put = (pos >= 0) & (pos < 3 * size)
    at = table[seq[put], pos[put] // size], pos[put] % size
    for got, x in ((kc, k), (vc, v)):
        want = torch.zeros(got.shape, dtype=torch.bfloat16)
        want[at] = x[put]
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("window, sinks", [(0, 0), (100, 3)])
def test_fp16_gradients_captured_and_replayed(window, sinks):
    """The units that score gradients are in follow the data of the replay, not of the capture."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    T, mask = 700, dict(window=window, sinks=sinks)
    q, k, v, dO = (torch.randn(T, h, 64, generator=gen, device="cuda").half() for h in (4, 2, 2, 4))
    cu = torch.tensor([0, 300, T], dtype=torch.int32, device="cuda")
    o, lse = gdn.attn_fwd(q, k, v, cu, want_lse=True, **mask)
    run = lambda: gdn.attn_bwd(q, k, v, cu, o, lse, dO, **mask)  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    whole = dO.clone()
    for size in (1, 2.0 ** -12, 2.0 ** 10, 1):
        dO.copy_(whole * size)
        g.replay()
        _ = torch.randn(300, 300, device="cuda") @ torch.randn(300, 300, device="cuda")
        torch.cuda.synchronize()
        want = run()
        assert all(torch.equal(got[n], want[n]) and bool(want[n].isfinite().all()) and bool(want[n].any()) for n in want), size
