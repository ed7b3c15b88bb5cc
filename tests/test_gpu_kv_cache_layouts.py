"""Caches in the orders of memory that the binding takes, and what it refuses, and rows of outputs that no sequence holds."""
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
