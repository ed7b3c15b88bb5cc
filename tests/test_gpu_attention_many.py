"""The softmax attention at the most sequences that a problem may have. Tolerances: relative 2-norms, as in test_long of the attention."""
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
