"""Gradients of the softmax attention where rows see few keys: dO . v - delta cancels there, so delta has to be more exact than a
rounded o gives it. Against fp64 on the GPU."""
import sys

import numpy as np
import pytest
import torch

from tests.test_gpu_attention import plain

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def gradients(lens, HQ, HK, D, dtype, window=0, sinks=0, seed=0):
    print(lens[:4], len(lens), HQ, HK, D, dtype, window, sinks, file=sys.stderr, flush=True)
    gen = torch.Generator().manual_seed(seed + D)
    T, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)]).tolist()
    q, k, v, dO = (torch.randn(T, h, D, generator=gen).to(dtype).cuda() for h in (HQ, HK, HK, HQ))
    dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, lse = gdn.attn_fwd(q, k, v, dcu, window=window, sinks=sinks, want_lse=True)
    g = gdn.attn_bwd(q, k, v, dcu, o, lse, dO, window=window, sinks=sinks)
    return q, k, v, dO, cu, g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens, HQ, HK, D, window", [([1] * 70, 4, 2, 64, 0), ([200, 3], 4, 1, 128, 1), ([90, 1], 2, 2, 256, 1)])
def test_one_key_has_no_gradient(lens, HQ, HK, D, window, dtype):
    """A weight of 1 whatever q and k are: dq = dk = 0. The weight is 1 up to e = 2 D 2^-24 scale |q| |k| + 2^-18 (its score twice, the
    exponential and lse, as in attention_bounds), and so is delta's share of it: a score's gradient is below 2 e scale |dO| |v|."""
    q, k, v, dO, cu, g = gradients(lens, HQ, HK, D, dtype, window)
    q, k, v, dO = (x.double().norm(dim=2) for x in (q, k, v, dO))
    k, v = (x.repeat_interleave(HQ // HK, 1) for x in (k, v))
    scale = D ** -0.5
    ds = 2 * (2 * D * 2.0 ** -24 * scale * q * k + 2.0 ** -18) * scale * dO * v
    assert bool((g["dq"].double().norm(dim=2) <= ds * k).all())
    assert bool((g["dk"].double().norm(dim=2) <= (ds * q).unflatten(1, (HK, -1)).sum(2)).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens, HQ, HK, D, window, sinks", [
    ([2] * 300, 4, 2, 64, 0, 0), ([3] * 200, 4, 1, 128, 0, 0), ([2] * 150, 2, 2, 256, 0, 0), ([3, 2, 1, 0] * 70, 8, 1, 64, 0, 0),
    ([300, 64], 4, 2, 64, 2, 0), ([300, 64], 4, 2, 128, 2, 1), ([150, 300], 3, 1, 256, 3, 0), ([700], 1, 1, 64, 20, 4),
])
def test_few_keys(lens, HQ, HK, D, window, sinks, dtype):
    """By 2-norms: a score gradient's rounding and the output's own, each at most u of a value, of any sign and evenly spread, so u /
    sqrt(3) of a tensor's norm, and sqrt(2 / 3) u both; a tenth of that for all sums in fp32."""
    q, k, v, dO, cu, g = gradients(lens, HQ, HK, D, dtype, window, sinks, seed=1)
    ref = plain(q, k, v, cu, window, sinks, D ** -0.5, dO)
    for n in ("dq", "dk"):
        off = float((g[n].double() - ref[n]).norm() / ref[n].norm())
        print(n, off / U[dtype], file=sys.stderr, flush=True)
        assert off <= 1.1 * (2 / 3) ** 0.5 * U[dtype], (n, off / U[dtype])
