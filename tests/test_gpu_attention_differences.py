"""The attention kernels' gradients against differences of the kernels' own forward. Bounds: see attention_differences."""
import pytest
import torch

from tests.attention_differences import check
from tests.gpu_helpers import f64
from tests.test_attention_differences_cpu import CASES, make

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens, HQ, HK, D, window, sinks", CASES + [([0, 70, 1, 200], 6, 2, 128, 0, 0), ([300], 8, 1, 64, 40, 5)])
def test_gradients_are_the_forwards(lens, HQ, HK, D, window, sinks, dtype):
    q, k, v, dO, cu = make(lens, HQ, HK, D, seed=1)
    to = lambda x: torch.from_numpy(x).to(dtype).cuda()  # noqa: E731
    dcu, mask = torch.tensor(cu, dtype=torch.int32, device="cuda"), dict(window=window, sinks=sinks)
    forward = lambda *x: f64(gdn.attn_fwd(*map(to, x), dcu, **mask)[0])  # noqa: E731
    o, lse = gdn.attn_fwd(to(q), to(k), to(v), dcu, want_lse=True, **mask)
    g = gdn.attn_bwd(to(q), to(k), to(v), dcu, o, lse, to(dO), **mask)
    assert check(forward, {n: f64(x) for n, x in g.items()}, q, k, v, dO, cu, window, sinks) <= 1
