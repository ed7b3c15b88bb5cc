"""Rotary positions of more tokens than one launch takes: 2^24 workgroups of 256 threads, one for each token,
are 2^32 threads, which a launch does not count. The rows are those of calls on parts of them, and the last ones
those of the fp64 oracle."""
import pytest
import torch

from oracle import layer as Y
from tests.gpu_helpers import f64
from tests.test_gpu_rotary import close

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn


@pytest.mark.parametrize("by_sequence", [False, True])
def test_more_tokens_than_a_launch_of_one_token_a_workgroup(by_sequence):
    T, H, D = 2 ** 24 + 5, 65, 2  # 65 units a token: more than a workgroup shares among tokens
    gen = torch.Generator(device="cuda").manual_seed(9)
    q = torch.randn(T, H, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    f = torch.full((1,), 0.37, device="cuda")
    bounds, past = [0, 2 ** 23 - 3, T - 70, T], [5, 0, 2 ** 20]
    pos = torch.cat([torch.arange(b - a, dtype=torch.int32, device="cuda") + o
                     for a, b, o in zip(bounds[:-1], bounds[1:], past)])
    if by_sequence:
        cu, off = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (bounds, past))
        out, _ = gdn.rotary(q, None, f, cu_seqlens=cu, offsets=off)
    else:
        out, _ = gdn.rotary(q, None, f, positions=pos)
    step = 2 ** 22
    for t in range(0, T, step):
        part, _ = gdn.rotary(q[t:t + step], None, f, positions=pos[t:t + step])
        assert torch.equal(out[t:t + step], part), t
    for t in (2 ** 23 - 9, 2 ** 24 - 9, T - 9):
        x = f64(q[t:t + 9])
        close(out[t:t + 9], x, Y.rotary(x, f64(pos[t:t + 9]), f64(f), False), 1.0)
