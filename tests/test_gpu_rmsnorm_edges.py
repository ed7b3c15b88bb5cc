"""The norm's e4m3 output where the weight or eps takes it to fp32's edges, against the fp64 oracle; the tolerances
are those of the norm's other tests."""
import sys

import numpy as np
import pytest
import torch

from oracle import layer as Y
from tests.gpu_helpers import f64
from tests.test_gpu_rmsnorm import make, within

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn

TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, D", [(3, 100), (2, 256), (3, 515), (2, 5120)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_weight_that_is_no_number_is_in_its_scale(rows, D, dtype, bad):
    """The largest |y| of a group with a NaN is NaN, and so are the group's scale and what is divided by it; with an
    infinity the scale is infinite. The other groups' scales and values stay."""
    print(rows, D, dtype, bad, file=sys.stderr, flush=True)
    x, w = make(rows, D, dtype, 1), make(1, D, dtype, 2)[0].contiguous()
    spoilt = w.clone()
    at = D - 2
    spoilt[at] = bad
    for quant in ("row", 128):
        want, got = (gdn.rmsnorm_fwd(x, t, quant=quant) for t in (w, spoilt))
        first = 0 if quant == "row" else at // 128 * 128
        scales = got["scales"] if quant == "row" else got["scales"][:, at // 128]
        y8 = got["y8"].float()
        if bad != bad:
            assert bool(scales.isnan().all()) and bool(y8[:, first:].isnan().all())
        else:
            assert bool((scales == bad).all()) and bool(y8[:, at].isnan().all())
            assert not y8[:, first:at].any() and not y8[:, at + 1:].any()
        assert torch.equal(got["y8"][:, :first].view(torch.uint8), want["y8"][:, :first].view(torch.uint8))
        if quant == 128:
            assert torch.equal(got["scales"][:, :at // 128], want["scales"][:, :at // 128])
