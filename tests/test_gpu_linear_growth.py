"""The linear attention's heads that grow (log_decay above 0), as far as e^(log_decay length) is in fp32's range.
Elementwise bounds of the linear attention's other tests; an fp32 power e^x with x up to 80 carries the
rounding of x besides, 2^-24 of it three times over (its factor, the product with log2 e, the product with the
tokens)."""
import sys

import numpy as np
import pytest
import torch

from tests.gpu_helpers import f64
from tests.test_gpu_linear import U16, U32, inputs, refs, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens, grow", [([1, 3, 2, 40, 17], [1.9, 1.45]), ([1], [60.0, 79.0]), ([7, 0, 55], [1.42, 0.5]),
                                        ([64, 70, 1], [1.1, -0.3]), ([400], [0.19, 0.02])])
@pytest.mark.parametrize("H", [2, 1])
@pytest.mark.parametrize("D", [64, 128])
def test_growth_in_short_sequences(lens, grow, H, D):
    print(lens, grow, H, D, file=sys.stderr, flush=True)
    x = inputs(lens, H, 2, D, seed=sum(lens), decay=grow)
    got, ref, size = run(x), refs(x), refs(x, absolute=True)
    for name, y in got.items():
        y, r, s = f64(y), ref[name], size[name]
        bound = 3 * U32 * (max(lens) + 64 + 80) * s
        if got[name].dtype == torch.bfloat16:
            bound = U16 * (np.abs(r) + s) * (1 + 2.0 ** -6)
        assert np.isfinite(y).all() and (np.abs(y - r) <= bound).all(), name
