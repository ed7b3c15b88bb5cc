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


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("eps", [1e-12, 1e-20, 1e-30])
@pytest.mark.parametrize("D", [64, 256, 301, 5120])
def test_rows_that_a_small_eps_lifts(dtype, eps, D):
    """Rows and groups of zeros give zeros and the least scale, tiny rows the values of their ratios."""
    print(dtype, eps, D, file=sys.stderr, flush=True)
    x = make(6, D, dtype, 3)
    x[0] = 0
    x[1], x[2] = x[1] * 2.0 ** -20, x[2] * 2.0 ** -24  # fp16's least values among them
    x[2, 128:] = 0
    x[3] = 0
    x[3, D // 2] = 2.0 ** -24
    x[4, :128] = 0
    w = make(1, D, dtype, 4)[0].contiguous()
    for weight in (None, w):
        y, _ = Y.rmsnorm(f64(x), None if weight is None else f64(weight), eps)
        for quant, group in (("row", 0), (128, 128)):
            out = gdn.rmsnorm_fwd(x, weight, quant=quant, want_y=True, eps=eps)
            within(out["y"], y)
            sc = Y.scales(y, group)
            within(out["scales"], sc)
            v = y / (np.repeat(sc, 128, 1)[:, :D] if group else sc[:, None])
            err = np.abs(f64(out["y8"].float()) - v)
            assert (err <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) * (1 + 2.0 ** -12)).all()
            assert not out["y8"][0].float().any()


@pytest.mark.parametrize("dtype", TYPES)
def test_a_row_of_zeros_without_eps_is_no_number(dtype):
    """0 / sqrt(0), in y, its scale and y8; the other rows stay."""
    x = make(3, 200, dtype, 5)
    x[1] = 0
    for quant in ("row", 128):
        out = gdn.rmsnorm_fwd(x, quant=quant, want_y=True, eps=0.0)
        for n in ("y", "scales", "y8"):
            t = out[n].float()
            assert bool(t[1].isnan().all()) and bool(t[[0, 2]].isfinite().all()), n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [1, 64, 333, 700, 4096, 16384])
def test_rows_whose_sum_of_squares_is_past_fp32(dtype, D):
    """The mean is in its range: 10^19 squared is 10^38. Rows beside them stay."""
    x = make(5, D, dtype, 8)
    want = gdn.rmsnorm_fwd(x, want_rstd=True, eps=0.0)
    x[1], x[3] = x[1].sign() * 1e19, x[3].clamp(-4, 4) * 2e18
    out = gdn.rmsnorm_fwd(x, quant=128, want_y=True, want_rstd=True, eps=0.0)
    y, rstd = Y.rmsnorm(f64(x), None, 0.0)
    within(out["y"], y)
    within(out["rstd"], rstd)
    within(out["scales"], Y.scales(y, 128))
    for i in (0, 2, 4):
        assert torch.equal(out["y"][i], want["y"][i]) and torch.equal(out["rstd"][i], want["rstd"][i])
    # the backward from it
    dy = make(5, D, dtype, 9).contiguous()
    g = gdn.rmsnorm_bwd(dy, x, None, out["rstd"])
    dx, _ = Y.rmsnorm_backward(f64(x), f64(dy), None, 0.0)
    n = np.abs(f64(x)) * rstd[:, None]
    size = rstd[:, None] * (np.abs(f64(dy)) + n * (np.abs(f64(dy)) * n).mean(1, keepdims=True))
    within(g["dx"], dx, size)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("s, w", [(1e18, 1e21), (1e18, 1e36), (1e-18, 1e-25), (2e19, 1e25)])
@pytest.mark.parametrize("D", [64, 333])
def test_large_and_small_weights(dtype, s, w, D):
    """The product with the weight passes fp32's range where y does, not where s (weight) alone would. With
    s = 2e19 the mean of squares is past fp32: rstd is zero, and so is y."""
    print(dtype, s, w, D, file=sys.stderr, flush=True)
    x, weight = (make(4, D, dtype, 6) * s).to(dtype), (make(1, D, dtype, 7)[0] * w).to(dtype)
    past = s > 1e19
    y, _ = Y.rmsnorm(f64(x), f64(weight), 0.0)
    for quant, group in (("row", 0), (128, 128)):
        out = gdn.rmsnorm_fwd(x, weight, quant=quant, want_y=True, eps=0.0)
        if past:
            assert not out["y"].any() and not out["y8"].float().any()
            continue
        within(out["y"], y)
        sc = Y.scales(y, group)
        within(out["scales"], sc)
        v = y / (np.repeat(sc, 128, 1)[:, :D] if group else sc[:, None])
        err = np.abs(f64(out["y8"].float()) - v)
        assert (err <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) * (1 + 2.0 ** -12)).all()
