"""The linear attention with every length of segment that packs are cut into, 256 to 4096 tokens, and packs of short
sequences that are left whole: o, hT and all gradients against the fp64 oracle, over whole sequences of sampled
heads. Their decays are none, slow (every chunk of a segment counts) and fast (the gather stops early).

The lengths follow from the extents; `saved` holds T // S + N states a head, which says what S was.

Tolerances: elementwise and, for bf16, in the 2-norm those of the linear attention's other tests. For the fp32
states in the 2-norm: a term's weight is a product of at most tokens / 64 + 4 powers of the decay, each within 2^-22
where it is not negligible (its exponent's rounding and exp2's), and it is added up in at most tokens / 16 + 64 fp32
steps of 2^-24 each; for 14443 tokens (231 x 4 + 967) 2^-24 < 2^-13, and partial sums are taken as up to twice the
last one: 2^-12."""
import sys

import numpy as np
import pytest
import torch

from oracle import linear as L
from tests.gpu_helpers import f64
from tests.test_gpu_linear import U16, U32

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn

DECAYS = [0.0, -0.5, -1e-3, -40.0, -0.02, -float("inf")]


def make(lens, H, HV, D, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    T, N = sum(lens), len(lens)
    return dict(q=r(T, H, D).bfloat16(), k=r(T, H, D).bfloat16(), v=r(T, HV, D).bfloat16(), dO=r(T, HV, D).bfloat16(),
                h0=0.3 * r(N, HV, D, D), dhT=0.3 * r(N, HV, D, D),
                log_decay=torch.tensor([DECAYS[i % len(DECAYS)] for i in range(HV)], device="cuda"),
                cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda"))


def check(x, got, h, scale, longest):
    """Key head h and its value heads."""
    G = x["v"].shape[1] // x["q"].shape[1]
    hv = slice(h * G, (h + 1) * G)
    i = {n: f64(x[n][:, h:h + 1]) for n in ("q", "k")} | {n: f64(x[n][:, hv]) for n in ("v", "dO", "h0", "dhT")}
    g, cu = f64(x["log_decay"][hv]), x["cu"].tolist()
    out = []
    for a in (lambda y: y, np.abs):
        q, k, v, dO, h0, dhT = (a(i[n]) for n in ("q", "k", "v", "dO", "h0", "dhT"))
        o, hT = L.forward(q, k, v, g, cu, h0, scale)
        out.append(dict(o=o, hT=hT, **L.backward(q, k, v, g, cu, dO, h0, dhT, scale)))
    for name, r in out[0].items():
        y, s = f64(got[name][:, h:h + 1] if name in ("dq", "dk") else got[name][:, hv]), out[1][name]
        half = got[name].dtype == torch.bfloat16
        bound = U16 * (np.abs(r) + s) * (1 + 2.0 ** -6) if half else 3 * U32 * (longest + 64) * s
        bad = np.abs(y - r) > bound + 1e-30
        assert not bad.any(), (name, h, np.argwhere(bad)[:4].tolist(), np.abs(y - r)[bad][:4], r[bad][:4])
        far, size = np.linalg.norm(y - r), np.linalg.norm(r)  # a gradient behind a decay of zero is zero
        assert far <= (U16 if half else 2.0 ** -12) * size, (name, h, far, size)


def forward_and_backward(x, scale):
    o, hT, saved = gdn.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], x["cu"], h0=x["h0"], scale=scale or 0.0,
                                  save_for_backward=True)
    return dict(o=o, hT=hT, **gdn.linear_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["cu"], saved, x["dO"], dhT=x["dhT"],
                                             scale=scale or 0.0)), saved


CASES = [  # tokens a segment, the sequences, H, HV, D, scale
    (256, [70, 933], 46, 46, 128, None), (512, [70, 1829], 24, 48, 128, 0.37), (1024, [70, 3621], 50, 50, 128, None),
    (2048, [70, 7205], 57, 114, 128, None), (4096, [70, 14373], 114, 114, 128, None),
    (256, [70, 933], 27, 54, 64, 1.5), (512, [1829], 126, 126, 64, None), (1024, [70, 5157], 44, 88, 64, None),
    (2048, [70, 7205], 128, 128, 64, None), (4096, [70, 14373], 128, 128, 64, None),
    (512, [1024, 512], 60, 60, 128, None),  # sequences that end with a segment
    (1024, [1000, 1900, 3, 1100], 16, 32, 128, None),  # cut by their mean length: most of them are one segment
    (512, [500, 900, 3, 700, 0, 600, 513, 512], 16, 16, 64, 0.2),
]


@pytest.mark.parametrize("S, lens, H, HV, D, scale", CASES)
def test_segments_match_the_oracle(S, lens, H, HV, D, scale):
    print(S, lens, H, HV, D, file=sys.stderr, flush=True)
    x = make(lens, H, HV, D, seed=S + D)
    got, saved = forward_and_backward(x, scale)
    assert saved.numel() == (sum(lens) // S + len(lens)) * HV * D * D * 4, "another length of segment: choose other extents"
    G = HV // H
    for h in (0, 1, 2, H - 1):  # G = 1: decays 0, -0.5, -1e-3; G = 2: 0 with -0.5, -1e-3 with -40, -0.02 with none
        check(x, got, h, scale, max(lens))
        print("head", h, "of", H, "group", G, file=sys.stderr, flush=True)
    # without the states: the same segments from the workspace
    o, hT, _ = gdn.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], x["cu"], h0=x["h0"], scale=scale or 0.0)
    assert torch.equal(o, got["o"]) and torch.equal(hT, got["hT"])


@pytest.mark.parametrize("scale", [0.25, 3.0])
def test_an_explicit_scale_of_pools_and_steps(scale):
    lens, H, HV, D = [150, 64, 1], 2, 4, 64
    x = make(lens, H, HV, D, seed=3)
    pool, idx = torch.randn(5, HV, D, D, device="cuda"), torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda")
    at = idx.long()
    o, hT, _ = gdn.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], x["cu"], h0=pool[at], scale=scale)
    mine = pool.clone()
    o2, _ = gdn.linear_fwd_paged(x["q"], x["k"], x["v"], x["log_decay"], x["cu"], mine, idx, scale=scale)
    assert torch.equal(o, o2) and torch.equal(mine[at], hT)
    q, k, v = (x[n][:3].contiguous() for n in ("q", "k", "v"))
    before = f64(mine)
    o = gdn.linear_step(q, k, v, x["log_decay"], mine, idx, scale=scale)
    ro, rp = L.step(f64(q), f64(k), f64(v), f64(x["log_decay"]), before, idx.tolist(), scale)
    so, sp = L.step(*(np.abs(f64(t)) for t in (q, k, v)), f64(x["log_decay"]), np.abs(before), idx.tolist(), scale)
    assert (np.abs(f64(o) - ro) <= U16 * np.abs(ro) + U32 * (D + 8) * so).all()
    assert (np.abs(f64(mine) - rp) <= 4 * U32 * sp).all()
