"""Rotary positions on the GPU against the fp64 oracle.

Tolerance: an output is a cos - b sin in fp32, rounded once: half a step of its type relative to the value
(bf16 2^-8, fp16 2^-11, fp32 2^-24), and before that 2^-20 of mscale (|a| + |b|) for the sine and cosine (a few
fp32 steps of an angle held to less than one fp32 step of a turn), their products and the sum. fp16's least
steps (2^-25) add to that."""
import sys

import numpy as np
import pytest
import torch

from oracle import layer as Y
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def close(got, x, ref, mscale):
    size = np.abs(x).max(-1, keepdims=True) * 2 * mscale
    bound = HALF[got.dtype] * np.abs(ref) + 2.0 ** -20 * size + (2.0 ** -25 if got.dtype == torch.float16 else 0)
    err = np.abs(f64(got) - ref)
    assert (err <= bound).all(), (err.max(), (err / bound).max())


def rows(T, heads, D, dtype, gen, pad):
    """A tensor [T, heads, D]: of its own, or a slice of wider rows."""
    x = torch.randn(T, heads * D + pad, generator=gen).to(dtype).cuda()
    return x[:, :heads * D].unflatten(1, (heads, D))


CASES = [  # lens, HQ, HK, D, R, dtype, padding of the rows
    ([1], 1, 1, 64, 64, torch.bfloat16, 0), ([3, 0, 70, 1], 4, 2, 128, 128, torch.bfloat16, 16),
    ([5] * 100, 3, 1, 80, 74, torch.float16, 3), ([130, 7], 16, 2, 256, 64, torch.float32, 0),
    ([33], 5, 0, 96, 32, torch.float16, 8), ([17], 2, 2, 6, 2, torch.float32, 1), ([9, 9], 1, 3, 1024, 1024, torch.bfloat16, 0),
    ([4100, 900], 2, 1, 64, 48, torch.bfloat16, 8), ([2500, 0, 1, 2000], 1, 1, 66, 66, torch.float32, 0),
]


@pytest.mark.parametrize("lens, HQ, HK, D, R, dtype, pad", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_matches_the_oracle(lens, HQ, HK, D, R, dtype, pad, interleaved):
    print(lens[:4], HQ, HK, D, R, dtype, interleaved, file=sys.stderr, flush=True)
    gen = torch.Generator().manual_seed(len(lens) + D)
    T = sum(lens)
    q = rows(T, HQ, D, dtype, gen, pad)
    k = rows(T, HK, D, dtype, gen, pad) if HK else None
    f, m = gdn.rotary_inv_freq(R, scaling="yarn", factor=4.0, original=512, device="cuda")
    cu = np.concatenate([[0], np.cumsum(lens)])
    past = torch.randint(0, 2000000, (len(lens),), generator=gen, dtype=torch.int32)
    how = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), offsets=past.cuda(), interleaved=interleaved, mscale=m)
    pos = Y.positions(cu.tolist(), past.tolist())
    for call, back in ((gdn.rotary, False), (gdn.rotary_bwd, True)):
        q0, k0 = q.clone(), k.clone() if HK else None
        qo, ko = call(q, k, f, **how)
        for x, y in ((q, qo), (k, ko)):
            if x is not None:
                close(y, f64(x), Y.rotary(f64(x), pos, f64(f), interleaved, m, back), m)
                assert torch.equal(y[..., R:], x[..., R:])
        assert torch.equal(q, q0) and (k is None or torch.equal(k, k0))
        # given positions, and in place
        given = dict(positions=torch.tensor(pos, dtype=torch.int32, device="cuda"), interleaved=interleaved, mscale=m)
        q2, k2 = call(q, k, f, **given)
        assert torch.equal(q2, qo) and (k is None or torch.equal(k2, ko))
        out = dict(q_out=q, k_out=k) if not back else dict(dq=q, dk=k)
        call(q, k, f, **given, **out)
        assert torch.equal(q, qo) and (k is None or torch.equal(k, ko))
        q.copy_(q0)
        if HK:
            k.copy_(k0)


def test_wide_and_narrow_paths_agree():
    gen = torch.Generator().manual_seed(1)
    f = gdn.rotary_inv_freq(64, device="cuda")[0]
    pos = torch.arange(40, dtype=torch.int32, device="cuda") * 1000
    for interleaved in (False, True):
        x = rows(40, 3, 64, torch.bfloat16, gen, 8)
        odd = torch.empty(40, 3 * 64 + 1, dtype=torch.bfloat16, device="cuda")[:, 1:].unflatten(1, (3, 64))
        odd.copy_(x)
        a, _ = gdn.rotary(x, None, f, positions=pos, interleaved=interleaved)
        b, _ = gdn.rotary(odd, None, f, positions=pos, interleaved=interleaved)
        assert torch.equal(a, b)


def test_rows_of_no_sequence_stay_and_infinities_keep_to_their_pair():
    f = gdn.rotary_inv_freq(8, device="cuda")[0]
    x = torch.randn(10, 2, 16, device="cuda")
    x[3, 1, 2] = float("nan")
    cu = torch.tensor([0, 4, 7], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 9.0)
    gdn.rotary(x, None, f, cu_seqlens=cu, q_out=out)
    assert bool((out[7:] == 9).all())
    bad = out.isnan().nonzero().tolist()
    assert bad == [[3, 1, 2], [3, 1, 6]]


def test_another_stream_and_a_captured_graph():
    gen = torch.Generator().manual_seed(2)
    q, k = rows(300, 4, 64, torch.bfloat16, gen, 0), rows(300, 2, 64, torch.bfloat16, gen, 0)
    f = gdn.rotary_inv_freq(32, device="cuda")[0]
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    want = gdn.rotary(q, k, f, cu_seqlens=cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = gdn.rotary(q, k, f, cu_seqlens=cu, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = gdn.rotary(q, k, f, cu_seqlens=cu)
    for _ in range(3):
        got[0].zero_(), got[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_the_binding_refuses_what_does_not_fit():
    q, k = torch.zeros(6, 2, 64, device="cuda"), torch.zeros(6, 1, 64, device="cuda")
    f, pos = torch.zeros(16, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    bad = [
        (ValueError, lambda: gdn.rotary(q, k, f)),
        (ValueError, lambda: gdn.rotary(q, k[:5], f, positions=pos)),
        (ValueError, lambda: gdn.rotary(q, k, f, positions=pos[:5])),
        (TypeError, lambda: gdn.rotary(q, k, f, positions=pos.long())),
        (TypeError, lambda: gdn.rotary(q, k.half(), f, positions=pos)),
        (TypeError, lambda: gdn.rotary(q.double(), k.double(), f, positions=pos)),
        (ValueError, lambda: gdn.rotary(q, k, f.cpu(), positions=pos)),
        (TypeError, lambda: gdn.rotary(q, k, f.half(), positions=pos)),
        (ValueError, lambda: gdn.rotary(q, k, f, cu_seqlens=cu, offsets=pos)),
        (ValueError, lambda: gdn.rotary(q, k, f, positions=pos, q_out=q[:3])),
        (ValueError, lambda: gdn.rotary(q.transpose(0, 1).contiguous().transpose(0, 1), k, f, positions=pos)),
        (gdn.GdnError, lambda: gdn.rotary(q, k, torch.zeros(33, device="cuda"), positions=pos)),
        (gdn.GdnError, lambda: gdn.rotary(q, k, f, cu_seqlens=cu, cu_seqlens_host=torch.tensor([0, 5], dtype=torch.int32))),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()


def test_many_sequences():
    lens = [0, 3] + [1, 0] * 2600 + [30, 0]
    gen = torch.Generator().manual_seed(3)
    q = rows(sum(lens), 1, 16, torch.float32, gen, 0)
    f = gdn.rotary_inv_freq(16, device="cuda")[0]
    cu = np.concatenate([[0], np.cumsum(lens)])
    past = torch.randint(0, 5000, (len(lens),), generator=gen, dtype=torch.int32)
    out, none = gdn.rotary(q, None, f, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), offsets=past.cuda())
    pos = Y.positions(cu.tolist(), past.tolist())
    close(out, f64(q), Y.rotary(f64(q), pos, f64(f), False), 1.0)
    assert none is None
    empty, _ = gdn.rotary(q[:0], None, f, positions=torch.empty(0, dtype=torch.int32, device="cuda"))
    assert empty.shape == (0, 1, 16)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("D,R", [(90, 90), (65, 30), (11, 10), (3, 2), (40, 18), (257, 34)])
def test_odd_heads_in_place_end_where_they_end(D, R, dtype, interleaved):
    """The last piece of an odd head: in place as out of place, and nothing between the rows is written."""
    T, H = 19, 3
    gen = torch.Generator().manual_seed(D)
    f = gdn.rotary_inv_freq(R, device="cuda")[0]
    pos = torch.randint(0, 4000, (T,), generator=gen, dtype=torch.int32).cuda()
    x = rows(T, H, D, dtype, gen, 0)
    want, _ = gdn.rotary(x, None, f, positions=pos, interleaved=interleaved)
    close(want, f64(x), Y.rotary(f64(x), pos.cpu().numpy(), f64(f), interleaved), 1.0)
    for pad in (1, 5):
        buf = torch.full((T, H * D + pad), 7.0, dtype=dtype, device="cuda")
        a = buf[:, :H * D].unflatten(1, (H, D))
        a.copy_(x)
        gdn.rotary(a, None, f, positions=pos, q_out=a, interleaved=interleaved)
        assert torch.equal(a, want) and bool((buf[:, H * D:] == 7).all())


def test_rows_past_32_bits():
    T, H, D = 2 ** 20 + 3, 16, 128
    gen = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randn(T, H, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    assert q.numel() > 2 ** 31
    f = gdn.rotary_inv_freq(D, device="cuda")[0]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    out, _ = gdn.rotary(q, None, f, positions=pos)
    last, _ = gdn.rotary(q[-50:].contiguous(), None, f, positions=pos[-50:].contiguous())
    assert torch.equal(out[-50:], last)
