"""The linear attention with a decay for each head on the GPU against the fp64 oracle.

Tolerances. A bf16 output carries its own rounding (2^-8 of the value at most) and one inner rounding
of the same size: of the carried state, or of a (q . k) with its decay, where they meet the other
operand. So elementwise |error| <= 2^-8 (|value| + the same sum over absolute values), and over a
whole output, where the inner errors have independent signs and each rounding's mean square is a third
of its greatest, the relative 2-norm is below sqrt(2 / 3) 2^-8 < 2^-8; a gradient summed over G value
heads has G inner roundings of its G parts, which is no more in proportion. fp32 outputs are sums of fp32
products: 2^-24 of the sum over absolute values for each of the (tokens + 64) additions and roundings on
the longest path, three products for each token.
"""
import sys

import numpy as np
import pytest
import torch

from oracle import linear as L
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn

U16, U32 = 2.0 ** -8, 2.0 ** -24


def inputs(lens, H, HV, D, seed=0, h0=True, decay=None, fused=False):
    gen = torch.Generator().manual_seed(seed)
    T, n = sum(lens), len(lens)
    rows = torch.randn(T, (2 * H + HV) * D + 8, generator=gen).to(torch.bfloat16)
    q, k, v, _ = rows.split([H * D, H * D, HV * D, 8], 1)
    q, k, v = (x.unflatten(1, (-1, D)) for x in (q, k, v))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    g = -torch.exp(torch.empty(HV).uniform_(-6.0, 0.5, generator=gen)) if decay is None else torch.tensor(decay)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    return dict(q=q, k=k, v=v, log_decay=g, cu=cu,
                h0=0.3 * torch.randn(n, HV, D, D, generator=gen) if h0 else None,
                dO=torch.randn(T, HV, D, generator=gen).to(torch.bfloat16),
                dhT=0.3 * torch.randn(n, HV, D, D, generator=gen))


def dev(x):
    if x["q"].is_contiguous() or x["q"].shape[0] == 0:
        return {k: v.cuda() if v is not None else None for k, v in x.items()}
    rows = x["q"]._base.cuda()  # the slices again, of the buffer on the GPU
    at = {k: torch.as_strided(rows, x[k].shape, x[k].stride(), x[k].storage_offset()) for k in ("q", "k", "v")}
    return {k: at.get(k, v.cuda() if v is not None else None) for k, v in x.items()}


def run(x, d=None, **how):
    d = dev(x) if d is None else d
    o, hT, saved = gdn.linear_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["cu"], h0=d["h0"], cu_seqlens_host=x["cu"],
                                  save_for_backward=True, **how)
    g = gdn.linear_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["cu"], saved, d["dO"], dhT=d["dhT"],
                       cu_seqlens_host=x["cu"], **how)
    return dict(o=o, hT=hT, **g)


def refs(x, absolute=False):
    a = np.abs if absolute else (lambda y: y)
    i = {k: a(f64(x[k])) if x[k] is not None else None for k in ("q", "k", "v", "h0", "dO", "dhT")}
    cu, g = x["cu"].tolist(), f64(x["log_decay"])
    o, hT = L.forward(i["q"], i["k"], i["v"], g, cu, i["h0"])
    return dict(o=o, hT=hT, **L.backward(i["q"], i["k"], i["v"], g, cu, i["dO"], i["h0"], i["dhT"]))


def check(got, x, names=("o", "hT", "dq", "dk", "dv", "dh0")):
    ref, size = refs(x), refs(x, absolute=True)
    longest = int(x["cu"].diff().max()) if x["cu"].numel() > 1 else 0
    for name in names:
        y, r, s = f64(got[name]), ref[name], size[name]
        if got[name].dtype == torch.bfloat16:
            bound = U16 * (np.abs(r) + s) * (1 + 2.0 ** -6)  # second-order terms of the two roundings
            if r.size >= 4096:
                assert np.linalg.norm(y - r) <= U16 * np.linalg.norm(r), name
        else:
            bound = 3 * U32 * (longest + 64) * s
        bad = np.abs(y - r) > bound + 1e-30
        assert not bad.any(), (name, np.argwhere(bad)[:4].tolist(), np.abs(y - r)[bad][:4], r[bad][:4])


SHAPES = [  # lens, H, HV, D
    ([1], 1, 1, 128), ([1], 1, 1, 64), ([64], 1, 1, 128), ([64], 1, 1, 64),
    ([63, 65, 0, 1, 128, 130], 2, 4, 128), ([0, 0, 7, 0, 200, 0], 3, 3, 64), ([33, 31, 2], 1, 5, 128),
    ([17, 449], 2, 6, 64), ([700], 1, 2, 128), ([5] * 70, 1, 1, 64), ([1] * 130 + [64, 3], 1, 1, 64),
]


@pytest.mark.parametrize("lens, H, HV, D", SHAPES)
def test_forward_and_backward_match_the_oracle(lens, H, HV, D):
    print(len(lens), sum(lens), H, HV, D, file=sys.stderr, flush=True)
    for h0, fused in ((True, False), (False, True)):
        x = inputs(lens, H, HV, D, seed=len(lens) + D, h0=h0, fused=fused)
        check(run(x), x)


@pytest.mark.parametrize("decay", [[0.0, -1e-4], [-60.0, -0.5], [-float("inf"), -200.0], [0.01, -1e30]])
def test_extreme_decays(decay):
    x = inputs([130, 5, 64, 1], 1, 2, 64, seed=3, decay=decay)
    check(run(x), x)


# long enough for every cut into segments, with sequences that end beside a segment's end
@pytest.mark.parametrize("lens, H, HV, D", [([4200], 1, 1, 64), ([2047, 2049, 1, 0, 513], 1, 2, 64), ([3100], 1, 2, 128)])
def test_long_sequences(lens, H, HV, D):
    print(lens, H, HV, D, file=sys.stderr, flush=True)
    x = inputs(lens, H, HV, D, seed=7)
    check(run(x), x)


def test_full_step_on_sampled_heads_and_its_bits_repeat():
    lens, H, HV, D = [8192, 8191], 16, 32, 128
    x = inputs(lens, H, HV, D, seed=11)
    d = dev(x)
    got = run(x, d)
    again = run(x, d)
    for name in got:
        assert torch.equal(got[name], again[name]), name
    t0, t1 = 8192, 8192 + 700  # a prefix of the second sequence: its outputs are the prefix's own
    h = 5
    hv = slice(2 * h, 2 * h + 2)
    cut = dict(q=x["q"][t0:t1, h:h + 1], k=x["k"][t0:t1, h:h + 1], v=x["v"][t0:t1, hv], log_decay=x["log_decay"][hv],
               cu=torch.tensor([0, 700]), h0=x["h0"][1:, hv], dO=x["dO"][t0:t1, hv], dhT=x["dhT"][1:, hv])
    check(dict(o=got["o"][t0:t1, hv]), cut, names=("o",))
    t0 = t0 + 8191 - 700  # a suffix of it, for what comes from the end: dv and dk do not see the earlier tokens
    cut = {k: (x[k][t0:, h:h + 1] if k in "qk" else x[k][t0:, hv]) for k in ("q", "k", "v", "dO")}
    cut |= dict(log_decay=x["log_decay"][hv], cu=torch.tensor([0, 700]), h0=None, dhT=x["dhT"][1:, hv])
    check(dict(dv=got["dv"][t0:, hv], dk=got["dk"][t0:, h:h + 1]), cut, names=("dv", "dk"))


@pytest.mark.parametrize("D, lens", [(128, [70, 1, 0, 200]), (64, [64, 65, 3, 0]), (64, [3000, 1, 1, 1500])])
def test_paged_equals_gathered(D, lens):
    H, HV, slots = 2, 4, 9
    x = inputs(lens, H, HV, D, seed=4)
    d = dev(x)
    gen = torch.Generator().manual_seed(1)
    pool = torch.randn(slots, HV, D, D, generator=gen).cuda()
    idx = torch.tensor([3, 0, 7, 5], dtype=torch.int32)
    init = torch.tensor([1, 1, 0, 0], dtype=torch.int32)
    for flags in (init, None):
        h0 = pool[idx.long()] * ((init if flags is not None else torch.ones(4)).cuda() != 0)[:, None, None, None]
        h0[1] = 0
        o, hT, saved = gdn.linear_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["cu"], h0=h0, save_for_backward=True)
        mine = pool.clone()
        o2, saved2 = gdn.linear_fwd_paged(d["q"], d["k"], d["v"], d["log_decay"], d["cu"], mine, idx.cuda(),
                                          None if flags is None else flags.cuda(), indices_host=idx,
                                          save_for_backward=True)
        want = pool.clone()
        want[idx[[0, 2, 3]].long()] = hT[[0, 2, 3]]
        assert torch.equal(o, o2) and torch.equal(mine, want)
        a, b = (gdn.linear_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["cu"], s, d["dO"]) for s in (saved, saved2))
        assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("D, H, HV, N", [(128, 2, 4, 12), (64, 3, 3, 5), (128, 1, 1, 1), (64, 1, 8, 33)])
def test_step(D, H, HV, N):
    x = inputs([N], H, HV, D, seed=N, fused=True)
    d = dev(x)
    slots = N + 4
    gen = torch.Generator().manual_seed(N)
    pool = torch.randn(slots, HV, D, D, generator=gen)
    idx = (torch.randperm(slots - 1, generator=gen)[:N] + 1).to(torch.int32)
    if N > 4:
        idx[1], idx[3] = 0, -5
    mine, before = pool.cuda(), pool.clone()
    o = gdn.linear_step(d["q"], d["k"], d["v"], d["log_decay"], mine, idx.cuda(), indices_host=idx)
    args = [f64(x[n]) for n in ("q", "k", "v", "log_decay")]
    ro, rp = L.step(*args, f64(pool), idx.tolist())
    so, sp = L.step(*[np.abs(a) if i < 3 else a for i, a in enumerate(args)], np.abs(f64(pool)), idx.tolist())
    # one rounding to bf16 after a sum of D products in fp32; a state value is two products and a sum
    assert (np.abs(f64(o) - ro) <= U16 * np.abs(ro) + U32 * (D + 8) * so).all()
    assert (np.abs(f64(mine) - rp) <= 4 * U32 * sp).all()
    rest = sorted(set(range(slots)) - {i for i in idx.tolist() if i > 0})
    assert torch.equal(mine.cpu()[rest], before[rest])
    # past the pool on the device: no state, a zero row, nothing written
    far = idx.clone()
    far[0] = slots + 100
    mine2 = pool.cuda()
    o = gdn.linear_step(d["q"], d["k"], d["v"], d["log_decay"], mine2, far.cuda())
    assert not o[0].any() and torch.equal(mine2[int(idx[0])].cpu(), before[int(idx[0])])


def test_prefill_then_steps_are_one_long_forward():
    D, H, HV, n = 128, 2, 4, 77
    x = inputs([n + 40], H, HV, D, seed=9, h0=False)
    d = dev(x)
    whole, hT, _ = gdn.linear_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["cu"])
    pool, idx = torch.full((3, HV, D, D), float("nan"), device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda")
    cu, fresh = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    o, _ = gdn.linear_fwd_paged(d["q"][:n], d["k"][:n], d["v"][:n], d["log_decay"], cu, pool, idx, fresh)
    outs = [o] + [gdn.linear_step(d["q"][t:t + 1], d["k"][t:t + 1], d["v"][t:t + 1], d["log_decay"], pool, idx)
                  for t in range(n, n + 40)]
    check(dict(o=torch.cat(outs), hT=pool[2:]), x, names=("o", "hT"))
    assert torch.equal(whole[:n], o)


def test_rows_behind_the_last_sequence_stay():
    x = inputs([70, 20], 1, 2, 64, seed=5)
    d = dev(x)
    short = torch.tensor([0, 50, 66], dtype=torch.int32, device="cuda")  # 24 of the 90 rows belong to nobody
    p = gdn.make_linear_problem(2, 90, 1, 2, 64, short)
    o = torch.full((90, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(gdn.gdn_linear_fwd_workspace_size(p), 16), dtype=torch.uint8, device="cuda")
    import ctypes
    st = gdn._lib.gdn_linear_fwd(ctypes.byref(p), d["q"].data_ptr(), d["k"].data_ptr(), d["v"].data_ptr(),
                                 d["log_decay"].data_ptr(), None, o.data_ptr(), None, None, ws.data_ptr(), ws.numel(),
                                 torch.cuda.current_stream().cuda_stream)
    assert st == 0
    want, _, _ = gdn.linear_fwd(d["q"][:66], d["k"][:66], d["v"][:66], d["log_decay"], short)
    assert torch.equal(o[:66], want) and bool((o[66:] == 7.0).all())


@pytest.mark.parametrize("H", [2, 1])
@pytest.mark.parametrize("lens", [[50, 16], [700, 3]])
def test_gradients_of_rows_behind_the_last_sequence_stay(lens, H):
    import ctypes
    used, T = sum(lens), sum(lens) + 24
    x = inputs(lens[:1] + [lens[1] + 24], H, 2, 64, seed=9)
    d = dev(x)
    cu = torch.tensor([0, lens[0], used], dtype=torch.int32, device="cuda")  # the last 24 rows belong to nobody
    p = gdn.make_linear_problem(2, T, H, 2, 64, cu)
    s = torch.cuda.current_stream().cuda_stream
    saved, ws = (torch.full((n + 16,), 255, dtype=torch.uint8, device="cuda")  # NaN as fp32
                 for n in (gdn.gdn_linear_saved_size(p), gdn.gdn_linear_bwd_workspace_size(p)))
    o = torch.empty_like(d["v"])
    ptrs = [ctypes.byref(p)] + [d[n].data_ptr() for n in ("q", "k", "v", "log_decay")]
    assert gdn._lib.gdn_linear_fwd(*ptrs, None, o.data_ptr(), None, saved.data_ptr(), ws.data_ptr(), ws.numel(), s) == 0
    dq, dk, dv = (torch.full_like(d[n], 7.0) for n in ("q", "k", "v"))
    assert gdn._lib.gdn_linear_bwd(*ptrs, saved.data_ptr(), d["dO"].data_ptr(), None, dq.data_ptr(), dk.data_ptr(),
                                   dv.data_ptr(), None, ws.data_ptr(), ws.numel(), s) == 0
    q, k, v, dO = (d[n][:used] for n in ("q", "k", "v", "dO"))
    _, _, saved = gdn.linear_fwd(q, k, v, d["log_decay"], cu, save_for_backward=True)
    want = gdn.linear_bwd(q, k, v, d["log_decay"], cu, saved, dO)
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(got[:used], want[name]) and bool((got[used:] == 7.0).all()), name


def test_two_streams_at_once():
    xs = [inputs([500, 64, 1, 3000], 2, 4, 64, seed=s) for s in (10, 11)]
    ds = [dev(x) for x in xs]
    want = [run(x, d) for x, d in zip(xs, ds)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [run(x, d, stream=s) for x, d, s in zip(xs, ds, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(g[n], w[n]) for n in w)


def test_nothing_leaks_between_sequences():
    x = inputs([70, 64, 70], 1, 1, 64, seed=6)
    d = dev(x)
    a = run(x, d)
    for name in ("q", "k", "v", "dO"):
        d[name] = d[name].clone()
        d[name][70:134] = float("nan")
    d["h0"][1], d["dhT"][1] = float("inf"), float("nan")
    b = run(x, d)
    for name in a:
        x0, x1 = (a[name], b[name])
        keep = [0, 2] if name in ("hT", "dh0") else list(range(70)) + list(range(134, 204))
        assert torch.equal(x0[keep], x1[keep]), name


def test_another_stream_and_a_captured_graph():
    x = inputs([300, 64, 1], 2, 2, 64, seed=8)
    d = dev(x)
    want = run(x, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(x, d, stream=s)
    s.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    got = run(x, d, stream=s.cuda_stream)
    s.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(x, d)
    for _ in range(3):
        for n in out:
            out[n].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in want)
        run(x, d)
        torch.cuda.synchronize()


def test_the_binding_refuses_what_does_not_fit():
    x = inputs([10, 6], 2, 4, 64)
    d = dev(x)
    q, k, v, g, cu = (d[n] for n in ("q", "k", "v", "log_decay", "cu"))
    pool, idx = torch.zeros(4, 4, 64, 64, device="cuda"), torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    saved = gdn.linear_fwd(q, k, v, g, cu, save_for_backward=True)[2]
    bad = [
        (TypeError, lambda: gdn.linear_fwd(q.float(), k, v, g, cu)),
        (ValueError, lambda: gdn.linear_fwd(q, k[:5], v, g, cu)),
        (ValueError, lambda: gdn.linear_fwd(q, k, v[:, :, :32], g, cu)),
        (ValueError, lambda: gdn.linear_fwd(q, k, v, g[:2], cu)),
        (ValueError, lambda: gdn.linear_fwd(q[:1].expand(16, 2, 64), k, v, g, cu)),
        (ValueError, lambda: gdn.linear_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, g, cu)),
        (ValueError, lambda: gdn.linear_fwd(q, k, v, g, cu.cpu())),
        (TypeError, lambda: gdn.linear_fwd(q, k, v, g, cu.long())),
        (ValueError, lambda: gdn.linear_fwd(q, k, v, g, cu, h0=pool[:1])),
        (ValueError, lambda: gdn.linear_fwd(q, k, v, g, cu, h0=pool[:2].cpu())),
        (gdn.GdnError, lambda: gdn.linear_fwd(q, k, v, g, cu, cu_seqlens_host=torch.tensor([0, 9, 15], dtype=torch.int32))),
        (ValueError, lambda: gdn.linear_fwd(q, k, v, g, cu, cu_seqlens_host=torch.tensor([0, 16], dtype=torch.int32))),
        (ValueError, lambda: gdn.linear_bwd(q, k, v, g, cu, saved[:-4], d["dO"])),
        (ValueError, lambda: gdn.linear_bwd(q, k, v, g, cu, saved, d["dO"][:, :2])),
        (ValueError, lambda: gdn.linear_fwd_paged(q, k, v, g, cu, pool[:, :2], idx)),
        (ValueError, lambda: gdn.linear_fwd_paged(q, k, v, g, cu, pool, idx[:1])),
        (gdn.GdnError, lambda: gdn.linear_fwd_paged(q, k, v, g, cu, pool, idx, indices_host=torch.tensor([1, 1], dtype=torch.int32))),
        (ValueError, lambda: gdn.linear_step(q, k, v, g, pool, idx)),
        (gdn.GdnError, lambda: gdn.linear_step(q[:2], k[:2], v[:2], g, pool, idx, indices_host=torch.tensor([1, 4], dtype=torch.int32))),
        (gdn.GdnError, lambda: gdn.linear_fwd(*(torch.zeros(3, 1, 32, dtype=torch.bfloat16, device="cuda"),) * 3, g[:1], cu)),
    ]
    for i, (error, f) in enumerate(bad):
        with pytest.raises(error):
            f()
            print("accepted", i)
    assert not pool.any()


def test_the_host_boundaries_change_no_bit():
    """They only spare launches where no sequence is cut."""
    for lens in ([256, 200, 1], [700, 3, 257]):
        x = inputs(lens, 2, 2, 64, seed=12)
        d = dev(x)
        want = run(x, d)
        o, hT, saved = gdn.linear_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["cu"], h0=d["h0"], save_for_backward=True)
        g = gdn.linear_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["cu"], saved, d["dO"], dhT=d["dhT"])
        o2, hT2, _ = gdn.linear_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["cu"], h0=d["h0"])
        o3, none, _ = gdn.linear_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["cu"], h0=d["h0"], output_final_state=False)
        g2 = gdn.linear_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["cu"], saved, d["dO"], dhT=d["dhT"], want_dh0=False)
        assert all(torch.equal(want[n], y) for n, y in dict(o=o, hT=hT, **g).items())
        assert torch.equal(o2, o) and torch.equal(hT2, hT) and torch.equal(o3, o) and none is None
        assert all(torch.equal(g2[n], g[n]) for n in ("dq", "dk", "dv")) and g2["dh0"] is None


def test_no_tokens_and_no_sequences():
    for lens in ([0, 0], []):
        x = inputs(lens, 2, 4, 128, seed=1)
        got = run(x)
        assert torch.equal(got["hT"].cpu(), x["h0"]) and torch.equal(got["dh0"].cpu(), x["dhT"])
        assert all(got[n].shape[0] == 0 for n in ("o", "dq", "dk", "dv"))
    o = gdn.linear_step(*(torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda"),) * 3, torch.zeros(2, device="cuda"),
                        torch.zeros(3, 2, 64, 64, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"))
    assert o.shape == (0, 2, 64)


def test_many_sequences():
    """More sequences than one wave's probes of the boundaries, and than their square; the first, the last and empty ones."""
    lens = [0, 3] + [1, 0] * 2600 + [300, 0, 0]
    x = inputs(lens, 1, 1, 64, seed=2)
    got = run(x)
    keep = {k: x[k][-320:] for k in ("q", "k", "v", "dO")} | dict(
        log_decay=x["log_decay"], cu=torch.tensor([0] + list(range(1, 21)) + [320], dtype=torch.int32),
        h0=torch.cat([x["h0"][:-3][-40::2], x["h0"][-3:-2]]), dhT=torch.cat([x["dhT"][:-3][-40::2], x["dhT"][-3:-2]]))
    part = {k: got[k][-320:] for k in ("o", "dq", "dk", "dv")}
    part |= {k: torch.cat([got[k][:-3][-40::2], got[k][-3:-2]]) for k in ("hT", "dh0")}
    check(part, keep)
    empty = [i for i, n in enumerate(lens) if n == 0]
    assert torch.equal(got["hT"][empty].cpu(), x["h0"][empty]) and torch.equal(got["dh0"][empty].cpu(), x["dhT"][empty])


def test_rows_past_32_bits():
    """More than 2^31 elements of v, o, dO and dv: the last sequence's rows are those of the sequence alone."""
    H, HV, D, tail = 2, 256, 128, 90
    T = 65560 + tail
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k = (torch.randn(T, H, D, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    v, dO = (torch.randn(T, HV, D, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    assert v.numel() > 2 ** 31
    g = -torch.exp(torch.linspace(-6, 0, HV, device="cuda"))
    cu = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    o, hT, saved = gdn.linear_fwd(q, k, v, g, cu, save_for_backward=True)
    b = gdn.linear_bwd(q, k, v, g, cu, saved, dO)
    del saved
    one = torch.tensor([0, tail], dtype=torch.int32, device="cuda")
    q, k, v, dO = (x[-tail:].contiguous() for x in (q, k, v, dO))
    o1, hT1, saved = gdn.linear_fwd(q, k, v, g, one, save_for_backward=True)
    b1 = gdn.linear_bwd(q, k, v, g, one, saved, dO)
    assert torch.equal(o[-tail:], o1) and torch.equal(hT[1:], hT1) and torch.equal(b["dh0"][1:], b1["dh0"])
    for n in ("dq", "dk", "dv"):
        assert torch.equal(b[n][-tail:], b1[n]), n


def test_step_in_a_pool_past_32_bits():
    HV, D, slots = 32, 128, 4100
    pool = torch.empty(slots, HV, D, D, device="cuda")
    assert pool.numel() > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (torch.randn(2, HV, D, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    g = torch.full((HV,), -0.1, device="cuda")
    small = torch.randn(3, HV, D, D, generator=gen, device="cuda")
    pool[[1, slots - 1]] = small[1:]
    o = gdn.linear_step(q, k, v, g, pool, torch.tensor([slots - 1, 1], dtype=torch.int32, device="cuda"))
    want = gdn.linear_step(q, k, v, g, small, torch.tensor([2, 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(o, want) and torch.equal(pool[[1, slots - 1]], small[1:])
