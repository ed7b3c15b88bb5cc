"""The operators of a linear-attention layer run together, as a model runs them: norm with the residual
-> projection -> short convolution -> rotary -> linear attention -> per-head norm. Decoding token by token
from the prompt's states, on the two pools, gives the rows that one pass over the whole text gives; and the
backward's gradients are the chain of the oracles' gradients."""
import numpy as np
import pytest
import torch

from oracle import layer as Y
from oracle import linear as L
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn

H, HV, D, W = 2, 4, 64, 4
HID, C = 256, (2 * H + HV) * D


class Layer:
    def __init__(self, seed=0):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        self.norm = (1 + 0.1 * r(HID)).bfloat16().cuda()
        self.proj = (r(HID, C) / HID ** 0.5).bfloat16().cuda()
        self.conv = (r(C, W) / W ** 0.5).bfloat16().cuda()
        self.head_norm = (0.1 * r(D)).bfloat16().cuda()
        self.log_decay = -torch.exp(torch.linspace(-4, -0.5, HV)).cuda()
        self.freq, self.m = gdn.rotary_inv_freq(32, scaling="yarn", factor=4.0, original=64, device="cuda")

    def heads(self, y):
        return [t.unflatten(1, (-1, D)) for t in y.split([H * D, H * D, HV * D], 1)]

    def before(self, x, res):
        n = gdn.rmsnorm_fwd(x, self.norm, residual=res)
        return n["residual_out"], n["y"] @ self.proj

    def after(self, o):
        return gdn.rmsnorm_fwd(o.reshape(-1, D), self.head_norm, unit_offset=True)["y"].view(o.shape)

    def prompt(self, x, res, cu, conv_pool, pool, idx, past):
        fresh = (past > 0).to(torch.int32)
        s, p = self.before(x, res)
        y = gdn.conv_fwd_paged(p, self.conv, None, cu, conv_pool, idx, has_initial_state=fresh)
        q, k, v = self.heads(y)  # slices of the convolution's rows, turned in place
        gdn.rotary(q, k, self.freq, cu_seqlens=cu, offsets=past, mscale=self.m, q_out=q, k_out=k)
        o, _ = gdn.linear_fwd_paged(q, k, v, self.log_decay, cu, pool, idx, has_initial_state=fresh)
        return s, self.after(o)

    def token(self, x, res, positions, conv_pool, pool, idx):
        s, p = self.before(x, res)
        q, k, v = self.heads(gdn.conv_update(p, self.conv, None, conv_pool, idx))
        q, k = gdn.rotary(q, k, self.freq, positions=positions, mscale=self.m)
        return s, self.after(gdn.linear_step(q, k, v, self.log_decay, pool, idx))


def test_prompt_then_tokens_are_one_text():
    lens, more = [70, 129], 9
    layer, gen = Layer(), torch.Generator().manual_seed(3)
    texts = [(torch.randn(n + more, HID, generator=gen).bfloat16().cuda(), torch.randn(n + more, HID, generator=gen).bfloat16().cuda())
             for n in lens]
    cu = lambda ns: torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device="cuda")  # noqa: E731
    idx = torch.tensor([4, 2], dtype=torch.int32, device="cuda")
    pools = lambda: (torch.zeros(6, C, W - 1, dtype=torch.bfloat16, device="cuda"), torch.zeros(6, HV, D, D, device="cuda"))  # noqa: E731
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")

    cp, pool = pools()
    whole_s, whole = layer.prompt(*(torch.cat([t[i] for t in texts]) for i in (0, 1)), cu([n + more for n in lens]), cp, pool, idx, zero)
    end = pool.clone()

    cp, pool = pools()
    first = [20, 64]  # the prompt in two pieces, the second resumed from the pools
    pieces = [[(t[0][:a], t[1][:a]) for t, a in zip(texts, first)], [(t[0][a:n], t[1][a:n]) for t, a, n in zip(texts, first, lens)]]
    got = [[], []]
    past = zero
    for piece in pieces:
        ns = [p[0].shape[0] for p in piece]
        _, o = layer.prompt(*(torch.cat([p[i] for p in piece]) for i in (0, 1)), cu(ns), cp, pool, idx, past)
        for i, part in enumerate(o.split(ns)):
            got[i].append(part)
        past = past + torch.tensor(ns, dtype=torch.int32, device="cuda")
    for j in range(more):
        x, r = (torch.stack([t[i][n + j] for t, n in zip(texts, lens)]) for i in (0, 1))
        _, o = layer.token(x, r, past, cp, pool, idx)
        past = past + 1
        for i in range(2):
            got[i].append(o[i:i + 1])
    # the head norm divides a row by its size: rows within 2^-7 of each other before it (two roundings to bf16 on each side of the
    # linear attention, as in its own tests), and one rounding after it
    for mine, want in zip(got, whole.split([n + more for n in lens])):
        a, b = f64(torch.cat(mine)), f64(want)
        assert np.linalg.norm(a - b) <= 2.0 ** -6 * np.linalg.norm(b)
    # the states gather the same bf16 rows in fp32, in another order
    assert torch.allclose(pool[[2, 4]], end[[2, 4]], rtol=0, atol=2.0 ** -24 * 256 * float(end.abs().max()))
    assert not pool[[0, 1, 3, 5]].any()


def test_training_chain_matches_the_oracles():
    """rotary -> linear attention -> norm: each operator's backward, fed by the next one's."""
    gen = torch.Generator().manual_seed(5)
    lens = [65, 40]
    T, cu = sum(lens), torch.tensor([0, 65, 105], dtype=torch.int32, device="cuda")
    r = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()  # noqa: E731
    q, k, v, w, dy = r(T, H, D), r(T, H, D), r(T, HV, D), r(D), r(T * HV, D)
    layer = Layer(1)
    turn = dict(cu_seqlens=cu, interleaved=True, mscale=layer.m)
    qr, kr = gdn.rotary(q, k, layer.freq, **turn)
    o, _, saved = gdn.linear_fwd(qr, kr, v, layer.log_decay, cu, save_for_backward=True)
    n = gdn.rmsnorm_fwd(o.view(-1, D), w, want_rstd=True)
    gn = gdn.rmsnorm_bwd(dy, o.view(-1, D), w, n["rstd"])
    g = gdn.linear_bwd(qr, kr, v, layer.log_decay, cu, saved, gn["dx"].view(o.shape))
    dq, dk = gdn.rotary_bwd(g["dq"], g["dk"], layer.freq, **turn)

    # the same chain in 64 bits from the tensors that each operator was given
    pos = Y.positions([0, 65, 105])
    dx, dw = Y.rmsnorm_backward(f64(o).reshape(-1, D), f64(dy), f64(w))
    ref = L.backward(f64(qr), f64(kr), f64(v), f64(layer.log_decay), [0, 65, 105], dx.reshape(T, HV, D))
    turned = {x: Y.rotary(ref[x], pos, f64(layer.freq), True, layer.m, back=True) for x in ("dq", "dk")}
    # relative 2-norms: a rounding to bf16 is below 2^-8 of a tensor's norm; dx carries one, what the linear attention makes of
    # it two more, the turn back a fourth
    near = lambda a, b, c: np.linalg.norm(f64(a).ravel() - b.ravel()) <= c * 2.0 ** -8 * np.linalg.norm(b)  # noqa: E731
    assert near(gn["dx"], dx, 1) and near(gn["dweight"], dw, 2.0 ** -8)
    assert near(g["dv"], ref["dv"], 3) and near(g["dh0"], ref["dh0"], 1)
    assert near(dq, turned["dq"], 4) and near(dk, turned["dk"], 4)


def test_e4m3_norm_in_front_of_a_product():
    """x + residual -> e4m3 rows with scales -> dequantised product, against the product of the bf16 norm: an element is off by
    2^-4 of its value at most, so a row's product, a sum with errors of any sign, by 2^-4 of the product of absolute values."""
    layer, gen = Layer(2), torch.Generator().manual_seed(6)
    x, r = (torch.randn(50, HID, generator=gen).bfloat16().cuda() for _ in range(2))
    out = gdn.rmsnorm_fwd(x, layer.norm, residual=r, quant=128, want_y=True)
    back = out["y8"].float() * out["scales"].repeat_interleave(128, 1)
    err = (back @ layer.proj.float() - out["y"].float() @ layer.proj.float()).abs()
    assert bool((err <= (2.0 ** -4 + 2.0 ** -7) * (out["y"].float().abs() @ layer.proj.float().abs())).all())
