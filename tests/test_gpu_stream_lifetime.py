"""A call on a given stream keeps its tensors' memory: inputs that the caller lets go of while the stream is still
busy are not handed out again before it is through."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from chunked_gated_delta_04_amd import gdn

T, H, HV, D = 200, 2, 4, 64


def bf(*shape, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=gen, device="cuda").bfloat16()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def linear():
    return dict(q=bf(T, H, D), k=bf(T, H, D, seed=1), v=bf(T, HV, D), log_decay=-torch.rand(HV, device="cuda"))


def linear_fwd():
    return gdn.linear_fwd, dict(linear(), cu_seqlens=ints(0, 130, T), h0=torch.randn(2, HV, D, D, device="cuda"))


def linear_fwd_paged():
    return gdn.linear_fwd_paged, dict(linear(), cu_seqlens=ints(0, 130, T), state_pool=torch.randn(5, HV, D, D, device="cuda"),
                                      ssm_state_indices=ints(3, 1), has_initial_state=ints(1, 0))


def linear_bwd():
    x = dict(linear(), cu_seqlens=ints(0, 130, T))
    x["saved"] = gdn.linear_fwd(**x, save_for_backward=True)[2]
    return gdn.linear_bwd, dict(x, dO=bf(T, HV, D, seed=2), dhT=torch.randn(2, HV, D, D, device="cuda"))


def linear_step():
    return gdn.linear_step, dict(linear(), state_pool=torch.randn(T + 1, HV, D, D, device="cuda"),
                                 ssm_state_indices=torch.arange(1, T + 1, dtype=torch.int32, device="cuda"))


def rotary():
    return gdn.rotary, dict(q=bf(T, H, D), k=bf(T, H, D, seed=1), inv_freq=gdn.rotary_inv_freq(32, device="cuda")[0],
                            cu_seqlens=ints(0, 130, T), offsets=ints(7, 9))


def rotary_bwd():
    return gdn.rotary_bwd, dict(dq_out=bf(T, H, D), dk_out=bf(T, H, D, seed=1), positions=torch.arange(T, dtype=torch.int32, device="cuda"),
                                inv_freq=gdn.rotary_inv_freq(32, device="cuda")[0])


def rmsnorm_fwd():
    return gdn.rmsnorm_fwd, dict(x=bf(T, 512), weight=bf(512), residual=bf(T, 512, seed=1))


def rmsnorm_bwd():
    return gdn.rmsnorm_bwd, dict(dy=bf(T, 512), s=bf(T, 512, seed=1), weight=bf(512), rstd=torch.rand(T, device="cuda"),
                                 dresidual_out=bf(T, 512, seed=2))


def flat(x):
    if isinstance(x, dict):
        x = list(x.values())
    return [x] if isinstance(x, torch.Tensor) else [t for t in x if t is not None]


OPERATORS = [linear_fwd, linear_fwd_paged, linear_bwd, linear_step, rotary, rotary_bwd, rmsnorm_fwd, rmsnorm_bwd]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("operator", OPERATORS)
def test_inputs_let_go_of_while_the_stream_is_busy(operator, raw):
    f, x = operator()
    mine, spare = ({n: t.clone() for n, t in x.items()} for _ in range(2))
    want = flat(f(**spare))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = flat(f(**mine, stream=side.cuda_stream if raw else side))
    held = {t.data_ptr() for t in mine.values()}
    sizes = [t.numel() * t.element_size() for t in mine.values()]
    del mine
    fresh = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    assert not side.query()
    assert not held & {t.data_ptr() for t in fresh}
    side.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
