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


def delta():
    return dict(q=bf(T, H, 128), k=bf(T, H, 128, seed=1), v=bf(T, HV, 128), g=-torch.rand(T, HV, device="cuda"),
                beta=torch.rand(T, HV, device="cuda"), cu_seqlens=ints(0, 130, T))


def chunk_fwd():
    return gdn.chunk_fwd, dict(delta(), h0=torch.randn(2, HV, 128, 128, device="cuda"))


def chunk_fwd_paged():
    return gdn.chunk_fwd_paged, dict(delta(), state_pool=torch.randn(5, HV, 128, 128, device="cuda"),
                                     ssm_state_indices=ints(3, 1), has_initial_state=ints(1, 0))


def chunk_bwd():
    x = delta()
    x["saved"] = gdn.chunk_fwd(**x, save_for_backward=True)[2]
    return gdn.chunk_bwd, dict(x, dO=bf(T, HV, 128, seed=2), dhT=torch.randn(2, HV, 128, 128, device="cuda"))


def chunk_bwd_recompute():
    return gdn.chunk_bwd_recompute, dict(delta(), dO=bf(T, HV, 128, seed=2))


def chunk_transition():
    return gdn.chunk_transition, delta()


def recurrent_step():
    return gdn.recurrent_step, dict(q=bf(T, H, 128), k=bf(T, H, 128, seed=1), v=bf(T, HV, 128), a=bf(T, HV), b=bf(T, HV, seed=1),
                                    A_log=torch.rand(HV, device="cuda"), dt_bias=torch.rand(HV, device="cuda"),
                                    state_pool=torch.randn(T + 1, HV, 128, 128, device="cuda"),
                                    ssm_state_indices=torch.arange(1, T + 1, dtype=torch.int32, device="cuda"))


def conv_fwd():
    return gdn.conv_fwd, dict(x=bf(T, 256), weight=bf(256, 4), bias=bf(256), cu_seqlens=ints(0, 130, T), state_in=bf(2, 256, 3))


def conv_fwd_paged():
    return gdn.conv_fwd_paged, dict(x=bf(T, 256), weight=bf(256, 4), bias=bf(256), cu_seqlens=ints(0, 130, T), state_pool=bf(5, 256, 3),
                                    indices=ints(3, 1), has_initial_state=ints(1, 0))


def conv_bwd():
    return gdn.conv_bwd, dict(x=bf(T, 256), weight=bf(256, 4), bias=bf(256), cu_seqlens=ints(0, 130, T), dy=bf(T, 256, seed=1),
                              state_in=bf(2, 256, 3))


def conv_update():
    return gdn.conv_update, dict(x=bf(T, 256), weight=bf(256, 4), bias=bf(256), state_pool=bf(T + 1, 256, 3),
                                 indices=torch.arange(1, T + 1, dtype=torch.int32, device="cuda"))


def flat(x):
    if isinstance(x, dict):
        x = list(x.values())
    return [x] if isinstance(x, torch.Tensor) else [t for t in x if t is not None]


OPERATORS = [linear_fwd, linear_fwd_paged, linear_bwd, linear_step, rotary, rotary_bwd, rmsnorm_fwd, rmsnorm_bwd,
             chunk_fwd, chunk_fwd_paged, chunk_bwd, chunk_bwd_recompute, chunk_transition, recurrent_step,
             conv_fwd, conv_fwd_paged, conv_bwd, conv_update]


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


@pytest.mark.parametrize("operator", OPERATORS)
def test_outputs_and_workspaces_are_the_streams_memory(operator):
    """What a call made on a busy stream lets go of at its end, its workspace, does not come back on another one; and the
    default stream by its handle."""
    f, x = operator()
    want = flat(f(**{n: t.clone() for n, t in x.items()}))
    side = torch.cuda.Stream()
    mine, again = ({n: t.clone() for n, t in x.items()} for _ in range(2))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = flat(f(**mine, stream=side))
    sizes = [2 ** n for n in range(9, 25) for _ in range(3)]
    fresh = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    assert not side.query()
    side.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
    got = flat(f(**again, stream=torch.cuda.default_stream().cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(fresh) == len(sizes)


@pytest.mark.parametrize("operator", [linear_fwd, linear_bwd, rotary, rmsnorm_bwd, chunk_fwd, conv_bwd])
def test_a_given_stream_that_is_being_captured(operator):
    """The capturing stream handed on by name, a tensor of the call let go of meanwhile; replays beside eager calls."""
    f, x = operator()
    want = flat(f(**{n: t.clone() for n, t in x.items()}))
    g, kept = torch.cuda.CUDAGraph(), {n: t.clone() for n, t in x.items()}
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = flat(f(**kept, stream=torch.cuda.current_stream()))
        other = {n: t.clone() for n, t in kept.items()}  # the graph's own memory
        f(**other, stream=torch.cuda.current_stream())
        del other
    for _ in range(3):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        f(**{n: t.clone() for n, t in x.items()})
        torch.cuda.synchronize()
