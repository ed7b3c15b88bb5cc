"""Problems of the attention entry points on the CPU that are allowed, or refused, for reasons of their own. No call here reaches a
launch; the addresses are never read."""
import ctypes

import pytest

from tests.test_attention_cpu import ALIGN, FAKE, LIB, NULL, ODD, OK, G, cache, call, problem, pytestmark  # noqa: F401


def test_step_reads_no_boundaries(G):
    """A problem that held a prompt's boundaries before: one token a sequence has none, and the array may be shorter than N + 1."""
    lib, ref = G._lib, ctypes.byref
    for host in ((0, 3, 1), (5, 5, 5), (7,)):
        p = problem(G, T=2, host=host, cu_seqlens=ODD)
        want = lib.gdn_attn_step_workspace_size(ref(problem(G, T=2)), ref(cache(G, columns=4096)))
        assert want > 0 and lib.gdn_attn_step_workspace_size(ref(p), ref(cache(G, columns=4096))) == want
        # the arguments behind them are looked at
        assert call(G, "step", host=host, ptr=dict(o=ODD)) == ALIGN
        assert call(G, "step", host=host, ptr=dict(q=None)) == NULL


@pytest.mark.parametrize("name", ["paged", "step"])
def test_a_cache_has_its_own_strides(G, name):
    """k_stride and v_stride are of token rows: with a cache they are not read."""
    size = getattr(G._lib, dict(paged="gdn_attn_fwd_paged", step="gdn_attn_step")[name] + "_workspace_size")
    big = cache(G, columns=4096)
    want = size(ctypes.byref(problem(G, T=2)), ctypes.byref(big))
    for odd in (dict(k_stride=-1), dict(k_stride=5), dict(v_stride=1 << 40)):
        assert want > 0 and size(ctypes.byref(problem(G, T=2, **odd)), ctypes.byref(big)) == want
        assert call(G, name, ptr=dict(o=ODD), **odd) == ALIGN
