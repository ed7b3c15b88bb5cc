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
