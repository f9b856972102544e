"""Sizes at the ends of what the paged cache's calls take, refused before any CUDA
call (made-up addresses: nothing is dereferenced or launched)."""
import pytest
import torch

import causal_head_self_gb300 as chs
from causal_head_self_gb300 import _binding
from causal_head_self_gb300 import build as _build

INVALID = chs.ATTN_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _binding.load()


def ptr(i):
    return (i + 1) << 38


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("budget", [2 ** 31 - 1, 2 ** 31 - 1024, 2 ** 31 - 16384])
def test_a_budget_that_the_kernels_could_not_count_to_is_refused(lib, budget, in_place):
    # (the list of kept rows would fit in memory; a 32-bit counter past its end would not)
    table_out, w_out = (None, None) if in_place else (ptr(5), ptr(6))
    for recent in (0, budget):
        assert lib.attn_cache_evict(ptr(0), ptr(1), ptr(2), 64, ptr(3), ptr(4), budget, recent,
                                    table_out, 4, w_out, 64, ptr(7), ptr(8), 1, 1, 10, 16, 4, 128,
                                    None) == INVALID


def test_the_workspace_query_checks_the_shapes():
    # (2^32 + 5 would reach the library as 5, and the answer would be for 5 columns)
    q, kp = torch.zeros(2, 4, 1, 64), torch.zeros(3, 2, 8, 64)
    table, one, big = torch.zeros(2, 5), torch.zeros(1), 2 ** 32 + 5
    for args in ((q, kp, one.expand(2, big)), (one.expand(2, big, 1, 64), kp, table),
                 (q, one.expand(3, big, 8, 64), table), (q, one.expand(3, 2, 2 ** 32 + 8, 64), table),
                 (one.expand(2 ** 32 + 2, 4, 1, 64), kp, one.expand(2 ** 32 + 2, 5)),
                 (q[:, :, :, :32], kp, table), (q, kp, table[:1]), (q.expand(2, 4, 3, 64), kp, table),
                 (q[0], kp, table), (q, kp[0], table), (q, kp, table[0])):
        with pytest.raises(ValueError):
            chs.attn_decode_paged_workspace(*args)
    with pytest.raises(TypeError):
        chs.attn_decode_paged_workspace(q, kp, None)
