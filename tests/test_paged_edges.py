"""The paged cache's calls on the GPU at sizes, values and settings that the
other tests do not reach."""
import math

import pytest
import torch

import causal_head_self_gb300 as chs
import paged_ref as ref
from causal_head_self_gb300 import build as _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


def status_ok():
    assert chs.attn_status() == chs.ATTN_OK


# The columns of all heads together, 128 a head where every query votes and 16 where one
# does, pass 32 bits.
@pytest.mark.parametrize("Hq,queries", [(2 ** 24 + 16, 0), (2 ** 27 + 16, 1)])
def test_key_weights_of_more_columns_than_32_bits_count(Hq, queries):
    q = torch.zeros(1, Hq, 1, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(1, Hq, 1, device="cuda")
    w = torch.full((1, 1, 1), 7.0, device="cuda")
    chs.attn_key_weights(q, k, lse, w, queries=queries, accumulate=False)
    status_ok()
    # each head adds e^0: whole numbers that 24 bits hold in each part of the sum, and at its end
    assert w.item() == Hq
