"""CPU tests: calls on the paged cache whose tokens do not divide among the
sequences are refused, also where one of the counts is 0; counts of 0 that fit
are empty work."""

import pytest
import torch

from exact_tiled_attention_19_gb300 import binding as B
from tests.test_abi_cache import P, append_call, paged_call


@pytest.mark.parametrize("kw", [
    dict(S=5, T=3, mq=0),   # fewer tokens than sequences: T // S is 0
    dict(S=5, T=10, mq=0),
    dict(S=0, T=3, mq=0), dict(S=0, T=3, mq=2),
    dict(S=5, T=9, mq=2),
])
def test_paged_tokens_that_do_not_divide_are_refused(kw):
    assert paged_call(**kw) == B.ETATTN_ERR_BAD_SHAPE


@pytest.mark.parametrize("kw", [dict(S=0, T=3), dict(S=5, T=3), dict(S=3, T=10)])
def test_append_tokens_that_do_not_divide_are_refused(kw):
    assert append_call(**kw) == B.ETATTN_ERR_BAD_SHAPE


def test_counts_of_zero_that_fit_are_empty_work():
    assert paged_call(S=5, T=0, mq=0) == 0
    assert paged_call(S=0, T=0, mq=3) == 0
    assert paged_call(S=5, T=0, mq=2) == 0
    assert paged_call(S=5, T=0, mq=2, cu=P[8]) == 0
    assert paged_call(S=5, T=3, mq=0, Hq=0) == 0
    assert paged_call(S=0, T=3, mq=2, cu=P[8]) == 0  # every row is behind the last sequence
    assert append_call(S=0, T=3, cu=P[12]) == 0
    assert append_call(S=0, T=0) == 0


def test_offsets_with_a_bound_of_zero_are_looked_at_on_the_device():
    """The offsets may say that nobody has a new token, or that the bound is
    wrong: only the device knows, so the call goes there (and needs no
    workspace)."""
    if not torch.cuda.is_available():
        assert paged_call(T=10, mq=0, cu=P[8]) == B.ETATTN_ERR_NO_DEVICE
        assert paged_call(T=10, mq=0, cu=P[8], ws=0, wsb=0) == B.ETATTN_ERR_NO_DEVICE
    assert paged_call(T=10, mq=0, cu=P[8], q=0) == B.ETATTN_ERR_NULL_PTR
