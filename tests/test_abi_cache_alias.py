"""CPU tests: outputs of the query/key and paged calls that overlap anything the
call reads are refused."""

import pytest
import torch

from exact_tiled_attention_19_gb300 import binding as B
from tests.test_abi_cache import P, append_call, bwd_call, paged_call, rope_call

OK = 12 if not torch.cuda.is_available() else None  # past the checks: no device here
ALIAS = B.ETATTN_ERR_ALIAS


@pytest.mark.parametrize("kw", [
    dict(wq=P[7]), dict(wk=P[7] + 1024), dict(wq=P[8]), dict(cos=P[8] + 16), dict(sin=P[7] + 4096), dict(pos=P[7] + 64),
    dict(pos=P[8] - 4), dict(cos=P[7] - 100 * 32 * 4 + 16),
])
def test_rope_outputs_over_what_it_reads(kw):
    assert rope_call(**kw) == ALIAS


def test_rope_neighbours_are_not_overlaps():
    if OK:
        assert rope_call(cos=P[7] - 100 * 32 * 4, sin=P[8] - 100 * 32 * 4) == OK
        assert rope_call(wq=P[7] + 10 * 4 * 64 * 2, pos=P[8] - 40) == OK
        # absent ones do not count
        assert rope_call(rope=0, cos=P[7], sin=P[7], pos=P[8]) == OK


@pytest.mark.parametrize("kw", [
    dict(wq=P[9]), dict(wk=P[10]), dict(cos=P[9] + 16), dict(sin=P[10]), dict(pos=P[9]), dict(wq=P[11]), dict(wk=P[12]),
    dict(cos=P[12]), dict(pos=P[11] + 4), dict(wk=P[13]), dict(sin=P[13] + 256), dict(pos=P[13]),
])
def test_rope_backward_outputs_over_what_it_reads(kw):
    assert bwd_call(**kw) == ALIAS


@pytest.mark.parametrize("kw", [
    dict(wq=P[7]), dict(wk=P[8] + 256), dict(cos=P[9]), dict(sin=P[7]), dict(bt=P[7] + 4), dict(bt=P[8]),
    dict(lens=P[9] + 8), dict(lens=P[8] - 16), dict(cu=P[9] - 8, S=3), dict(cu=P[7], S=3), dict(bt=P[9] - 4 * 30 + 4),
])
def test_append_outputs_over_what_it_reads(kw):
    assert append_call(**kw) == ALIAS


@pytest.mark.parametrize("kw", [
    dict(bt=P[3]), dict(lens=P[3] + 4), dict(cu=P[3] + 16), dict(bt=P[4]), dict(lens=P[4]), dict(cu=P[4] + 8),
    dict(bt=P[7]), dict(lens=P[7] + 1024), dict(cu=P[7] + 4),
])
def test_paged_outputs_over_what_it_reads(kw):
    assert paged_call(**kw) == ALIAS
