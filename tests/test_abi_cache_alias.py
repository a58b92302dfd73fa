"""CPU tests: outputs of the query/key and paged calls that overlap anything the
call reads, and pages of keys that share an element with pages of values, are
refused; pages that interleave in one buffer are not."""

import itertools
import random

import pytest
import torch

from exact_tiled_attention_19_gb300 import binding as B
from tests.test_abi_cache import P, append_call, bwd_call, packed, paged_call, rope_call

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


# ---------------------------------------------------------------- pages of keys and of values

def pages_call(k_at, v_at, k_strides, v_strides, pages, heads, page=8, D=32):
    """attn_paged_append with pages at element offsets of one buffer."""
    st = packed(4, D) + packed(heads, D) * 2 + packed(4, D) + k_strides + [1] + v_strides + [1]
    return append_call(Hkv=heads, D=D, page=page, pages=pages, rope=D, strides=st, kp=P[8] + 2 * k_at,
                       vp=P[8] + 2 * v_at)


LAYOUTS = {  # strides (page, head, slot) and the offset of the values; 3 heads, pages of 8 slots, heads of 32
    "page, k/v, slot, head": ([2 * 768, 32, 96], 768),
    "page, k/v, head, slot": ([2 * 768, 256, 32], 768),
    "page, slot, k/v, head": ([2 * 768, 32, 192], 96),
    "page, slot, head, k/v": ([2 * 768, 64, 192], 32),
    "page, head, slot, k/v": ([2 * 768, 512, 64], 32),
    "page, head, k/v, slot": ([2 * 768, 512, 32], 256),
    "slot outermost": ([96 * 2, 32, 5 * 96 * 2], 96),
    "k/v, page, slot, head": ([768, 32, 96], 5 * 768),
    "layers between": ([7 * 2 * 768, 32, 96], 5 * 768),
}


@pytest.mark.parametrize("name", LAYOUTS)
def test_interleaved_pages_pass_and_shifted_ones_do_not(name):
    strides, at = LAYOUTS[name]
    for a, b in ((0, at), (at, 0)):
        if OK:
            assert pages_call(a, b, strides, strides, 5, 3) == OK
        if name not in ("k/v, page, slot, head", "layers between"):  # (there a shift finds room)
            for shift in (8, -8, 24):
                assert pages_call(a + 64, b + 64 + shift, strides, strides, 5, 3) == ALIAS


def test_pages_of_unlike_strides():
    """Keys by head, values by slot, in halves of each page."""
    k, v = [2 * 768, 256, 32], [2 * 768, 32, 96]
    if OK:
        assert pages_call(0, 768, k, v, 5, 3) == OK
        assert pages_call(768, 0, k, v, 5, 3) == OK
    assert pages_call(0, 760, k, v, 5, 3) == ALIAS
    assert pages_call(0, 0, k, v, 5, 3) == ALIAS
    assert pages_call(0, 768, k, [3 * 768, 32, 96], 5, 3) == ALIAS  # other periods meet sooner or later
    assert pages_call(0, 0, k, k, 1, 3) == ALIAS


def cells(at, strides, pages, heads, page, D):
    """The 16-byte cells of a pages tensor."""
    return {(at + p * strides[0] + h * strides[1] + s * strides[2] + d) // 8
            for p, h, s, d in itertools.product(range(pages), range(heads), range(page), range(0, D, 8))}


@pytest.mark.skipif(OK is None, reason="fake addresses: for machines without a GPU")
def test_pages_against_brute_force():
    """Random nested layouts of equal strides at random distances: refused
    exactly when some element is shared."""
    rng, seen = random.Random(5), [0, 0]
    for _ in range(600):
        pages, heads, page, D = rng.choice([1, 2, 3, 5]), rng.choice([1, 2, 3]), 8, 32
        extent = {0: pages, 1: heads, 2: page}
        order, inner, strides = rng.sample([0, 1, 2], 3), D, [0, 0, 0]
        for axis in order:  # innermost first, with room for others between
            strides[axis] = inner * rng.choice([1, 1, 2, 3]) + 8 * rng.choice([0, 0, 1, 4])
            inner = strides[axis] * (extent[axis] - 1) + inner
        far = rng.choice([D, strides[order[0]], strides[order[1]], strides[order[2]], inner]) + 8 * rng.choice([0, 0, 1, -1])
        a, b = 4096, 4096 + rng.choice([-1, 1]) * far
        shared = bool(cells(a, strides, pages, heads, page, D) & cells(b, strides, pages, heads, page, D))
        assert pages_call(a, b, strides, strides, pages, heads) == (ALIAS if shared else OK), (strides, far, pages, heads)
        seen[shared] += 1
    assert min(seen) > 100
