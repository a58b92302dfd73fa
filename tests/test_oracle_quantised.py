"""CPU pins of the oracle's 4-bit cache and page bookkeeping: PyTorch's casts,
worked examples, and the bounds that the definitions promise."""

import numpy as np
import pytest
import torch

from oracle import quantised as Q

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_rounding_is_the_type_cast(dt):
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(4000, generator=g) * s for s in (1e-6, 1.0, 3e4)]).float()  # (FP32: one rounding)
    want = x.to(DT[dt]).double().numpy()
    got = Q.rounded(x.double().numpy(), dt)
    assert np.array_equal(got, want)
    assert np.array_equal(Q.from_bits(Q.to_bits(want, dt), dt), want)


def test_rounding_is_done_once():
    # Just above a tie of BF16, by less than FP32 shows: up, and not to the even neighbour.
    x = 1.0 + 2.0 ** -8 + 2.0 ** -40
    assert Q.rounded(x, "bf16") == 1.0 + 2.0 ** -7 and Q.rounded(1.0 + 2.0 ** -8, "bf16") == 1.0
    assert float(torch.tensor(x, dtype=torch.float64).to(torch.bfloat16)) == 1.0  # by way of FP32


def test_a_worked_group():
    x = np.zeros(64)
    x[:4] = [-1.0, 0.5, 2.0, 1.25]           # minimum -1, spread 3: scale 0.2, rounded up in BF16
    c, s, m = Q.quantise(x, "bf16")
    assert m == -1.0 and s == 0.2001953125   # the BF16 numbers next to 0.2 are 0.19921875 and this one
    assert list(c[:5]) == [0, 7, 15, 11, 5]  # 1.5 / s = 7.49, 3 / s = 14.99, 2.25 / s = 11.24, 1 / s = 4.995
    c, s, m = Q.quantise(np.full(64, 3.5), "f16")
    assert s == 0 and m == 3.5 and not c.any()
    x[5] = np.inf
    c, s, m = Q.quantise(x, "bf16")
    assert np.isnan(s) and np.isnan(m) and not c.any()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_values_are_half_a_scale_off_at_most(D, dt):
    rng = np.random.default_rng(D)
    x = Q.rounded(rng.standard_normal((50, D)) * 10.0 ** rng.uniform(-4, 3, (50, 1)), dt)
    c, s, m = Q.quantise(x.reshape(50, -1, Q.group_of(D)), dt)
    assert c.max() == 15 and c.min() == 0
    err = np.abs(Q.values(c, s, m) - x.reshape(c.shape))
    assert np.all(err <= s[..., None] / 2 * (1 + 1e-12))
    assert np.array_equal(Q.stored(x, dt), Q.values(c, s, m).reshape(x.shape))


@pytest.mark.parametrize("D,per_slot", [(32, 20), (64, 36), (128, 72)])
def test_blocks_hold_what_was_packed(D, per_slot):
    rng = np.random.default_rng(D)
    x = Q.rounded(rng.standard_normal((3, 2, 8, D)), "f16")
    b = Q.pack(x, "f16")
    assert b.shape == (3, 2, 8 * per_slot) and b.dtype == np.uint8
    assert np.array_equal(Q.unpack(b, 8, D, "f16"), Q.stored(x, "f16"))
    # the second row's first two codes: byte G/2 of the block, the first in the low half
    c, s, m = Q.quantise(x[0, 0, 1, :Q.group_of(D)], "f16")
    G = Q.group_of(D)
    assert b[0, 0, G // 2] == c[0] | (c[1] << 4)
    assert b[0, 0, 8 * G // 2 + 4:8 * G // 2 + 8].tobytes() == Q.to_bits([s, m], "f16").tobytes()


def test_pages_by_hand():
    table = np.full((3, 4), -1)
    table[0, 0], table[1, :2] = 9, [7, 5]
    # 3, 8 and 0 keys on pages of 4: 2, 1 and 6 new ones
    t, lens, cu, pos, slots, left = Q.extend([2, 1, 6], [3, 8, 0], table, [1, 2, 3, 4, 6], 4, 11)
    assert lens == [5, 9, 6] and cu == [0, 2, 3, 9] and left == [1]
    assert t.tolist() == [[9, 6, -1, -1], [7, 5, 4, -1], [3, 2, -1, -1]]
    assert pos == [3, 4, 8, 0, 1, 2, 3, 4, 5, 0, 0]
    assert slots == [39, 24, 16, 12, 13, 14, 15, 8, 9, -1, -1]
    lens, free = Q.truncate([4, 0, 6], lens, t, left, 4)
    assert lens == [4, 0, 6] and free == [1, 6, 7, 5, 4]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_code_15_stands_for_no_more_than_the_type_holds(dt):
    big = float(torch.finfo(DT[dt]).max)
    for low in (-big if dt == "f16" else -big / 512, 0.0, big / 2):  # (spreads within FP32)
        low = float(Q.rounded(low, dt))
        x = np.full((1, 64), low)
        x[0, ::3], x[0, 1] = big, Q.rounded(low / 2 + big / 4, dt)
        c, s, m = Q.quantise(x, dt)
        v = Q.values(c, s, m)
        assert c.max() == 15 and np.all(np.abs(v) <= big) and np.all(np.abs(v - x) <= s[..., None] * 0.6)
