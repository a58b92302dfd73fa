"""GPU tests of what the append to a 4-bit cache stores at the edges of its
arithmetic, byte by byte: spreads that FP32 rounds, and code 15 next to the type's
largest number."""

import numpy as np
import pytest
import torch

from exact_tiled_attention_19_gb300 import binding
from oracle import quantised
from tests.test_gpu_q4 import DT, blocks_of, check_append, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert binding.etattn_read_device_status(clear=True) == 0


def stored(x, D, dt, page=8, k=None, **kw):
    """The parts of a cache after rows x [T, H, D] are appended as values (and k as keys)."""
    T, H = x.shape[:2]
    k_pages, v_pages = binding.q4_pages(-(-T // page), H, page, D)
    binding.paged_append_q4(x if k is None else k, x, k_pages, v_pages, torch.arange(T).cuda(), **kw)
    pages = v_pages if k is None else k_pages
    at, slot = np.arange(T) // page, np.arange(T) % page
    return tuple(p[at, :, slot] for p in quantised.parts(blocks_of(pages), page, D, dt))


def same(got, rows, D, dt):
    """Scales and minima as defined; codes from them by the definition's roundings: x - m and
    the quotient to FP32, then to whole numbers."""
    T, H = rows.shape[:2]
    groups = rows.reshape(T, H, -1, quantised.group_of(D))
    with np.errstate(all="ignore"):
        _, s, m = quantised.quantise(groups, dt)
        c = np.rint((groups - m[..., None]).astype(np.float32) / s.astype(np.float32)[..., None])
        c = np.where(s[..., None] > 0, c, 0)
    gc, gs, gm = got
    assert np.array_equal(quantised.to_bits(gs, dt), quantised.to_bits(s, dt))
    assert np.array_equal(gm, m, equal_nan=True)  # (zeros of either sign)
    assert np.array_equal(gc, c.reshape(T, H, D))


@pytest.mark.parametrize("D", [32, 64, 128])
def test_spreads_that_fp32_rounds(D):
    """A maximum of 15 s (or a step of it more) beside a minimum of either sign so small that
    FP32 has the spread 15 s exactly: the scale has to be the next one where the minimum is
    negative, and s where it is positive."""
    g = torch.Generator().manual_seed(D)
    rows = []
    for s in (1.0, 2.0 ** -40, 2.0 ** 60, 17.0, 1.0625 * 2.0 ** 5):
        for low in (-2.0 ** -30, 2.0 ** -30, -2.0 ** -50, 2.0 ** -25, -2.0 ** -24, 0.0):
            x = torch.rand(D, generator=g, dtype=torch.float64) * 15 * s
            x[::7], x[3::7] = 15 * s, low * s
            rows.append(x)
            rows.append(-x)
    x = torch.stack(rows).reshape(-1, 2, D).bfloat16()
    hit = f64(x).reshape(x.shape[0], 2, -1, quantised.group_of(D))
    span = hit.max(-1) - hit.min(-1)
    assert (span != span.astype(np.float32)).sum() > 20
    same(stored(x.cuda(), D, "bf16"), f64(x), D, "bf16")


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_code_15_next_to_the_types_largest_number(D, dt):
    """A maximum of the type's largest number with minima from 0 up, some so small that FP32
    rounds 15 s + m to that number although it is more."""
    big = torch.finfo(DT[dt]).max
    g = torch.Generator().manual_seed(D)
    rows = []
    for e in range(0, 127 if dt == "bf16" else 15, 3):
        for low in (2.0 ** e, 2.0 ** -e, -(2.0 ** -e), 0.0):
            x = torch.rand(D, generator=g, dtype=torch.float64) * big * 0.9 + abs(low)
            x[::7], x[3::7] = big, low
            rows.append(x)
    x = torch.stack(rows).reshape(-1, 2, D).to(DT[dt])
    same(stored(x.cuda(), D, dt), f64(x), D, dt)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_large_and_small_rows_of_values_and_unnormed_keys(dt):
    x = torch.randn(50, 6, 128, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    x *= 2.0 ** torch.linspace(-14 if dt == "f16" else -120, 13 if dt == "f16" else 120, 50).double()[:, None, None]
    check_append(50, 2, 2, 128, DT[dt], 16, rope_dim=0, weighted=False, x=x, seed=4)
