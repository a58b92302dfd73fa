"""GPU tests of what the append to a 4-bit cache stores of normed keys whose squares
leave FP32's range, byte by byte: very large and very small rows, large elements in
rows of ordinary ones, infinities and NaN."""

import numpy as np
import pytest
import torch

from exact_tiled_attention_19_gb300 import binding
from oracle import cache, quantised
from tests.test_gpu_q4 import DT, code_of, f64
from tests.test_gpu_q4_rounding import same, stored

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert binding.etattn_read_device_status(clear=True) == 0


def keys_with_norm(x, dtype, eps, rope, seed):
    """(keyword arguments, the keys that norm and rotation leave, in 64 bits)."""
    T, H, D = x.shape
    g = torch.Generator().manual_seed(seed)
    wk = (1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda()
    kw = dict(k_weight=wk, eps=eps)
    c = s = None
    if rope:
        cos, sin = binding.rope_tables(3000, rope)
        pos = torch.randint(0, 3000, (T,), generator=g, dtype=torch.int32)
        kw.update(rope_cos=cos, rope_sin=sin, positions=pos.cuda())
        c, s = f64(cos)[pos.numpy()], f64(sin)[pos.numpy()]
    return kw, quantised.rounded(cache.norm_rope(f64(x), f64(wk), c, s, False, eps=float(np.float32(eps))), code_of(dtype))


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", [5, 3000])
@pytest.mark.parametrize("rope", [0, 1])
def test_normed_keys_of_any_size(D, T, rope):
    """Rows of BF16 from 2^-110 to 2^126, and rows with single elements of such sizes: what
    exact arithmetic leaves, rounded once.  (eps far below the squares, or beside them.)"""
    g = torch.Generator().manual_seed(D + T)
    x = torch.randn(T, 6, D, generator=g, dtype=torch.float64)
    e = torch.randint(-110, 124, (T, 6, 1), generator=g).double()
    x = x * 2.0 ** e
    x[::5, :, 7] *= 2.0 ** 20
    x[1::5] = torch.randn(x[1::5].shape, generator=g, dtype=torch.float64)  # rows as they mostly are, beside them
    x[2::5, 0] = 0
    x[2::5, 1] = torch.sign(x[2::5, 1]) * 2.0 ** 126
    x[3::5, 2, 5] = 2.0 ** 70                                                # one large element
    x = x.clamp(-3e38, 3e38).to(torch.bfloat16)
    for eps in (1e-6, 1e-30):
        kw, want = keys_with_norm(x, torch.bfloat16, eps, D if rope else 0, T)
        got = stored(x.cuda(), D, "bf16", k=x.cuda(), **kw)
        same(got, want, D, "bf16")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_normed_keys_with_infinities_and_nan(D, dt):
    """An infinite element makes itself NaN and the others 0, so that a group without one
    is of zeros; a NaN makes the whole row NaN."""
    x = torch.randn(9, 2, D, generator=torch.Generator().manual_seed(D)).to(DT[dt])
    x[1, 0, 3], x[2, 1, D - 1], x[3, 0, 5], x[4, 1, 6] = float("inf"), float("-inf"), float("nan"), float("inf")
    x[4, 1, 7] = float("nan")
    with np.errstate(invalid="ignore"):
        kw, want = keys_with_norm(x, DT[dt], 1e-6, 0, 1)
    same(stored(x.cuda(), D, dt, k=x.cuda(), **kw), want, D, dt)
