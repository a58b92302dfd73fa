"""GPU tests of the weights in attention over a paged cache where one key has
nearly all of the weight and very many others share the rest."""

import math

import pytest
import torch

from exact_tiled_attention_19_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert binding.etattn_read_device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("n,Hq,shares", [(1, 4, None), (1, 4, 1), (5, 8, None)])  # 16 and 32 rows a unit
@pytest.mark.parametrize("first", [True, False])
def test_small_weights_of_many_keys_count(dtype, D, n, Hq, shares, first):
    """Logits 0 but for one key's, 17.6875: the others weigh 2^-25.5 each beside
    its 1, which no normal FP16 value holds, and 2^-8.5 together.  Values are 1
    but for that key's 0, so O is the others' part.  The logits are exact.  The
    scaling by log2(e) and the exponential move a weight by under 2^-18, its
    rounding by u = eps / 2, and in FP16, where the largest weight is held as
    2^15, by 2^-40 at the least; O's rounding adds u again.  A row's sum has 16
    running parts (4 warps of 4 lanes) of at most L / 16 FP32 additions, each
    off by 2^-24 of it; its products with V 4 running parts of L / 64 additions
    of 16 keys, each off by 2^-23 (chopped): in relative terms L 2^-28 and
    L 2^-29, with one share; with more it is less."""
    L, page = 1 << 17, 256
    table = torch.randperm(L // page, dtype=torch.int32)[None].cuda()
    k_pages = torch.zeros(L // page, 1, page, D, dtype=dtype, device="cuda")
    v_pages = torch.ones_like(k_pages)
    at = 7 if first else L - 100
    hit = int(table[0, at // page]), 0, at % page
    k_pages[hit][0], v_pages[hit][:] = 17.6875, 0
    if dtype == torch.bfloat16:
        k_pages[hit][0] = 17.625  # 8 bits
    peak = float(k_pages[hit][0])
    q = torch.zeros(n, Hq, D, dtype=dtype, device="cuda")
    q[..., 0] = 1
    seqlens = torch.tensor([L], dtype=torch.int32, device="cuda")
    o, lse = binding.attention_paged(q, k_pages, v_pages, table, seqlens, scale=1.0, num_shares=shares)
    u, sums = torch.finfo(dtype).eps / 2, L * (2.0 ** -28 + 2.0 ** -29)
    for i in range(n):
        others = (L - n + i) * math.exp(-peak)
        want = others / (1 + others)
        got = o[i].double()
        assert float((got - want).abs().max()) <= (2 * u + sums + 2.0 ** -18 + 2.0 ** -40 / math.exp(-peak)) * want
        assert float((lse[:, i].double() - peak - math.log1p(others)).abs().max()) <= L * 2.0 ** -28 + 2.0 ** -16


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("shares", [1, 6])
def test_logits_of_any_size(dtype, sign, shares):
    """Keys of one logit each, from 1 to 2^40 and beyond the steps of FP32: all
    weights are the same, so O is the mean of the values (all 1, exactly), and
    lse the logit, within its own roundings (2^-22) and ln of the keys."""
    L, page, D = 300, 16, 64
    table = torch.randperm(19, dtype=torch.int32)[None].cuda()
    k_pages = torch.zeros(19, 2, page, D, dtype=dtype, device="cuda")
    k_pages[..., 0] = sign * 4096
    v_pages = torch.ones_like(k_pages)
    seqlens = torch.tensor([L], dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 8, D, dtype=dtype, device="cuda")
    q[0, :, 0] = torch.tensor([1, 3, 1024, 1536, 8192, 11264, 20480, 65280]).to(dtype)
    for scale in [2.0 ** e * f for e in range(-12, 12) for f in (1.0, 1.13, 0.71)]:
        o, lse = binding.attention_paged(q, k_pages, v_pages, table, seqlens, scale=scale, num_shares=shares)
        assert bool((o == 1).all()), scale
        want = q[0, :, 0].double() * (sign * 4096 * scale)
        assert bool(((lse[:, 0].double() - want - math.log(L)).abs() <= 2.0 ** -22 * want.abs() + 2.0 ** -18).all()), scale
