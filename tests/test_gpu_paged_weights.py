"""GPU tests of the weights in attention over a paged cache: their precision, very
many small ones beside a large one, logits of any size, and rows of one unit of
which some read keys that are not finite."""

import math

import numpy as np
import pytest
import torch

from exact_tiled_attention_19_gb300 import binding
from oracle import cache
from tests.test_gpu_paged import make_cache
from tests.test_gpu_rope import f64, half_step

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


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("n,Hq,Hkv", [(1, 8, 2), (4, 8, 2), (5, 8, 2), (9, 8, 1)])  # 16, 32 and several times 32 rows
@pytest.mark.parametrize("kw", [dict(), dict(num_shares=7), dict(window_left=40), dict(causal=False)])
def test_weights_are_not_rounded_to_16_bits(dtype, D, n, Hq, Hkv, kw):
    """One-hot queries make every score one exact product, so that the weights'
    own errors show.  They are 2^-20 (the exponential, in a weight and in the
    sum), 2^-22 of a score of at most 10 for its scaling by log2(e) (counted
    four times), and that of the two 16-bit parts that meet V: 2^-16 relative
    in BF16, 2^-22 in FP16 (and 2^-40 of the largest).  FP32 sums: at
    most L / 16 additions in l and 2 L / 64 of 16 keys each in O per running
    part, the joins of at most 8 parts and of four warps, 2^-23 each: under
    (L / 8 + 64) 2^-23.  Rounding O adds u |O|, and 2^-25 where FP16 has no
    normal value.  (One rounding of the weights to BF16 is 2^-8 of them.)"""
    lens, page = [n + 4, 90, 700], 16
    k_pages, v_pages, table, seqlens = make_cache(lens, page, Hkv, D, dtype, seed=D + n)
    g = torch.Generator().manual_seed(n)
    q = torch.zeros(3 * n, Hq, D)
    q.scatter_(2, torch.randint(0, D, (3 * n, Hq, 1), generator=g), 2.0)
    q = q.to(dtype).cuda()
    o, lse = binding.attention_paged(q, k_pages, v_pages, table, seqlens, scale=1.0, **kw)
    cu = [0, n, 2 * n, 3 * n]
    where = dict(causal=kw.get("causal", True), window_left=kw.get("window_left", -1), scale=1.0)
    args = table.cpu().numpy(), lens, cu
    ro, rl = cache.attention_paged(f64(q), f64(k_pages), f64(v_pages), *args, **where)
    ra, _ = cache.attention_paged(f64(q), f64(k_pages), np.abs(f64(v_pages)), *args, **where)
    bf16 = dtype == torch.bfloat16
    for s, L in enumerate(lens):
        rows = slice(cu[s], cu[s + 1])
        part = (2.0 ** -16 if bf16 else 2.0 ** -22) + 2.0 ** -20 + 4 * 2.0 ** -22 * 10 + (L / 8 + 64) * 2.0 ** -23
        bound = part * ra[rows] + half_step(dtype) * np.abs(ro[rows])
        bound += 1e-30 if bf16 else 2.0 ** -25 + L * 2.0 ** -39 * float(v_pages.abs().max())
        err = np.abs(f64(o)[rows] - ro[rows])
        assert np.all(err <= bound), f"sequence {s}: {np.max(err / bound):.2f} of the bound"
        assert np.all(np.abs(f64(lse)[:, rows] - rl[:, rows]) <= 2.0 ** -18 + (L / 16 + 8) * 2.0 ** -24)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["key", "value"])
def test_each_row_meets_its_own_non_finite_keys_alone(dtype, D, bad, where):
    """Eight new tokens, a window of 20: keys with an infinite or NaN value that
    some rows of a unit read and others do not, before and after the rows'
    ranges.  Rows that read none of them are those of the call without, bit for
    bit; the others are not finite."""
    n, Hq, Hkv, L = 8, 8, 2, 333
    k_pages, v_pages, table, seqlens = make_cache([L], 16, Hkv, D, dtype, seed=D)
    q = torch.randn(n, Hq, D, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    ref, lref = binding.attention_paged(q, k_pages, v_pages, table, seqlens, window_left=20)
    for at in ([L - 1], [L - 3], [L - 27], [L - 24, L - 2], [L - 60], [L - 8 - 10]):
        pages = [k_pages.clone(), v_pages.clone()]
        for j in at:
            pages[where == "value"][int(table[0, j // 16]), :, j % 16] = bad
        o, lse = binding.attention_paged(q, *pages, table, seqlens, window_left=20)
        for i in range(n):
            pos = L - n + i
            if any(pos - 20 <= j <= pos for j in at):
                assert not bool(torch.isfinite(o[i]).all(-1).any()) or where == "key"
            else:
                assert torch.equal(o[i], ref[i]) and torch.equal(lse[:, i], lref[:, i]), (at, i)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("n,Hq", [(1, 4), (3, 4), (5, 8)])
@pytest.mark.parametrize("shares", [1, 9])
def test_an_infinite_value_that_a_row_reads_is_its_result(dtype, D, n, Hq, shares):
    """Infinite values of one sign with weights above 0 make infinity in their
    column, whatever the weights (one key, equal keys, random ones); of both
    signs, or NaN, NaN.  Other columns are not touched."""
    lens, page = [n, 40, 300], 16
    k_pages, v_pages, table, seqlens = make_cache(lens, page, 1, D, dtype, seed=D)
    k_pages[table[1, :3].long()] = 0.25  # the second sequence's keys are equal
    q = torch.randn(3 * n, Hq, D, generator=torch.Generator().manual_seed(2)).to(dtype).cuda() * 0.5
    ref, _ = binding.attention_paged(q, k_pages, v_pages, table, seqlens, num_shares=shares)
    inf, nan = float("inf"), float("nan")
    for L, s in zip(lens, range(3)):
        for j in (0, L - n):  # every row reads both
            v = v_pages[int(table[s, j // page]), 0, j % page]
            v[1], v[3], v[D - 1] = inf, -inf, nan
            v[5] = inf if j else -inf  # both signs where j differs
    o, lse = binding.attention_paged(q, k_pages, v_pages, table, seqlens, num_shares=shares)
    finite = [d for d in range(D) if d not in (1, 3, 5, D - 1)]
    assert torch.equal(o[..., finite], ref[..., finite])
    assert bool((o[..., 1] == inf).all()) and bool((o[..., 3] == -inf).all()) and bool(torch.isnan(o[..., D - 1]).all())
    assert bool(torch.isnan(o[n:, :, 5]).all()) and bool((o[:n, :, 5] == -inf).all())
