"""GPU tests of the weights in attention over a 4-bit cache, row by row: keys whose
values have far larger scales than the others', read by some rows of a unit and not
by the rest, or with a weight that does not count; very many small weights; and
pages larger than a tile.

Bounds.  For row i, key j and a group with scale s, minimum m and codes c, let p be
the weight.  The kernel adds p s (c - 8) and p (m + 8 s), so with
    B = sum_j p_j (s_j |c_jd - 8| + |m_j + 8 s_j|)
the terms of tests/test_gpu_q4.py stand: ds_j for a key's score (and the sum's is their mean),
w of p s for its rounding to FP16 (2^-11 in one part, for BF16 outputs; 2^-21 in two), 2^-20
for exponential and sum.  A tile's products with c are added to -8 times its weights, so
partial sums reach 8 sum p s and more, whatever c is: the sums' (32 + keys / 16) 2^-24 are of
    A = sum_j p_j (8 s_j + s_j |c_jd - 8| + |m_j + 8 s_j|).
P s is multiplied by a power of two for each row, warp and group, which takes the largest
so far to 2^5.5 and more; a score that passes the row's reference may leave it a factor of two
lower, and the tests here have at most one such time after the largest P s.  FP16's denormals
lose 2^-25 a part, |c - 8| is 8 at most: 2^-24 8 / 2^4.5 < 2^-25 of the row's largest p s a key, and
    |dO| <= (w + 2^-20) B + (32 + keys/16) 2^-24 A + B weighted by ds + u |O| + 2^-25 keys max_j p_j s_j,
with 2^-25 more for FP16 outputs.  max_j is over the keys that the row itself reads."""

import math

import numpy as np
import pytest
import torch

from exact_tiled_attention_19_gb300 import binding
from oracle import quantised
from tests.test_gpu_q4 import DT, attend, blocks_of, code_of, f64, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    torch.manual_seed(0)
    yield
    assert binding.etattn_read_device_status(clear=True) == 0


def rows_of(pages, page, table, L, dtype):
    """(codes [Hkv, L, D], scales [Hkv, L, D / G], minima) of one sequence's keys."""
    D = {20: 32, 36: 64, 72: 128}[pages.shape[2] // page]
    at, slot = table.cpu().numpy()[np.arange(L) // page], np.arange(L) % page
    return tuple(x[at, :, slot].transpose(1, 0, 2) for x in quantised.parts(blocks_of(pages), page, D, code_of(dtype)))


def check_rows(o, q, k_pages, v_pages, page, table, L, scale=None):
    """One sequence, causal, against 64 bits; every row's bound by what it reads itself."""
    n, Hq, D = q.shape
    dtype = q.dtype
    G, scale = quantised.group_of(D), D ** -0.5 if scale is None else scale
    u = torch.finfo(dtype).eps / 2
    w, least = (2.0 ** -21, 2.0 ** -25) if dtype == torch.float16 else (2.0 ** -11, 1e-30)
    kc, ks, km = rows_of(k_pages, page, table, L, dtype)
    vc, vs, vm = rows_of(v_pages, page, table, L, dtype)
    wide = lambda x: np.repeat(x, G, -1)  # noqa: E731
    group = Hq // kc.shape[0]
    for i in range(n):
        keys = L - n + i + 1
        for h in range(Hq):
            hk = h // group
            k, s, m = kc[hk, :keys], vs[hk, :keys], vm[hk, :keys]
            Q = f64(q)[i, h]
            S = (k * wide(ks[hk, :keys]) + wide(km[hk, :keys])) @ Q * scale
            A = (k * wide(ks[hk, :keys]) + np.abs(wide(km[hk, :keys]))) @ np.abs(Q) * scale
            p = np.exp(S - S.max())
            p /= p.sum()
            ds = (2 * D + 16) * 2.0 ** -23 * A + 2.0 ** -38 * np.abs(Q).max() * scale * D * 8
            V = vc[hk, :keys] * wide(s) + wide(m)
            terms = wide(s) * np.abs(vc[hk, :keys] - 8) + np.abs(wide(m) + 8 * wide(s))
            want = p @ V
            bound = ((w + 2.0 ** -20) * (p @ terms) + (32 + keys / 16) * 2.0 ** -24 * (p @ (8 * wide(s) + terms))
                     + 1.1 * (p * (ds + p @ ds)) @ terms + u * np.abs(want)
                     + 2.0 ** -25 * keys * wide((p[:, None] * s).max(0)) + least)
            x = np.abs(f64(o)[i, h] - want)
            assert np.all(x <= bound), f"row {i}, head {h}: {np.max(x / bound):.2f} of the bound"


def set_value(pages, page, table, j, dtype, scale, minimum=0.0):
    """Scale and minimum of key j's values, in every head and group."""
    D = {20: 32, 36: 64, 72: 128}[pages.shape[2] // page]
    G = quantised.group_of(D)
    at, slot, part = int(table[j // page]), j % page, page * (G // 2 + 4)
    word = quantised.to_bits(np.array([scale, minimum]), code_of(dtype)).tobytes()
    for g in range(D // G):
        place = g * part + page * (G // 2) + slot * 4
        pages[at, :, place:place + 4] = torch.tensor(list(word), dtype=torch.uint8, device="cuda")


LARGE = [("bf16", 2.0 ** 20), ("bf16", 2.0 ** 33), ("bf16", 2.0 ** 100), ("f16", 4096.0)]


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt,large", LARGE)
@pytest.mark.parametrize("n,Hq,Hkv", [(2, 4, 2), (4, 2, 2), (4, 4, 2), (4, 8, 2), (3, 20, 1)])  # 4, 8 and 16 rows a unit
def test_a_large_scale_that_only_later_tokens_read(D, dt, large, n, Hq, Hkv):
    """The last token's value has a far larger scale than all others: the earlier tokens'
    rows are what they are without it, bit for bit."""
    dtype, page, L = DT[dt], 16, 300
    k_pages, v_pages, table, seqlens = make_cache([L], page, Hkv, D, dtype, seed=n + D)
    q = torch.randn(n, Hq, D).to(dtype).cuda()
    for shares in (1, 3):
        want, want_lse = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens, num_shares=shares)
        check_rows(want, q, k_pages, v_pages, page, table[0], L)
        vp = v_pages.clone()
        set_value(vp, page, table[0], L - 1, dtype, large)
        o, lse = binding.attention_paged_q4(q, k_pages, vp, table, seqlens, num_shares=shares)
        assert torch.equal(o[:n - 1], want[:n - 1]) and torch.equal(lse, want_lse)
        check_rows(o, q, k_pages, vp, page, table[0], L)


@pytest.mark.parametrize("D,dt", [(32, "bf16"), (64, "f16"), (128, "f16"), (128, "bf16")])
@pytest.mark.parametrize("n,Hq", [(1, 4), (1, 8), (4, 4)])
def test_a_row_does_not_see_the_other_rows_scores(D, dt, n, Hq):
    """One head's queries 50 times as large: weights against another reference there, the
    other heads' rows bit for bit as before."""
    dtype, L = DT[dt], 900
    k_pages, v_pages, table, seqlens = make_cache([L], 16, 1, D, dtype, seed=D)
    q = torch.randn(n, Hq, D).to(dtype).cuda()
    want, want_lse = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens)
    q[:, 1] *= 50
    o, lse = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens)
    others = [h for h in range(Hq) if h != 1]
    assert torch.equal(o[:, others], want[:, others]) and torch.equal(lse[others], want_lse[others])
    assert not torch.equal(o[:, 1], want[:, 1])


def with_scores(D, dtype, page, L, scores, q, seed):
    """A cache of one sequence and head whose keys have about these scores with every row of
    q (rows of one direction, of length sqrt(D)), and random values."""
    rng = np.random.default_rng(seed)
    k_pages, v_pages, table, seqlens = make_cache([L], page, 1, D, dtype, seed=seed)
    K = np.outer(scores, f64(q)[0, 0]) / D ** 0.5 + 0.1 * rng.standard_normal((L, D))
    tab, blocks = table.cpu().numpy()[0], np.zeros((k_pages.shape[0], 1, page, D))
    blocks[tab[np.arange(L) // page], 0, np.arange(L) % page] = K
    name = code_of(dtype)
    k_pages.copy_(torch.from_numpy(quantised.pack(quantised.rounded(blocks, name), name)))
    return k_pages, v_pages, table, seqlens


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt,large", LARGE[:3] + [("f16", 2048.0)])
@pytest.mark.parametrize("rows", [1, 8, 16])
@pytest.mark.parametrize("at", [3, 450, 896])
def test_a_large_scale_of_a_weight_that_does_not_count(D, dt, large, rows, at):
    """One key's value has a large scale, and its score lies 80 below the others' (a weight of
    2^-115): the row is that of the other keys."""
    dtype, page, L = DT[dt], 16, 900
    q = torch.randn(1, 1, D)
    q = (q * (D ** 0.5 / q.norm())).to(dtype).expand(1, rows, D).contiguous().cuda()
    scores = np.random.default_rng(at).uniform(-3, 3, L)
    scores[at] = -80
    k_pages, v_pages, table, seqlens = with_scores(D, dtype, page, L, scores, q, seed=at)
    for shares in (1, 4):
        set_value(v_pages, page, table[0], at, dtype, large)
        o, _ = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens, num_shares=shares)
        check_rows(o, q, k_pages, v_pages, page, table[0], L)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt,large", LARGE[:3] + [("f16", 2048.0)])
@pytest.mark.parametrize("rows", [1, 8, 16])
@pytest.mark.parametrize("later_first", [False, True])
def test_large_scales_left_behind_by_larger_scores(D, dt, large, rows, later_first):
    """A third of the keys has values of a large scale and scores 70 below those of the
    rest, which come after them (or before)."""
    dtype, page, L = DT[dt], 16, 900
    q = torch.randn(1, 1, D)
    q = (q * (D ** 0.5 / q.norm())).to(dtype).expand(1, rows, D).contiguous().cuda()
    low = np.arange(L) >= 600 if later_first else np.arange(L) < 300
    scores = np.random.default_rng(D).uniform(-3, 3, L) - 70 * low
    k_pages, v_pages, table, seqlens = with_scores(D, dtype, page, L, scores, q, seed=rows)
    for j in np.nonzero(low)[0]:
        set_value(v_pages, page, table[0], int(j), dtype, large)
    for shares in (1, 4):
        o, _ = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens, num_shares=shares)
        check_rows(o, q, k_pages, v_pages, page, table[0], L)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 8, 16])
def test_values_whose_scales_climb_by_a_power_of_two_each_tile(D, dt, rows):
    """Equal scores, and scales from 2^-14 to 2^12 (FP16) or 2^-100 to 2^100: the power of two
    of every row goes down step by step."""
    dtype, page, L = DT[dt], 64, 3000
    lo, hi = (-14, 11) if dt == "f16" else (-100, 100)
    q = torch.randn(1, rows, D).to(dtype).cuda()
    k_pages, v_pages, table, seqlens = make_cache([L], page, 1, D, dtype, seed=rows, spread=0.1)
    for j in range(L):
        set_value(v_pages, page, table[0], j, dtype, 2.0 ** (lo + (hi - lo) * j // L), -8 * 2.0 ** (lo + (hi - lo) * j // L))
    for shares in (1, 5):
        o, _ = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens, num_shares=shares)
        check_rows(o, q, k_pages, v_pages, page, table[0], L)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 8, 16])
@pytest.mark.parametrize("first", [True, False])
def test_small_weights_of_many_keys_count(D, dt, rows, first):
    """Scores 0 but for one key's, 17.625: the others weigh 2^-25.4 each beside its 1, and
    2^-8.4 together.  That key's value is 0 (scale and minimum 0), the others have s = 1 / 16, m = 0,
    so O_d is the others' part times c_d / 16, and the row's largest p s is one of theirs: P s is
    normal in FP16.  The scores are exact.  Scaling by log2(e) and the exponential: under 2^-18 of a
    weight; P s, the same for all of them, has an exact power of two and the exponential's 24
    bits: w = 2^-11 or 2^-21 of it, on products of both signs (c - 8), 8 / 16 at most where O's part is
    c / 16.  Sums: a row's 16 running parts of L / 16 FP32 additions at most, 2^-24 each: L 2^-28;
    the products' L / 16 chopped sums, 2^-23 of 8 / 16: L 2^-28, and of 8 s in the minima's term as many."""
    dtype, page, L = DT[dt], 256, 1 << 17
    table = torch.randperm(L // page, dtype=torch.int32)[None].cuda()
    k_pages, v_pages = binding.q4_pages(L // page, 1, page, D)
    G = quantised.group_of(D)
    part = page * (G // 2 + 4)
    codes = (np.arange(D) * 7) % 16
    packed = torch.tensor(codes[0::2] | codes[1::2] << 4, dtype=torch.uint8, device="cuda")
    for g in range(D // G):
        place = g * part
        v_pages[:, 0, place:place + page * G // 2] = packed[g * G // 2:(g + 1) * G // 2].repeat(page)
        word = torch.tensor(list(quantised.to_bits(np.array([1 / 16, 0.0]), dt).tobytes()), dtype=torch.uint8, device="cuda")
        v_pages[:, 0, place + page * G // 2:place + part] = word.repeat(page)
    at = 7 if first else L - 100
    set_value(k_pages, page, table[0], at, dtype, 0.0, 17.625)  # all D elements; q has one that is not 0
    set_value(v_pages, page, table[0], at, dtype, 0.0, 0.0)
    q = torch.zeros(1, rows, D, dtype=dtype, device="cuda")
    q[..., 0] = 1
    seqlens = torch.tensor([L], dtype=torch.int32, device="cuda")
    for shares in (None, 1):
        o, lse = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens, scale=1.0, num_shares=shares)
        others = (L - 1) * math.exp(-17.625)
        weight = others / (1 + others)
        want = codes / 16 * weight
        u, w = torch.finfo(dtype).eps / 2, 2.0 ** -21 if dt == "f16" else 2.0 ** -11
        bound = u * want + (w + 2.0 ** -17 + 3 * L * 2.0 ** -28) * weight + (2.0 ** -25 if dt == "f16" else 0)
        assert np.all(np.abs(f64(o)[0] - want) <= bound)
        assert float((lse.double() - 17.625 - math.log1p(others)).abs().max()) <= L * 2.0 ** -28 + 2.0 ** -16


# ---------------------------------------------------------------- pages larger than a tile, and the 16-bit cache

@pytest.mark.parametrize("page", [256, 512, 4096])
@pytest.mark.parametrize("n,Hq", [(1, 8), (1, 16), (4, 8), (9, 8)])  # 4, 8, 16 and more rows for either KV head
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_pages_larger_than_a_tile(page, n, Hq, D, dt):
    attend([900, 20, 257, 4200], n, Hq, 2, D, DT[dt], page, "pair", seed=page + n)


@pytest.mark.parametrize("page", [512, 4096])
@pytest.mark.parametrize("n", [1, 3])
def test_windows_over_pages_larger_than_a_tile(page, n):
    for D, dt in ((32, "f16"), (64, "bf16"), (128, "f16")):
        attend([900, 20, 5000], n, 16, 2, D, DT[dt], page, "heads", seed=page, window_left=300)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n,Hq", [(1, 8), (3, 8)])
def test_the_16_bit_cache_of_the_unpacked_values(D, dt, n, Hq):
    """Both calls round their output once (u |O|), and their weights by w (here) and 2^-16 of
    themselves.  The 16-bit cache has values rounded by u, and keys, which move a score by at most
    d = max_j |scale q (k16_j - k_j)|, computed here, and a weight by a factor within e^(2 d).  What
    is left of either call's own bound (scores and sums in FP32) is 2^-14 of the sums for sizes like these."""
    dtype, page, Hkv, lens = DT[dt], 16, 2, [333, 40, n]
    k_pages, v_pages, table, seqlens = make_cache(lens, page, Hkv, D, dtype, seed=D + n)
    q = torch.randn(len(lens) * n, Hq, D).to(dtype).cuda()
    o4, _ = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens)
    k16, v16 = (binding.paged_unpack_q4(p, D, dtype) for p in (k_pages, v_pages))
    o16, _ = binding.attention_paged(q, k16, v16, table, seqlens)
    u, w, scale = torch.finfo(dtype).eps / 2, 2.0 ** -21 if dt == "f16" else 2.0 ** -11, D ** -0.5
    for s, L in enumerate(lens):
        parts = [rows_of(p, page, table[s], L, dtype) for p in (k_pages, v_pages)]
        K, V = (c * np.repeat(a, quantised.group_of(D), -1) + np.repeat(m, quantised.group_of(D), -1) for c, a, m in parts)
        at, slot = table[s].cpu().numpy()[np.arange(L) // page], np.arange(L) % page
        K16 = f64(k16)[at, :, slot].transpose(1, 0, 2)
        for i in range(n):
            keys = L - n + i + 1
            for h in range(Hq):
                hk, Q = h // (Hq // Hkv), f64(q)[s * n + i, h]
                S = K[hk, :keys] @ Q * scale
                d = np.abs((K16[hk, :keys] - K[hk, :keys]) @ Q).max() * scale
                p = np.exp(S - S.max())
                p /= p.sum()
                O, B = p @ V[hk, :keys], p @ np.abs(V[hk, :keys])
                c, a, m = (x[hk, :keys] for x in parts[1])
                a, m = (np.repeat(x, quantised.group_of(D), -1) for x in (a, m))
                own = p @ (a * np.abs(c - 8) + np.abs(m + 8 * a))
                x = np.abs(f64(o4)[s * n + i, h] - f64(o16)[s * n + i, h])
                bound = 2 * u * np.abs(O) + (u + math.expm1(2 * d) + 2.0 ** -14) * 1.01 * B + (w + 2.0 ** -14) * own + 2.0 ** -24
                assert np.all(x <= bound), f"{np.max(x / bound):.2f} of the bound"
