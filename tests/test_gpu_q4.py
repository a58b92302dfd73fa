"""GPU tests of the paged cache held in 4 bits (append, the way back, attention
over it) against the FP64 definitions.

Codes, scales and minima are compared byte by byte: values are stored from 16-bit
numbers by rules without a choice, and keys are computed to 2^-46 before they are
rounded, so a byte could differ from the definition's only where FP64 itself is that
near a tie (none is, for the inputs here).

Bounds for attention, from the arithmetic; u is the output type's half step
(finfo.eps / 2).  For a row, key j and group h with scale s, minimum m and codes c:
  S: a product of q, scaled by a power of two, and a code is exact; D of them and the
     minima's terms are added with chopped bits, each at most 2^-23 of the sum of the
     absolute terms A = scale sum_h (s <|q|, c> + |m| sum |q|); the sums of q take D
     roundings of their own and the scaling by log2(e) a few: ds = (2 D + 16) 2^-23 A.
     Elements of q below 2^-28 of the largest lose bits: 2^-38 max|q| scale sum |k| more.
  P: 2 ds + 2^-21 (the exponential), as in the 16-bit cache's tests.
  P s to FP16: in one part (BF16 outputs) 2^-11 of itself, in two (FP16) 2^-21; below
     the normal range 2^-25 2^-15 of the largest scale's power of two: keys 2^-38 smax 15.
  O: products are chopped within a tile (two keys' worth of 2^-23 each), tiles and parts
     are added in FP32: (32 + keys / 16) 2^-24 of the sums' size at most.
With B = sum_j p_j (s_j c_jd + |m_j|):
    |dO| <= (w + 2 ds + 2^-20 + (32 + keys/16) 2^-24) B + u |O| + 2^-30 keys smax, w = 2^-11 or 2^-21,
  and 2^-25 more for FP16 outputs, whose steps below the normal range are 2^-24,
    |dlse| <= ds + 2^-20 (1 + |lse|)."""

import numpy as np
import pytest
import torch

from exact_tiled_attention_19_gb300 import binding
from oracle import cache, quantised

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _device_status_clean():
    torch.manual_seed(0)
    yield
    assert binding.etattn_read_device_status(clear=True) == 0


def f64(t):
    return t.detach().cpu().double().numpy()


def code_of(dtype):
    return "f16" if dtype == torch.float16 else "bf16"


def blocks_of(pages):
    return pages.cpu().numpy()


def holder(num, Hkv, page, D, layout="pair"):
    """An empty cache: keys and values of a page beside each other, apart, or with the
    heads outside."""
    block = binding.attn_paged_q4_block_bytes(page, D)
    if layout == "pair":
        return binding.q4_pages(num, Hkv, page, D)
    if layout == "heads":
        x = torch.zeros(2, Hkv, num, block, dtype=torch.uint8, device="cuda")
        return x[0].transpose(0, 1), x[1].transpose(0, 1)
    x = torch.zeros(2, num, Hkv, block, dtype=torch.uint8, device="cuda")
    return x[0], x[1]


# ---------------------------------------------------------------- append, and the way back

def check_append(T, Hq, Hkv, D, dtype, page, layout="pair", rope_dim=None, interleaved=False, weighted=True, seed=0,
                 scale=1.5, x=None):
    rope_dim = D if rope_dim is None else rope_dim
    g = torch.Generator().manual_seed(seed)
    num = T // page + 3
    k_pages, v_pages = holder(num, Hkv, page, D, layout)
    for pages in (k_pages, v_pages):  # what was there stays
        pages.copy_(torch.randint(0, 256, pages.shape, generator=g, dtype=torch.uint8))
    before = blocks_of(k_pages), blocks_of(v_pages)
    fused = ((torch.randn(T, Hq + 2 * Hkv, D, generator=g) * scale) if x is None else x).to(dtype).cuda()
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    places = torch.randperm(num * page, generator=g)[:T]
    gone = torch.rand(T, generator=g) < 0.1
    slots = torch.where(gone, -1 - places, places).cuda()
    kw = {}
    if weighted:
        wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2))
        kw.update(q_weight=wq, k_weight=wk)
    if rope_dim:
        cos, sin = binding.rope_tables(5000, rope_dim)
        pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32)
        kw.update(rope_cos=cos, rope_sin=sin, positions=pos.cuda())
    q_out = torch.full((T, Hq, D), 9.0, dtype=dtype, device="cuda")
    got = binding.paged_append_q4(k, v, k_pages, v_pages, slots, q=q if Hq else None, interleaved=interleaved,
                                  q_out=q_out if Hq else None, **kw)
    name = code_of(dtype)
    here = ~gone.numpy()
    if Hq:  # as the call without a cache, and left alone where there is no place
        want, _ = binding.qk_norm_rope(q, k, interleaved=interleaved, **kw)
        assert torch.equal(got[here], want[here]) and bool((got[~here] == 9.0).all())
    else:
        assert got is None
    c64, s64 = (f64(kw["rope_cos"])[pos.numpy()], f64(kw["rope_sin"])[pos.numpy()]) if rope_dim else (None, None)
    wk64 = f64(kw["k_weight"]) if weighted else None
    with np.errstate(invalid="ignore", over="ignore"):
        k64 = quantised.rounded(cache.norm_rope(f64(k), wk64, c64, s64, interleaved, eps=float(np.float32(1e-6))), name)
    for pages, rows, old in ((k_pages, k64, before[0]), (v_pages, f64(v), before[1])):
        now = blocks_of(pages)
        codes, scales, minima = quantised.parts(old, page, D, name)
        G = quantised.group_of(D)
        c, s, m = quantised.quantise(rows.reshape(T, Hkv, -1, G), name)
        at, slot = slots.cpu().numpy()[here] // page, slots.cpu().numpy()[here] % page
        codes[at, :, slot] = c[here].reshape(-1, Hkv, D)
        scales[at, :, slot], minima[at, :, slot] = s[here], m[here]
        gc, gs, gm = quantised.parts(now, page, D, name)
        assert np.array_equal(gc, codes)
        assert np.array_equal(quantised.to_bits(gs, name)[at, :, slot], quantised.to_bits(scales, name)[at, :, slot])
        assert np.array_equal(gm[at, :, slot], minima[at, :, slot], equal_nan=True)  # (zeros of either sign)
        taken = np.zeros((num, page), bool)
        taken[at, slot] = True
        untouched = np.broadcast_to(~taken[:, None], gs.shape[:3])
        raw = [quantised.parts(b, page, D, name)[1:] for b in (old, now)]
        assert all(np.array_equal(x[untouched], y[untouched], equal_nan=True) for x, y in zip(*raw))
    return k_pages, v_pages


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 7, 130, 1500])
def test_append(T, D, dt):
    check_append(T, 8, 2, D, DT[dt], 16, seed=T + D)


@pytest.mark.parametrize("page", [8, 16, 64, 512, 4096])
@pytest.mark.parametrize("layout", ["pair", "apart", "heads"])
@pytest.mark.parametrize("D", [32, 128])
def test_append_pages_and_layouts(page, layout, D):
    check_append(90, 3, 3, D, torch.bfloat16, page, layout, seed=page)


@pytest.mark.parametrize("D,rope_dim", [(32, 0), (32, 16), (64, 16), (64, 48), (128, 0), (128, 32), (128, 64), (128, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_append_parts_rotated(D, rope_dim, interleaved, weighted):
    for T in (5, 700):
        check_append(T, 4, 2, D, torch.float16, 16, rope_dim=rope_dim, interleaved=interleaved, weighted=weighted, seed=T)


@pytest.mark.parametrize("Hq,Hkv", [(0, 1), (0, 8), (1, 1), (5, 5), (17, 17), (40, 8)])
def test_append_heads(Hq, Hkv):
    for T in (3, 400):
        check_append(T, Hq, Hkv, 64, torch.bfloat16, 32, seed=Hq)


@pytest.mark.parametrize("D,dt,Hq,Hkv,T,rope_dim,interleaved", [
    (128, "bf16", 35, 5, 2700, 128, False), (128, "f16", 16, 8, 4000, 96, True), (128, "bf16", 0, 4, 15000, 0, False),
    (128, "f16", 8, 1, 12000, 128, True), (64, "bf16", 40, 5, 4800, 48, False), (64, "f16", 0, 17, 7000, 64, True),
    (32, "bf16", 32, 8, 10000, 32, False), (32, "f16", 17, 17, 9300, 16, False)])
def test_append_many_tokens(D, dt, Hq, Hkv, T, rope_dim, interleaved):
    """More than 7296 blocks of one head each, where a thread takes several heads."""
    assert T * (Hq + 2 * Hkv) > 7296 * 128 // (D // 16)
    check_append(T, Hq, Hkv, D, DT[dt], 16, rope_dim=rope_dim, interleaved=interleaved, weighted=rope_dim > 0, seed=T)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_append_values_where_rounding_decides(dt, D):
    """Whole numbers and halves of them, so that very many quotients are ties; constant
    groups; spreads from denormals to the type's largest numbers."""
    g = torch.Generator().manual_seed(D)
    T, H = 60, 6
    x = torch.randint(-30, 31, (T, H, D), generator=g).float() / 2
    x[5:9] = x[5:9, :, :1]
    x[9:12] = 0
    x[12:16] = x[12:16].round() * torch.finfo(DT[dt]).tiny / 4
    x[16:18] *= torch.finfo(DT[dt]).max / 40
    x[18:22, :, 1:] = 100.0
    if dt == "bf16":
        x[22:25] *= 2.0 ** -120
        x[25:27] = x[25:27].sign() * 3e38  # the spread passes FP32: reads as NaN
    check_append(T, 2, 2, D, DT[dt], 16, rope_dim=0, weighted=False, x=x, seed=1)


def test_groups_with_infinities_and_nan_read_as_nan():
    x = torch.randn(8, 6, 128)
    x[1, 2, 3], x[2, 4, 100], x[3, 3, 64], x[4, 5, 0] = float("inf"), float("-inf"), float("nan"), float("nan")
    k_pages, v_pages = check_append(8, 2, 2, 128, torch.bfloat16, 8, rope_dim=0, weighted=False, x=x)
    got = torch.cat([binding.paged_unpack_q4(p, 128, torch.bfloat16) for p in (k_pages, v_pages)])
    assert bool(got.isnan().any())


def test_bad_slots_and_positions_are_skipped_and_recorded():
    k_pages, v_pages = binding.q4_pages(4, 2, 16, 64)
    k = torch.randn(5, 2, 64).half().cuda()
    cos, sin = binding.rope_tables(10, 64)
    q = torch.randn(5, 4, 64).half().cuda()

    def run(slots, positions):
        k_pages.fill_(255), v_pages.fill_(255)
        out = torch.full_like(q, 9.0)
        binding.paged_append_q4(k, k, k_pages, v_pages, torch.tensor(slots).cuda(), q=q, q_out=out, rope_cos=cos,
                                rope_sin=sin, positions=torch.tensor(positions, dtype=torch.int32).cuda())
        rows = [bool((out[t] != 9.0).any()) for t in range(5)]
        slots_written = (quantised.parts(blocks_of(v_pages), 16, 64, "f16")[0][:, 0, :, 0] != 15) | \
            (quantised.parts(blocks_of(v_pages), 16, 64, "f16")[0][:, 0].min(-1) != 15)
        return rows, sorted(zip(*(x.tolist() for x in np.nonzero(slots_written))))

    rows, there = run([0, 63, 17, 5, -1], [0, 9, 3, 4, 99])
    assert rows == [True] * 4 + [False] and there == [(0, 0), (0, 5), (1, 1), (3, 15)]
    assert binding.etattn_read_device_status(clear=True) == 0  # (a token without a place needs no position)
    for slots, positions in (([0, 64, 17, 5, 2], [0] * 5), ([0, 2 ** 40, 17, 5, 2], [0] * 5),
                             ([0, 1, 17, 5, 2], [0, 10, 0, 0, 0]), ([0, 1, 17, 5, 2], [0, -1, 0, 0, 0])):
        rows, there = run(slots, positions)
        assert rows == [True, False, True, True, True] and len(there) == 4
        assert binding.etattn_read_device_status(clear=True) == 13


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [32, 128])
def test_the_types_largest_numbers_read_as_finite(dt, D):
    big = torch.finfo(DT[dt]).max
    x = torch.rand(8, 2, D, dtype=torch.float64)  # from 0 to the largest number: spreads within FP32
    x[:, :, 1::9] = 1.0
    x[0], x[1, :, 1:], x[2] = 1.0, 0.0, -1.0
    x[3] -= 1.0
    if dt == "f16":
        x[4] = x[4] * 2 - 1
    x = (x * big).to(DT[dt]).cuda()
    k_pages, v_pages = binding.q4_pages(1, 2, 8, D)
    binding.paged_append_q4(x, x, k_pages, v_pages, torch.arange(8).cuda())
    for pages in (k_pages, v_pages):
        got = f64(binding.paged_unpack_q4(pages, D, DT[dt])[0]).transpose(1, 0, 2)
        assert np.array_equal(got, quantised.rounded(quantised.stored(f64(x), code_of(DT[dt])), code_of(DT[dt])))
        assert np.all(np.isfinite(got)) and np.abs(got - f64(x)).max() <= 0.05 * big * (2 if dt == "f16" else 1)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("page,layout", [(8, "pair"), (16, "heads"), (256, "apart")])
def test_unpack_is_the_value_rounded(D, dt, page, layout):
    rng = np.random.default_rng(page)
    k_pages, _ = holder(5, 3, page, D, layout)
    x = quantised.rounded(rng.standard_normal((5, 3, page, D)) * 3, dt)
    k_pages.copy_(torch.from_numpy(quantised.pack(x, dt)))
    want = quantised.rounded(quantised.stored(x, dt), dt)
    assert np.array_equal(f64(binding.paged_unpack_q4(k_pages, D, DT[dt])), want)
    out = torch.zeros(5, page, 3, D, dtype=DT[dt], device="cuda").permute(0, 2, 1, 3)  # token-major storage
    assert binding.paged_unpack_q4(k_pages, D, DT[dt], out=out) is out
    assert np.array_equal(f64(out), want)


# ---------------------------------------------------------------- attention

def make_cache(lens, page, Hkv, D, dtype, layout="pair", seed=0, spare=3, spread=1.0, offset=0.0):
    """Pages with random contents, a shuffled block table, and the lengths."""
    rng = np.random.default_rng(seed)
    need = [-(-L // page) for L in lens]
    pool = sum(need) + spare
    order = rng.permutation(pool)
    table = np.full((len(lens), max(max(need), 1)), -1)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    pages = []
    for empty in holder(pool, Hkv, page, D, layout):
        x = rng.standard_normal((pool, Hkv, page, D)) * spread + offset
        empty.copy_(torch.from_numpy(quantised.pack(quantised.rounded(x, code_of(dtype)), code_of(dtype))))
        pages.append(empty)
    return pages[0], pages[1], torch.from_numpy(table).int().cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def check_attention(o, lse, q, k_pages, v_pages, page, table, lens, cu, causal=True, wl=-1, wr=-1, scale=None):
    dtype, D, T = q.dtype, q.shape[2], q.shape[0]
    scale = D ** -0.5 if scale is None else scale
    name, G = code_of(dtype), quantised.group_of(q.shape[2])
    q64, go, gl, tab = f64(q), f64(o), f64(lse), table.cpu().numpy()
    group = q.shape[1] // k_pages.shape[1]
    u = torch.finfo(dtype).eps / 2
    w, least = (2.0 ** -21, 2.0 ** -25) if dtype == torch.float16 else (2.0 ** -11, 1e-30)
    kb, vb = (quantised.parts(blocks_of(p), page, D, name) for p in (k_pages, v_pages))
    wl, wr = (1 << 30 if wl < 0 else wl), (0 if causal else 1 << 30 if wr < 0 else wr)
    for s, L in enumerate(lens):
        a, b = cu[s], cu[s + 1]
        n = b - a
        if n == 0:
            continue
        at, slot = tab[s, np.arange(L) // page], np.arange(L) % page
        kc, ks, km = (x[at, :, slot].transpose(1, 0, 2) for x in kb)  # [Hkv, L, D or D / G]
        vc, vs, vm = (x[at, :, slot].transpose(1, 0, 2) for x in vb)
        wide = lambda x: np.repeat(x, G, -1)  # noqa: E731
        c = np.arange(n) + L - n
        key = np.arange(L)
        seen = (key >= c[:, None] - wl) & (key <= c[:, None] + wr)      # [n, L]
        for hk in range(k_pages.shape[1]):
            any_seen = seen.any(0)
            K = np.where(any_seen[:, None], kc[hk] * wide(ks[hk]) + wide(km[hk]), 0)
            V = np.where(any_seen[:, None], vc[hk] * wide(vs[hk]) + wide(vm[hk]), 0)
            KA = np.where(any_seen[:, None], kc[hk] * wide(ks[hk]) + np.abs(wide(km[hk])), 0)
            VA = np.where(any_seen[:, None], vc[hk] * wide(vs[hk]) + np.abs(wide(vm[hk])), 0)
            smax = np.where(any_seen[:, None], vs[hk], 0).max() if L else 0.0
            for h in range(hk * group, (hk + 1) * group):
                Q = q64[a:b, h]
                S = np.where(seen, Q @ K.T * scale, -np.inf)
                A = np.where(seen, np.abs(Q) @ KA.T * scale, 0)
                tiny = 2.0 ** -38 * np.abs(Q).max(-1) * scale * np.abs(K).sum(-1).max(initial=0)
                ds = (2 * D + 16) * 2.0 ** -23 * A.max(-1, initial=0) + tiny
                m = S.max(-1, initial=-np.inf)
                e = np.exp(S - np.where(np.isneginf(m), 0, m)[:, None])
                z = e.sum(-1)
                empty = z == 0
                P = e / np.where(empty, 1, z)[:, None]
                ro, rb = P @ V, P @ VA
                rl = np.where(empty, -np.inf, m + np.log(np.where(empty, 1, z)))
                assert np.array_equal(np.isneginf(gl[h, a:b]), empty) and np.all(go[a:b, h][empty] == 0)
                x = np.abs(np.where(empty, 0, gl[h, a:b] - np.where(empty, 0, rl)))
                bound = ds + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, rl)))
                assert np.all(x <= bound), f"lse of sequence {s}, head {h}: {np.max(x / bound):.2f} of the bound"
                keys = seen.sum(-1)[:, None]
                bound = ((w + 2 * ds[:, None] + 2.0 ** -20 + (32 + keys / 16) * 2.0 ** -24) * rb + u * np.abs(ro)
                         + 2.0 ** -30 * keys * smax + least)
                x = np.abs(go[a:b, h] - ro)
                assert np.all(x <= bound), f"O of sequence {s}, head {h}: {np.max(x / bound):.2f} of the bound"


def attend(lens, n, Hq, Hkv, D, dtype, page, layout="pair", seed=0, shares=None, cu=None, q_scale=1.0, spread=1.0,
           offset=0.0, **kw):
    k_pages, v_pages, table, seqlens = make_cache(lens, page, Hkv, D, dtype, layout, seed, spread=spread, offset=offset)
    g = torch.Generator().manual_seed(seed + 100)
    S = len(lens)
    ragged = cu is not None
    cu = cu if ragged else [n * i for i in range(S + 1)]
    q = (torch.randn(cu[-1], Hq, D, generator=g) * q_scale).to(dtype).cuda()
    extra = dict(cu_seqlens_q=torch.tensor(cu, dtype=torch.int32).cuda(),
                 max_seqlen_q=max(b - a for a, b in zip(cu, cu[1:]))) if ragged else {}
    o, lse = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens, num_shares=shares, **extra, **kw)
    check_attention(o, lse, q, k_pages, v_pages, page, table, lens, cu, causal=kw.get("causal", True),
                    wl=kw.get("window_left", -1), wr=kw.get("window_right", -1), scale=kw.get("scale"))
    return o, lse


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 127, 128, 129, 255, 257, 700])
def test_one_sequence_lengths(D, dt, L):
    attend([L], 1, 4, 2, D, DT[dt], 16, seed=L + D)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 512, 4096])
@pytest.mark.parametrize("layout", ["pair", "apart", "heads"])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_page_sizes_and_layouts(page, layout, D):
    attend([300, 5, 64, 1057], 1, 8, 2, D, torch.bfloat16, page, layout, seed=page)


@pytest.mark.parametrize("shares", [1, 2, 3, 7, 16, 50, 456, 1000])
def test_any_number_of_shares(shares):
    attend([1000, 1, 130, 0, 64, 500], 1, 6, 3, 128, torch.bfloat16, 32, seed=shares, shares=shares)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (5, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 1), (32, 8), (6, 2)])
@pytest.mark.parametrize("D,dt", [(32, "bf16"), (64, "f16"), (128, "f16"), (128, "bf16")])
def test_head_groups(Hq, Hkv, D, dt):
    attend([333, 90], 1, Hq, Hkv, D, DT[dt], 16, seed=Hq)


@pytest.mark.parametrize("n", [2, 3, 4, 8, 13])
@pytest.mark.parametrize("page", [8, 32, 64])
@pytest.mark.parametrize("D,dt", [(32, "f16"), (64, "bf16"), (128, "bf16")])
def test_several_new_tokens(n, page, D, dt):
    attend([400, n, 77, 260], n, 8, 2, D, DT[dt], page, seed=n + page)


@pytest.mark.parametrize("kw", [dict(window_left=0), dict(window_left=17), dict(window_left=300),
                                dict(causal=False), dict(causal=False, window_left=20, window_right=3),
                                dict(causal=False, window_right=0), dict(scale=2.5), dict(scale=1e-3)])
@pytest.mark.parametrize("n,page", [(1, 16), (5, 16), (3, 64)])
def test_masks_and_scales(kw, n, page):
    attend([500, 64, 129, 31], n, 4, 2, 128, torch.bfloat16, page, seed=n, **kw)


@pytest.mark.parametrize("kw", [dict(window_left=0), dict(window_left=17), dict(window_left=300),
                                dict(causal=False, window_left=20, window_right=3), dict(causal=False)])
@pytest.mark.parametrize("n,Hq,Hkv", [(1, 8, 2), (2, 4, 2), (4, 2, 2), (3, 1, 1)])
@pytest.mark.parametrize("D,dt,page", [(32, "f16", 8), (64, "bf16", 64), (64, "f16", 16), (128, "f16", 16)])
def test_masks_of_up_to_four_rows(kw, n, Hq, Hkv, D, dt, page):
    attend([700, 64, 129, 260, n], n, Hq, Hkv, D, DT[dt], page, seed=n, **kw)


def test_ragged_new_tokens_and_empty_rows():
    # No new token; more new tokens than keys (rows without a key); no keys at all.
    attend([40, 300, 3, 0, 150], None, 8, 2, 64, torch.float16, 16, cu=[0, 0, 3, 8, 9, 11], seed=3)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("spread,offset", [(1e-6, 0.0), (3e3, 0.0), (0.5, 40.0), (0.0, 1.0)])
def test_scales_and_offsets(dt, spread, offset):
    attend([700, 65], 1, 4, 2, 128, DT[dt], 16, seed=5, spread=spread, offset=offset, q_scale=1e-3 if spread > 1 else 1.0)


@pytest.mark.parametrize("q_scale", [1e-30, 1e-3, 30.0, 1e4])
def test_queries_of_any_size(q_scale):
    attend([300], 1, 4, 2, 64, torch.bfloat16, 16, seed=6, q_scale=q_scale, scale=0.125 / max(q_scale, 1e-20))


def test_scales_of_values_that_grow_and_shrink():
    """Values whose scales rise by 2^40 along the sequence, and fall again: what a small
    one leaves beside a large one is below the bound, and nothing overflows."""
    L, page, D = 900, 16, 128
    rng = np.random.default_rng(0)
    k_pages, v_pages, table, seqlens = make_cache([L], page, 1, D, torch.bfloat16, seed=1)
    x = rng.standard_normal((1, L, D)) * 2.0 ** (40 - np.abs(np.arange(L) - 450) / 450 * 40)[None, :, None]
    x[..., 64:] *= 2.0 ** -30  # the groups' scales are apart
    tab, blocks = table.cpu().numpy()[0], np.zeros((v_pages.shape[0], 1, page, D))
    for j in range(L):
        blocks[tab[j // page], 0, j % page] = x[0, j]
    v_pages.copy_(torch.from_numpy(quantised.pack(quantised.rounded(blocks, "bf16"), "bf16")))
    q = torch.randn(1, 4, D).bfloat16().cuda()
    for shares in (1, 5):
        o, lse = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens, num_shares=shares)
        kc, vc = (quantised.unpack(blocks_of(p), page, D, "bf16")[tab[np.arange(L) // page], 0, np.arange(L) % page]
                  for p in (k_pages, v_pages))
        S = f64(q)[0] @ kc.T / D ** 0.5
        P = np.exp(S - S.max(-1, keepdims=True))
        P /= P.sum(-1, keepdims=True)
        ro, rb = P @ vc, P @ np.abs(vc)
        assert np.all(np.abs(f64(o)[0] - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -9 * rb)


@pytest.mark.parametrize("n,Hq,Hkv", [(3, 24, 2), (7, 5, 1), (50, 36, 3), (9, 48, 1), (130, 8, 8), (2, 2, 1)])
@pytest.mark.parametrize("D,dt", [(32, "bf16"), (64, "f16"), (128, "bf16")])
def test_row_tiles_across_tokens_of_any_group(n, Hq, Hkv, D, dt):
    attend([n + 200, n, 301], n, Hq, Hkv, D, DT[dt], 16, seed=n + D)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("n", [1, 5])
def test_values_whose_scales_are_near_the_types_largest(D, n):
    """Scales of 2^112 and more: the power of two that takes them to FP16, times that
    of the codes, passes FP32."""
    lens, page = [100, 20], 16
    k_pages, _, table, seqlens = make_cache(lens, page, 2, D, torch.bfloat16, seed=2)
    _, v_pages, _, _ = make_cache(lens, page, 2, D, torch.bfloat16, seed=2, spread=4e34)
    assert quantised.parts(blocks_of(v_pages), page, D, "bf16")[1].max() > 2.0 ** 113
    q = torch.randn(2 * n, 8, D).bfloat16().cuda()
    for shares in (1, 3):
        o, lse = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens, num_shares=shares)
        assert bool(o.isfinite().all())
        check_attention(o, lse, q, k_pages, v_pages, page, table, lens, [0, n, 2 * n])


@pytest.mark.parametrize("page", [8, 32, 128])
@pytest.mark.parametrize("n", [1, 2, 6])
def test_nothing_outside_a_rows_keys_reaches_it(page, n):
    """Slots past the end, pages before the window and a key that only later rows read
    hold NaN and infinite scales."""
    for D, dt in ((64, "f16"), (128, "bf16")):
        lens = [200, 77, 140]
        kw = dict(window_left=50)
        k_pages, v_pages, table, seqlens = make_cache(lens, page, 2, D, DT[dt], seed=page + n)
        q = torch.randn(3 * n, 8, D, generator=torch.Generator().manual_seed(n)).to(DT[dt]).cuda()
        want = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens, **kw)
        cu = [0, n, 2 * n, 3 * n]
        check_attention(*want, q, k_pages, v_pages, page, table, lens, cu, wl=50)
        tab = table.cpu().numpy()
        for bits in (0x7fff, 0x7c00 if dt == "f16" else 0x7f80, 0x7bff):
            kp, vp = k_pages.clone(), v_pages.clone()
            for pages in (kp, vp):
                b = blocks_of(pages)
                G, H = quantised.group_of(D), D // quantised.group_of(D)
                part = page * (G // 2 + 4)
                free = np.ones((b.shape[0], page), bool)
                for s, L in enumerate(lens):
                    for j in range(max(0, L - n - 50), L):
                        free[tab[s, j // page], j % page] = False
                for h in range(H):
                    sm = b[..., h * part + page * G // 2:(h + 1) * part].reshape(b.shape[0], 2, page, 4)
                    sm[np.broadcast_to(free[:, None], sm.shape[:3])] = np.frombuffer(np.uint16([bits, 0xfc00]).tobytes(), np.uint8)
                    b[..., h * part + page * G // 2:(h + 1) * part] = sm.reshape(b.shape[0], 2, page * 4)
                pages.copy_(torch.from_numpy(b))
            got = binding.attention_paged_q4(q, kp, vp, table, seqlens, **kw)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_a_key_that_only_later_tokens_read(dt):
    """NaN in the last key: the rows of earlier tokens are as without it, those of the
    last one NaN."""
    D, page, L, n = 128, 16, 130, 4
    k_pages, v_pages, table, seqlens = make_cache([L], page, 2, D, DT[dt], seed=8)
    q = torch.randn(n, 8, D).to(DT[dt]).cuda()
    want, want_lse = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens)
    at, slot = int(table[0, (L - 1) // page]), (L - 1) % page
    for which in (0, 1):
        pages = [k_pages.clone(), v_pages.clone()]
        for h in range(2):
            place = h * page * 36 + page * 32 + slot * 4
            pages[which][at, :, place:place + 4] = torch.tensor([255, 127, 255, 127], dtype=torch.uint8, device="cuda")
        o, lse = binding.attention_paged_q4(q, *pages, table, seqlens)
        assert torch.equal(o[:3], want[:3]) and torch.equal(lse[:, :3], want_lse[:, :3])
        assert bool(o[3].isnan().all())


def test_bad_lengths_and_pages_are_recorded():
    k_pages, v_pages, table, seqlens = make_cache([60, 50, 40], 16, 2, 64, torch.bfloat16, seed=13)
    q = torch.randn(3, 4, 64).bfloat16().cuda()
    ref, _ = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens)

    def run(table=table, seqlens=seqlens):
        out = torch.full((3, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens, out=out)
        return out, binding.etattn_read_device_status(clear=True)

    for bad in (-1, 65):  # (four pages of 16 a row)
        lens = seqlens.clone()
        lens[1] = bad
        out, code = run(seqlens=lens)
        assert code == 9 and bool((out[1] == 9.0).all()) and torch.equal(out[[0, 2]], ref[[0, 2]])
    for bad in (-1, k_pages.shape[0], 2 ** 31 - 1):
        tab = table.clone()
        tab[1, 2] = bad
        out, code = run(table=tab)
        assert code == 13 and torch.equal(out[[0, 2]], ref[[0, 2]])


def test_caches_past_32_bit_offsets():
    """Pages at the end of a cache of more than 2^32 bytes: what is appended there is
    what attention and the way back read."""
    page, Hkv, D = 128, 8, 128
    block = binding.attn_paged_q4_block_bytes(page, D)
    pool = (1 << 32) // (block * Hkv) + 9
    k_pages, v_pages = (torch.empty(pool, Hkv, block, dtype=torch.uint8, device="cuda") for _ in range(2))
    lens = [300, 129]
    table = torch.tensor([[pool - 1, pool - 4, pool - 2], [pool - 3, 0, -1]], dtype=torch.int32).cuda()
    seqlens = torch.tensor(lens, dtype=torch.int32).cuda()
    pos = torch.cat([torch.arange(L) for L in lens])
    seq = torch.tensor([0] * 300 + [1] * 129)
    slots = table.cpu()[seq, pos // page].long() * page + pos % page
    k, v = (torch.randn(429, Hkv, D).bfloat16().cuda() for _ in range(2))
    binding.paged_append_q4(k, v, k_pages, v_pages, slots.cuda())
    q = torch.randn(2, Hkv, D).bfloat16().cuda()
    o, lse = binding.attention_paged_q4(q, k_pages, v_pages, table, seqlens)
    used = torch.tensor([pool - 1, pool - 4, pool - 2, pool - 3, 0], device="cuda")
    kp, vp = k_pages[used].contiguous(), v_pages[used].contiguous()
    at = torch.tensor([[0, 1, 2], [3, 4, -1]], dtype=torch.int32)
    check_attention(o, lse, q, kp, vp, page, at, lens, [0, 1, 2])
    got = binding.paged_unpack_q4(k_pages[pool - 5:], D, torch.bfloat16)
    want = quantised.rounded(quantised.stored(f64(k), "bf16"), "bf16")
    assert np.array_equal(f64(got[4, :, 5]), want[5]) and np.array_equal(f64(got[2, :, 0]), want[300])


# ---------------------------------------------------------------- the step as a user runs it

@pytest.mark.parametrize("D,dt,page", [(64, "f16", 8), (128, "bf16", 16)])
def test_serving_steps_eager_and_captured(D, dt, page):
    """Prompts, decode steps, rejected drafts and a request that ends: pages handed out,
    keys and values appended, attention over them.  The same steps over a 16-bit cache of
    the unpacked values; and decode steps replayed from one graph give what eager ones give."""
    dtype, S, Hq, Hkv, pool, width = DT[dt], 4, 8, 2, 64, 20
    g = torch.Generator().manual_seed(D)
    cos, sin = binding.rope_tables(width * page, D)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2))
    norm = dict(q_weight=wq, k_weight=wk, rope_cos=cos, rope_sin=sin)
    k_pages, v_pages = binding.q4_pages(pool, Hkv, page, D)
    table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    free, count = torch.randperm(pool, generator=g).int().cuda(), torch.tensor([pool], dtype=torch.int32, device="cuda")

    def step(new, fused, T):
        _, cu, pos, slots, _ = binding.paged_extend(new, lens, table, free, count, page_size=page, total_tokens=T,
                                                    seqlens_out=lens, free_count_out=count)
        q = binding.paged_append_q4(fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:], k_pages, v_pages, slots,
                                    q=fused[:, :Hq], positions=pos, q_out=torch.zeros(T, Hq, D, dtype=dtype, device="cuda"),
                                    **norm)
        o, lse = binding.attention_paged_q4(q, k_pages, v_pages, table, lens, cu_seqlens_q=cu, max_seqlen_q=T,
                                            max_seqlen_k=width * page, out=torch.zeros_like(q))
        return q, o, lse, cu

    def inputs(T):
        return torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda()

    for new, T in (([37, 5, 0, 90], 140), ([1, 1, 0, 1], 4), ([3, 2, 17, 4], 26)):
        q, o, lse, cu = step(torch.tensor(new, dtype=torch.int32).cuda(), inputs(T), T)
        total = int(cu[-1])
        assert total == sum(new)
        check_attention(o[:total], lse[:, :total], q[:total], k_pages, v_pages, page, table, lens.tolist(), cu.tolist())
        assert not o[total:].any()  # rows of no sequence
        wide = [binding.paged_unpack_q4(p, D, dtype) for p in (k_pages, v_pages)]
        o16, lse16 = binding.attention_paged(q, *wide, table, lens, cu_seqlens_q=cu, max_seqlen_q=T)
        near = 4 * torch.finfo(dtype).eps * (1 + wide[1].abs().max().item())
        assert (o16[:total] - o[:total]).abs().max().item() <= near * 8
    keep = lens - torch.tensor([2, 0, 17, 3], dtype=torch.int32).cuda()
    binding.paged_truncate(keep, lens, table, free, count, page_size=page, seqlens_out=lens, free_count_out=count)
    held = [-(-int(x) // page) for x in lens]
    assert int(count) == pool - sum(held)

    # Decode steps: eager on a copy of the state, then the same from a graph.
    state = [lens, table, free, count, k_pages, v_pages]
    start = [x.clone() for x in state]
    ones, tokens = torch.ones(S, dtype=torch.int32).cuda(), [inputs(S) for _ in range(2 * page)]
    eager = [step(ones, x, S)[1:3] for x in tokens]
    after = [x.clone() for x in state]
    for x, y in zip(state, start):
        x.copy_(y)
    fused = torch.empty_like(tokens[0])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            _, o, lse, _ = step(ones, fused, S)
        for x, (eo, el) in zip(tokens, eager):
            fused.copy_(x)
            graph.replay()
            stream.synchronize()
            assert torch.equal(o, eo) and torch.equal(lse, el)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(state, after))


def test_two_calls_at_once_on_two_streams():
    k_pages, v_pages, table, seqlens = make_cache([900, 40, 333], 16, 4, 128, torch.bfloat16, seed=21)
    q = torch.randn(2, 3, 8, 128).bfloat16().cuda()
    want = [binding.attention_paged_q4(q[i], k_pages, v_pages, table, seqlens) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[binding.attention_paged_q4(q[i], k_pages, v_pages, table, seqlens, stream=streams[i]) for i in range(2)]
           for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for (o, lse), (wo, wl) in zip(pair, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)
