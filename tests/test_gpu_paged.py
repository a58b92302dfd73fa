"""GPU tests of the paged cache (append, attention over it) against the FP64
oracle.

Bounds for attention, from the arithmetic; u is the type's half step
(finfo.eps / 2).  A score is a sum of D exact products in FP32, at most
ds = 2 D 2^-24 max_j sum_d |q_d k_jd| * scale off (a step per addition, chopped
additions allowed), plus 2^-22 of itself in the scaling by log2(e); a weight
moves by twice that in relative terms, and by 2^-21 in the exponential.
Rounding the weights to the input type adds u, and in FP16, below the normal
range, 2^-25 absolute against a sum of at least 1.  Rounding O adds u |O|.
So with A = sum_j p_j |v_j|:
    |dO| <= (u + 2 ds + 2^-20) A + u |O| + 2^-25 keys max|v| (FP16),
    |dlse| <= ds + 2^-20 (1 + |lse|)."""

import numpy as np
import pytest
import torch

from exact_tiled_attention_19_gb300 import binding
from exact_tiled_attention_19_gb300 import workloads as W
from oracle import cache
from tests.test_gpu_rope import check_forward, f64, half_step

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert binding.etattn_read_device_status(clear=True) == 0


def make_cache(lens, page, Hkv, D, dtype, layout="hnd", seed=0, spare=3, fill=None):
    """Pages with random contents, a shuffled block table, and the lengths."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-L // page) for L in lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=g)
    width = max(max(need), 1)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n].to(torch.int32)
        at += n
    pages = []
    for _ in range(2):
        x = torch.randn(pool, Hkv, page, D, generator=g)
        if fill is not None:  # what no sequence owns
            used = torch.zeros(pool, page, dtype=torch.bool)
            for s, L in enumerate(lens):
                for j in range(L):
                    used[int(table[s, j // page]), j % page] = True
            x = torch.where(used[:, None, :, None], x, torch.tensor(fill))
        x = x.to(dtype)
        if layout == "nhd":
            x = x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
        elif layout == "pair":  # keys and values interleaved in one buffer
            x = x.cuda()
        else:
            x = x.cuda()
        pages.append(x)
    if layout == "pair":
        buf = torch.stack([p.permute(0, 2, 1, 3) for p in pages], 1)  # [pages, 2, slot, head, d]
        pages = [buf[:, i].permute(0, 2, 1, 3) for i in range(2)]
    return pages[0], pages[1], table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def check_attention(o, lse, q, k_pages, v_pages, table, lens, cu, causal=True, wl=-1, wr=-1, scale=None):
    dtype, D = q.dtype, q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    q64, k64, v64 = f64(q), f64(k_pages), f64(v_pages)
    tab = table.cpu().numpy()
    kw = dict(causal=causal, scale=scale, window_left=wl, window_right=wr)
    ro, rl = cache.attention_paged(q64, k64, v64, tab, lens, cu, **kw)
    ra, _ = cache.attention_paged(q64, k64, np.abs(v64), tab, lens, cu, **kw)
    go, gl = f64(o), f64(lse)
    group = q.shape[1] // k_pages.shape[1]
    u = half_step(dtype)
    for s, L in enumerate(lens):
        a, b = cu[s], cu[s + 1]
        if a == b:
            continue
        empty = np.isneginf(rl[:, a:b])
        assert np.array_equal(np.isneginf(gl[:, a:b]), empty)
        assert np.all(go[a:b][empty.T] == 0)
        if L == 0:
            continue
        K, V = cache.gather(k64, tab[s], L), cache.gather(v64, tab[s], L)
        K, V = (np.repeat(np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0), group, axis=0) for x in (K, V))
        mags = np.einsum("thd,hjd->htj", np.abs(q64[a:b]), np.abs(K)).max(-1) * scale   # [Hq, n]
        ds = 2 * D * 2.0 ** -24 * mags + 2.0 ** -22 * mags
        lse_bound = ds + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, rl[:, a:b])))
        err = np.abs(np.where(empty, 0, gl[:, a:b] - np.where(empty, 0, rl[:, a:b])))
        assert np.all(err <= lse_bound), f"lse of sequence {s}: {np.max(err / lse_bound):.2f} of the bound"
        sub = L * 2.0 ** -25 * np.abs(V).max() if dtype == torch.float16 else 1e-30
        bound = (u + 2 * ds.T[:, :, None] + 2.0 ** -20) * ra[a:b] + u * np.abs(ro[a:b]) + sub
        err = np.abs(go[a:b] - ro[a:b])
        assert np.all(err <= bound), f"O of sequence {s}: {np.max(err / bound):.2f} of the bound"


def attend(lens, n, Hq, Hkv, D, dtype, page, layout="hnd", seed=0, shares=None, fill=None, cu=None, q_scale=1.0, **kw):
    k_pages, v_pages, table, seqlens = make_cache(lens, page, Hkv, D, dtype, layout, seed, fill=fill)
    g = torch.Generator().manual_seed(seed + 100)
    S = len(lens)
    ragged = cu is not None
    cu = cu if ragged else [n * i for i in range(S + 1)]
    q = (torch.randn(cu[-1], Hq, D, generator=g) * q_scale).to(dtype).cuda()
    extra = dict(cu_seqlens_q=torch.tensor(cu, dtype=torch.int32).cuda(),
                 max_seqlen_q=max(b - a for a, b in zip(cu, cu[1:]))) if ragged else {}
    o, lse = binding.attention_paged(q, k_pages, v_pages, table, seqlens, num_shares=shares, **extra, **kw)
    check_attention(o, lse, q, k_pages, v_pages, table, lens, cu, causal=kw.get("causal", True),
                    wl=kw.get("window_left", -1), wr=kw.get("window_right", -1), scale=kw.get("scale"))
    return o, lse


@pytest.mark.parametrize("D,dt", [(32, "f16"), (64, "bf16"), (64, "f16"), (128, "bf16"), (128, "f16"), (32, "bf16")])
@pytest.mark.parametrize("L", [1, 2, 63, 64, 65, 129, 700])
def test_one_sequence_lengths(D, dt, L):
    attend([L], 1, 4, 2, D, DT[dt], 16, seed=L + D)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "pair"])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_page_sizes_and_layouts(page, layout, D):
    attend([300, 5, 64, 257], 1, 8, 2, D, torch.bfloat16, page, layout, seed=page)


@pytest.mark.parametrize("shares", [1, 2, 3, 7, 16, 50, 304, 1000])
def test_any_number_of_shares(shares):
    attend([1000, 1, 130, 0, 64, 500], 1, 6, 3, 128, torch.bfloat16, 32, "nhd", seed=shares, shares=shares)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (5, 1), (7, 1), (16, 1), (17, 1), (40, 1), (32, 8), (6, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_head_groups(Hq, Hkv, D):
    attend([333, 90], 1, Hq, Hkv, D, torch.float16, 16, seed=Hq)


@pytest.mark.parametrize("n", [2, 3, 8, 20, 70])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "f16"), (32, "bf16")])
def test_several_new_tokens(n, causal, D, dt):
    attend([200, n, 75 + n], n, 4, 2, D, DT[dt], 16, seed=n, causal=causal)


@pytest.mark.parametrize("wl,wr,causal", [(0, -1, True), (10, -1, True), (63, -1, True), (200, -1, True), (40, 3, False),
                                          (-1, 0, False), (0, 0, False), (100000, -1, True)])
@pytest.mark.parametrize("n", [1, 5])
def test_windows(wl, wr, causal, n):
    attend([700, 40, n, 129], n, 4, 2, 64, torch.bfloat16, 16, seed=wl + 7, window_left=wl, window_right=wr,
           causal=causal)


def test_ragged_new_tokens_and_rows_without_keys():
    """Sequences with no new token, with more new tokens than keys (rows before
    the first key are empty), and an unused slot (no keys)."""
    attend([100, 50, 2, 0, 400], 0, 4, 2, 128, torch.bfloat16, 16, seed=3, cu=[0, 3, 3, 8, 9, 11], shares=9)
    attend([100, 50, 2, 0, 400], 0, 4, 2, 128, torch.float16, 64, seed=4, cu=[0, 30, 30, 41, 42, 44], causal=False)


def test_rows_behind_the_last_sequence_stay():
    k_pages, v_pages, table, seqlens = make_cache([40, 20], 16, 2, 64, torch.bfloat16)
    q = torch.randn(6, 4, 64).bfloat16().cuda()
    cu = [0, 1, 3]
    out = torch.full((6, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 6), 5.0, device="cuda")
    binding.attention_paged(q, k_pages, v_pages, table, seqlens, max_seqlen_q=2, out=out, lse=lse,
                            cu_seqlens_q=torch.tensor(cu, dtype=torch.int32).cuda())
    check_attention(out[:3], lse[:, :3], q[:3], k_pages, v_pages, table, [40, 20], cu)
    assert bool((out[3:] == 5).all()) and bool((lse[:, 3:] == 5).all())


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("shares", [1, 6])
def test_unused_slots_do_not_matter(fill, shares):
    attend([70, 1, 17, 128], 1, 4, 2, 128, torch.bfloat16, 32, "nhd", seed=1, fill=fill, shares=shares)
    attend([70, 4, 17, 131], 4, 8, 2, 64, torch.bfloat16, 16, seed=2, fill=fill, shares=shares)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_masked_key_does_not_reach_a_row(bad):
    """The last of three new tokens holds NaN or infinity: the two before it do
    not read it.  Keys before the window hold them too."""
    k_pages, v_pages, table, seqlens = make_cache([90], 16, 2, 64, torch.bfloat16, seed=5)
    q = torch.randn(3, 4, 64).bfloat16().cuda()
    ref, lref = binding.attention_paged(q, k_pages, v_pages, table, seqlens, window_left=50)
    for pages in (k_pages, v_pages):
        for j in [89] + list(range(0, 37)):  # rows at positions 87, 88 read keys 37 (38) .. 87 (88)
            pages[int(table[0, j // 16]), :, j % 16] = bad
    o, lse = binding.attention_paged(q, k_pages, v_pages, table, seqlens, window_left=50)
    assert torch.equal(o[:2], ref[:2]) and torch.equal(lse[:, :2], lref[:, :2])
    assert bool(torch.isnan(o[2]).any())


def test_pages_outside_the_window_are_not_looked_at():
    k_pages, v_pages, table, seqlens = make_cache([500], 16, 2, 64, torch.float16, seed=6)
    q = torch.randn(1, 4, 64).half().cuda()
    ref, lref = binding.attention_paged(q, k_pages, v_pages, table, seqlens, window_left=99)
    table[0, :25] = 1 << 30  # keys 0 .. 399; the row reads 400 .. 499
    o, lse = binding.attention_paged(q, k_pages, v_pages, table, seqlens, window_left=99)
    assert torch.equal(o, ref) and torch.equal(lse, lref)


@pytest.mark.parametrize("scale", [30.0, 0.001])
def test_large_and_small_logits(scale):
    attend([900, 31], 1, 4, 1, 128, torch.bfloat16, 16, seed=8, q_scale=scale)


def test_a_nan_query_or_key_shows():
    k_pages, v_pages, table, seqlens = make_cache([300, 1], 16, 1, 64, torch.bfloat16, seed=7)
    q = torch.randn(2, 2, 64).bfloat16().cuda()
    ref, _ = binding.attention_paged(q, k_pages, v_pages, table, seqlens, num_shares=5)
    q[0, 1, 3] = float("nan")
    k_pages[int(table[1, 0]), :, 0, 0] = float("nan")  # the only key of the second sequence
    for shares in (1, 5):
        o, lse = binding.attention_paged(q, k_pages, v_pages, table, seqlens, num_shares=shares)
        assert bool(torch.isnan(o[0, 1]).all()) and bool(torch.isnan(o[1]).all()) and bool(torch.isnan(lse[:, 1]).all())
        assert float((o[0, 0].float() - ref[0, 0].float()).abs().max()) <= 2 ** -6


def test_results_do_not_depend_on_the_workspace_and_repeat():
    k_pages, v_pages, table, seqlens = make_cache([700, 90, 33], 16, 2, 128, torch.bfloat16, seed=9)
    q = torch.randn(3, 8, 128).bfloat16().cuda()
    need = binding.attn_fwd_paged_workspace_size(8, 2, 1, 128, 13)
    got = []
    for byte in (0, 0xff, 0x7f):
        ws = torch.full((need,), byte, dtype=torch.uint8, device="cuda")
        got.append(binding.attention_paged(q, k_pages, v_pages, table, seqlens, num_shares=13, workspace=ws))
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])


def test_without_lse_and_strided_rows():
    k_pages, v_pages, table, seqlens = make_cache([100, 64, 7], 16, 2, 64, torch.bfloat16, seed=10)
    fused = torch.randn(3, 8, 64).bfloat16().cuda()
    q = fused[:, 2:6]
    ref, _ = binding.attention_paged(q.contiguous(), k_pages, v_pages, table, seqlens)
    buf = torch.zeros(4, 3, 64, dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)  # heads outermost
    o, lse = binding.attention_paged(q, k_pages, v_pages, table, seqlens, out=buf, return_lse=False)
    assert lse is None and torch.equal(buf, ref)
    wide = torch.full((3, 20), -1, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + table.shape[1]] = table
    o2, _ = binding.attention_paged(q, k_pages, v_pages, wide[:, 3:3 + table.shape[1]], seqlens)
    assert torch.equal(o2, ref)


def test_many_sequences():
    """More sequences than a CTA has threads."""
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 90, 500)]
    attend(lens, 1, 2, 1, 32, torch.bfloat16, 16, seed=11)


def test_another_stream_and_a_replayed_graph():
    k_pages, v_pages, table, seqlens = make_cache([700, 90, 33], 16, 2, 128, torch.bfloat16, seed=12)
    q = torch.randn(3, 8, 128).bfloat16().cuda()
    kw = dict(num_shares=40)
    ref, lref = binding.attention_paged(q, k_pages, v_pages, table, seqlens, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse = binding.attention_paged(q, k_pages, v_pages, table, seqlens, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, ref) and torch.equal(lse, lref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = binding.attention_paged(q, k_pages, v_pages, table, seqlens, **kw)
    # the lengths are the device's: the same graph serves other ones
    lens = [650, 90, 1]
    seqlens.copy_(torch.tensor(lens, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    check_attention(o, lse, q, k_pages, v_pages, table, lens, [0, 1, 2, 3])


def test_calls_on_two_streams_at_once():
    """Two problems in flight on two streams, given as the helpers' stream,
    many times over: each gives its own result every time."""
    jobs = []
    for seed, lens, Hq in ((1, [900, 40, 333], 8), (2, [64, 1200], 6)):
        k_pages, v_pages, table, seqlens = make_cache(lens, 16, 2, 64, torch.bfloat16, seed=seed)
        q = torch.randn(len(lens), Hq, 64).bfloat16().cuda()
        ref = binding.attention_paged(q, k_pages, v_pages, table, seqlens, num_shares=50)
        jobs.append((q, k_pages, v_pages, table, seqlens, torch.cuda.Stream(), ref))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (q, k_pages, v_pages, table, seqlens, stream, _) in enumerate(jobs):
            got[i].append(binding.attention_paged(q, k_pages, v_pages, table, seqlens, num_shares=50, stream=stream))
    torch.cuda.synchronize()
    for i, job in enumerate(jobs):
        for o, lse in got[i]:
            assert torch.equal(o, job[6][0]) and torch.equal(lse, job[6][1])


def test_two_graphs_replayed_in_turn():
    """Two captured graphs, each with a workspace of its own from its pool."""
    graphs = []
    for seed, lens in ((3, [500, 77]), (4, [1000, 9])):
        k_pages, v_pages, table, seqlens = make_cache(lens, 16, 2, 128, torch.float16, seed=seed)
        q = torch.randn(2, 8, 128).half().cuda()
        ref = binding.attention_paged(q, k_pages, v_pages, table, seqlens, num_shares=30)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = binding.attention_paged(q, k_pages, v_pages, table, seqlens, num_shares=30)
        graphs.append((graph, out, ref, q, k_pages, v_pages, table, seqlens))
    for _ in range(3):
        for graph, *_ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for _, out, ref, *_ in graphs:
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])


def test_a_stream_of_another_kind_is_refused():
    class Elsewhere:
        device = torch.device("cuda", 7)
        cuda_stream = 0

    k_pages, v_pages, table, seqlens = make_cache([20], 16, 1, 32, torch.float16)
    q = torch.zeros(1, 1, 32, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        binding.attention_paged(q, k_pages, v_pages, table, seqlens, stream=Elsewhere())


@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_caches_past_32_bit_offsets(layout):
    """Pages at the end of a cache of more than 2^31 elements (and so bytes):
    what is appended there is what attention reads back."""
    page, Hkv, D = 128, 8, 128
    pool = (1 << 31) // (page * Hkv * D) + 9
    shape = (pool, Hkv, page, D) if layout == "hnd" else (pool, page, Hkv, D)
    k_pages, v_pages = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if layout == "nhd":
        k_pages, v_pages = k_pages.permute(0, 2, 1, 3), v_pages.permute(0, 2, 1, 3)
    lens = [300, 129]
    table = torch.tensor([[pool - 1, pool - 4, pool - 2], [pool - 3, 0, -1]], dtype=torch.int32).cuda()
    seqlens = torch.tensor(lens, dtype=torch.int32).cuda()
    cu = [0, 300, 429]
    k, v = (torch.randn(429, Hkv, D).bfloat16().cuda() for _ in range(2))
    binding.paged_append(k, v, k_pages, v_pages, table, seqlens,
                         cu_seqlens_q=torch.tensor(cu, dtype=torch.int32).cuda())
    q = torch.randn(2, Hkv, D).bfloat16().cuda()
    o, lse = binding.attention_paged(q, k_pages, v_pages, table, seqlens)
    used = torch.tensor([pool - 1, pool - 4, pool - 2, pool - 3, 0], device="cuda")  # alone, for the oracle
    kp, vp = k_pages[used].contiguous(), v_pages[used].contiguous()
    at = torch.tensor([[0, 1, 2], [3, 4, -1]], dtype=torch.int32)
    check_attention(o, lse, q, kp, vp, at, lens, [0, 1, 2])
    assert torch.equal(kp[0, :, 5], k[5]) and torch.equal(vp[4, :, 0], v[300 + 128])


def test_bad_lengths_offsets_and_pages_are_recorded():
    k_pages, v_pages, table, seqlens = make_cache([60, 50, 40], 16, 2, 64, torch.bfloat16, seed=13)
    q = torch.randn(3, 4, 64).bfloat16().cuda()
    ref, _ = binding.attention_paged(q, k_pages, v_pages, table, seqlens)

    def run(**kw):
        out = torch.full((3, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        args = dict(table=table, seqlens=seqlens)
        args.update({k: v for k, v in kw.items() if k in args})
        rest = {k: v for k, v in kw.items() if k not in args}
        binding.attention_paged(q, k_pages, v_pages, args["table"], args["seqlens"], out=out, **rest)
        return out, binding.etattn_read_device_status(clear=True)

    for bad in (-1, 65):  # 65 > 4 pages of 16
        lens = seqlens.clone()
        lens[1] = bad
        out, status = run(seqlens=lens)
        assert status == binding.ETATTN_ERR_BAD_SEQLENS
        assert bool((out[1] == 9).all()) and torch.equal(out[[0, 2]], ref[[0, 2]])
    for cu in ([0, 1, 4, 3], [0, 2, 1, 3], [0, 1, 2, 4], [-1, 1, 2, 3]):
        out, status = run(cu_seqlens_q=torch.tensor(cu, dtype=torch.int32).cuda(), max_seqlen_q=2)
        assert status == binding.ETATTN_ERR_BAD_SEQLENS
    for page in (-1, k_pages.shape[0], 1 << 30):
        t = table.clone()
        t[1, 2] = page
        out, status = run(table=t)
        assert status == binding.ETATTN_ERR_BAD_INDEX
        assert torch.equal(out[[0, 2]], ref[[0, 2]]) and bool(torch.isfinite(out[1]).all())


# ---------------------------------------------------------------- append

def append_case(lens, cu, page, Hq, Hkv, D, dtype, layout, rope_dim, interleaved, weighted, seed, uniform=False):
    k_pages, v_pages, table, seqlens = make_cache(lens, page, Hkv, D, dtype, layout, seed)
    before = k_pages.clone(), v_pages.clone()
    g = torch.Generator().manual_seed(seed + 50)
    T = cu[-1]
    fused = (torch.randn(T, Hq + 2 * Hkv, D, generator=g) * 1.5).to(dtype).cuda()
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    kw, cos, sin = {}, None, None
    if weighted:
        kw.update(q_weight=(1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda(),
                  k_weight=(1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda())
    if rope_dim:
        cos, sin = binding.rope_tables(max(max(lens), 1), rope_dim)
        kw.update(rope_cos=cos, rope_sin=sin)
    q_out = torch.full((T, Hq, D), 7.0, dtype=dtype, device="cuda")
    got = binding.paged_append(k, v, k_pages, v_pages, table, seqlens, q=q if Hq else None, interleaved=interleaved,
                               q_out=q_out if Hq else None,
                               cu_seqlens_q=None if uniform else torch.tensor(cu, dtype=torch.int32).cuda(), **kw)
    torch.cuda.synchronize()
    assert (got is None) == (Hq == 0)
    placed = cache.new_tokens(lens, cu)
    tok = [t for _, t, _ in placed]
    pos = torch.tensor([p for _, _, p in placed], dtype=torch.int32)
    pages = torch.tensor([int(table[s, p // page]) for s, _, p in placed], dtype=torch.long, device="cuda")
    slots = (pos.long() % page).cuda()
    rows = dict(kw, positions=pos) if rope_dim else {}
    if placed:
        check_forward(k_pages[pages, :, slots], k[tok], kw.get("k_weight"), rows, interleaved, 1e-6, dtype)
        assert torch.equal(v_pages[pages, :, slots], v[tok])
        if Hq:
            check_forward(q_out[tok], q[tok], kw.get("q_weight"), rows, interleaved, 1e-6, dtype)
    lost = [t for t in range(T) if t not in tok]
    assert bool((q_out[lost] == 7).all())
    # every other slot is as it was
    for now, then in ((k_pages, before[0]), (v_pages, before[1])):
        now = now.clone()
        now[pages, :, slots] = then[pages, :, slots]
        assert torch.equal(now, then)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "pair"])
@pytest.mark.parametrize("D,dt,rope_dim,interleaved", [(128, "bf16", 128, False), (64, "f16", 32, True),
                                                        (32, "bf16", 16, False), (64, "bf16", 0, False)])
@pytest.mark.parametrize("page", [8, 64])
def test_append_one_token_each(layout, D, dt, rope_dim, interleaved, page):
    lens = [1, 8, 9, 100, 64, 65, 17]
    append_case(lens, list(range(8)), page, 4, 2, D, DT[dt], layout, rope_dim, interleaved, True, D, uniform=True)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (0, 3), (8, 8)])
def test_append_ragged_tokens(weighted, Hq, Hkv):
    """Prompts from nothing, continued ones, a sequence without new tokens, an
    unused slot, more tokens than places, and a token on the last slot."""
    append_case([40, 33, 16, 0, 3, 128], [0, 40, 45, 45, 46, 51, 52], 16, Hq, Hkv, 64, torch.bfloat16, "nhd", 64, False,
                weighted, 3)


def test_append_of_more_than_the_l2_holds_equals_pieces_of_it():
    """140 MB of prompts at once (eight heads a group) leave the bits that the
    same tokens leave when they come 60 at a time (one head a group)."""
    S, Hq, Hkv, D, page = 4, 24, 8, 128, 32
    n = (140 << 20) // (4 * D * (Hq + 2 * Hkv)) // S // 60 * 60 + 60
    k_pages, v_pages, table, _ = make_cache([n] * S, page, Hkv, D, torch.bfloat16, "nhd", seed=3)
    k2, v2 = k_pages.clone(), v_pages.clone()
    x = torch.randn(S, n, Hq + 2 * Hkv, D).bfloat16().cuda()
    cos, sin = binding.rope_tables(n, D)
    w = (1 + 0.2 * torch.randn(D)).bfloat16().cuda()
    kw = dict(q_weight=w, k_weight=w, rope_cos=cos, rope_sin=sin)

    def append(rows, keys, kp, vp):
        q, k, v = rows[..., :Hq, :], rows[..., Hq:Hq + Hkv, :], rows[..., Hq + Hkv:, :]
        flat = lambda t: t.reshape(-1, t.shape[-2], D)  # noqa: E731
        lens = torch.full((S,), keys, dtype=torch.int32, device="cuda")
        return binding.paged_append(flat(k), flat(v), kp, vp, table, lens, q=flat(q), **kw).view(S, -1, Hq, D)

    whole = append(x, n, k_pages, v_pages)
    for a in list(range(0, n, 60)):
        part = append(x[:, a:a + 60], a + 60, k2, v2)
        if a in (0, 600, n - 60):
            assert torch.equal(part, whole[:, a:a + 60])
    assert torch.equal(k_pages, k2) and torch.equal(v_pages, v2)


def test_append_rows_behind_the_last_sequence_stay():
    k_pages, v_pages, table, seqlens = make_cache([20, 10], 16, 2, 64, torch.bfloat16)
    before = k_pages.clone()
    k = torch.randn(6, 2, 64).bfloat16().cuda()
    q_out = torch.full((6, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    binding.paged_append(k, k, k_pages, v_pages, table, seqlens, q=k, q_out=q_out,
                         cu_seqlens_q=torch.tensor([0, 1, 3], dtype=torch.int32).cuda())
    assert bool((q_out[3:] == 7).all()) and torch.equal(q_out[:3], k[:3])
    assert int((k_pages != before).any(1).any(-1).sum()) == 3


def test_append_bad_places_are_recorded_and_skipped():
    k_pages, v_pages, table, seqlens = make_cache([30, 20, 10], 16, 2, 64, torch.bfloat16)
    cos, sin = binding.rope_tables(25, 64)
    k = torch.randn(3, 2, 64).bfloat16().cuda()

    def run(code, table=table, seqlens=seqlens, cu=None, rope=False):
        kp, vp = k_pages.clone(), v_pages.clone()
        kw = dict(rope_cos=cos, rope_sin=sin) if rope else {}
        binding.paged_append(k, k, kp, vp, table, seqlens, cu_seqlens_q=cu, **kw)
        assert binding.etattn_read_device_status(clear=True) == code
        return int((kp != k_pages).any(1).any(-1).sum())

    assert run(binding.ETATTN_ERR_BAD_INDEX, rope=True) == 2  # position 29 of 25
    for page in (-1, k_pages.shape[0], -(1 << 31)):
        t = table.clone()
        t[1, 1] = page
        assert run(binding.ETATTN_ERR_BAD_INDEX, table=t) == 2
    lens = seqlens.clone()
    lens[0] = 33  # two pages of 16 hold 32
    assert run(binding.ETATTN_ERR_BAD_SEQLENS, seqlens=lens) == 2
    lens[0] = -5
    assert run(binding.ETATTN_ERR_BAD_SEQLENS, seqlens=lens) == 2
    for cu in ([0, 1, 5, 3], [2, 2, 2, 3], [0, -1, 2, 3]):
        run(binding.ETATTN_ERR_BAD_SEQLENS, cu=torch.tensor(cu, dtype=torch.int32).cuda())


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_prefill_then_decode_equals_attention_over_everything(layout):
    """A user's run: a prompt through norm, rotation and packed attention while
    its keys go to the cache; then decode steps (append, attention over the
    cache).  Every decode row must equal, within the rounding of the weights
    and of O, the last row of causal attention over the whole sequence, whose
    keys the packed path normed and rotated to the same bits."""
    dtype, D, Hq, Hkv, page, steps = torch.bfloat16, 64, 8, 2, 16, 4
    prompts = [37, 5, 64]
    S = len(prompts)
    final = [p + steps for p in prompts]
    k_pages, v_pages, table, _ = make_cache(final, page, Hkv, D, dtype, layout, seed=21)
    cos, sin = binding.rope_tables(max(final), D)
    g = torch.Generator().manual_seed(22)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2))
    x = [torch.randn(L, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda() for L in final]
    norm = dict(q_weight=wq, k_weight=wk, rope_cos=cos, rope_sin=sin)

    def split(rows):
        return rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]

    # prompts, packed
    q, k, v = split(torch.cat([r[:p] for r, p in zip(x, prompts)]))
    cu = W.cu_seqlens_of(prompts)
    pos = torch.cat([torch.arange(p, dtype=torch.int32) for p in prompts]).cuda()
    q1, k1 = binding.qk_norm_rope(q, k, positions=pos, **norm)
    o1, _ = binding.attention_varlen(q1, k1, v, cu.cuda(), max(prompts), causal=True)
    lens = torch.tensor(prompts, dtype=torch.int32).cuda()
    q2 = binding.paged_append(k, v, k_pages, v_pages, table, lens, q=q, cu_seqlens_q=cu.cuda(), **norm)
    assert torch.equal(q1, q2)
    for step in range(steps):
        lens += 1
        q, k, v = split(torch.stack([r[p + step] for r, p in zip(x, prompts)]))
        qr = binding.paged_append(k, v, k_pages, v_pages, table, lens, q=q, **norm)
        o, lse = binding.attention_paged(qr, k_pages, v_pages, table, lens, max_seqlen_k=max(final))
        check_attention(o, lse, qr, k_pages, v_pages, table, [p + step + 1 for p in prompts], list(range(S + 1)))
        for s, p in enumerate(prompts):
            n = p + step + 1
            qs, ks, vs = split(x[s][:n])
            qn, kn = binding.qk_norm_rope(qs, ks, positions=torch.arange(n, dtype=torch.int32).cuda(), **norm)
            ro, rl = binding.attention_varlen(qn, kn, vs, torch.tensor([0, n], dtype=torch.int32).cuda(), n,
                                              causal=True)
            assert torch.equal(qn[-1], qr[s])
            amax = float(vs.float().abs().max())
            # both sides round their weights (2^-8 of at most max|v|) and O
            assert float((ro[-1].float() - o[s].float()).abs().max()) <= 4 * 2.0 ** -8 * amax
            assert float((rl[:, -1] - lse[:, s]).abs().max()) <= 1e-4


def test_training_chain_gradients():
    """qk_norm_rope -> attention -> attention_backward -> qk_norm_rope_backward
    against float64 autograd of the whole chain.  The 16-bit intermediate q, k,
    o, dq, dk each carry a half step (2^-11) of their own size and the chain's
    derivative mixes them; the relative error of each gradient tensor in the
    2-norm stays under 16 half steps."""
    dtype, B, N, Hq, Hkv, D = torch.float16, 2, 70, 4, 2, 64
    g = torch.Generator().manual_seed(31)
    q, k, v = (torch.randn(B * N, h, D, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2))
    dout = torch.randn(B, Hq, N, D, generator=g).to(dtype).cuda()
    cos, sin = binding.rope_tables(N, D)
    pos = torch.arange(N, dtype=torch.int32).repeat(B).cuda()
    kw = dict(q_weight=wq, k_weight=wk, rope_cos=cos, rope_sin=sin, positions=pos)

    def batched(t):  # [B * N, H, D] -> [B, H, N, D]
        return t.view(B, N, t.shape[1], D).permute(0, 2, 1, 3)

    qn, kn = binding.qk_norm_rope(q, k, **kw)
    o, lse = binding.attention(batched(qn), batched(kn), batched(v), causal=True)
    outs = {n: torch.empty(B, N, h, D, dtype=dtype, device="cuda").permute(0, 2, 1, 3)
            for n, h in (("dq", Hq), ("dk", Hkv), ("dv", Hkv))}
    dqn, dkn, dv = binding.attention_backward(batched(qn), batched(kn), batched(v), o, lse, dout, causal=True, **outs)
    packed = lambda t: t.permute(0, 2, 1, 3).reshape(B * N, t.shape[1], D)  # noqa: E731
    dq, dk, dwq, dwk = binding.qk_norm_rope_backward(q, k, packed(dqn), packed(dkn), **kw)

    leaves = [t.double().cpu().requires_grad_() for t in (q, k, v, wq, wk)]
    c, s_ = cos.double().cpu()[pos.cpu().long()][:, None], sin.double().cpu()[pos.cpu().long()][:, None]

    def nr(x, w):
        n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = n[..., :D // 2], n[..., D // 2:]
        return torch.cat((a * c - b * s_, b * c + a * s_), -1)

    Q, K, V = batched(nr(leaves[0], leaves[3])), batched(nr(leaves[1], leaves[4])), batched(leaves[2])
    K, V = K.repeat_interleave(Hq // Hkv, 1), V.repeat_interleave(Hq // Hkv, 1)
    z = (Q @ K.transpose(-1, -2) * D ** -0.5).masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), -np.inf)
    (torch.softmax(z, -1) @ V * dout.double().cpu()).sum().backward()
    for name, got, leaf in zip("q k v wq wk".split(), (dq, dk, packed(dv), dwq, dwk), leaves):
        rel = float((got.double().cpu() - leaf.grad).norm() / leaf.grad.norm())
        assert rel <= 16 * 2.0 ** -11, f"gradient of {name}: {rel:.2e}"
