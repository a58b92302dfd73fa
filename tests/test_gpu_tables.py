"""GPU tests of the pages' bookkeeping (extend, truncate) against the definition
that takes and gives back pages one by one.  Whole numbers: everything is equal."""

import numpy as np
import pytest
import torch

from exact_tiled_attention_19_gb300 import binding
from oracle import quantised

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert binding.etattn_read_device_status(clear=True) == 0


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def make(S, longest, page, seed, spare=7, extra=3, wide=0):
    """Lengths, a block table that holds them, and the free pages, in random order."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, S)
    width = -(-longest // page) + extra
    need = -(-lens // page)
    total = S * width + spare
    order = rng.permutation(total)
    table = np.full((S, width + wide), -1)
    at = 0
    for s in range(S):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
    return rng, lens, table, list(order[at:]), width


def stack(free, capacity):
    out = np.full(capacity, -7)
    out[:len(free)] = free
    return i32(out), i32([len(free)])


def check_extend(S, longest, page, seed, most, padding=0, in_place=False, wide=0):
    rng, lens, table, free, width = make(S, longest, page, seed, wide=wide)
    new = rng.integers(0, most + 1, S)
    new = np.minimum(new, width * page - lens)
    new[rng.random(S) < 0.2] = 0
    T = int(new.sum()) + padding
    want = quantised.extend(new, lens, table, free, page, T)
    pages, count = stack(free, len(free) + 5)
    dl, dt = i32(lens), i32(table)[:, :width]
    before = pages.clone()
    out = dict(seqlens_out=dl, free_count_out=count) if in_place else {}
    got = binding.paged_extend(i32(new), dl, dt, pages, count, page_size=page, total_tokens=T, **out)
    seqlens, cu, positions, slots, left = (x.cpu().tolist() for x in got)
    assert np.array_equal(dt.cpu().numpy(), want[0][:, :width])
    assert (seqlens, cu, positions, slots) == tuple(want[1:5])
    assert left == [len(want[5])] and torch.equal(pages, before)
    if in_place:
        assert got[0] is dl and got[4] is count
    else:
        assert dl.tolist() == list(lens) and count.tolist() == [len(free)]


@pytest.mark.parametrize("S", [1, 2, 31, 33, 257, 1000, 1024, 1025, 3000, 4096, 4097, 9000])
@pytest.mark.parametrize("page", [8, 16, 4096])
def test_extend_decode_steps(S, page):
    check_extend(S, 3 * page, page, S + page, 1)


@pytest.mark.parametrize("S,longest,page,most", [(1, 0, 8, 1), (3, 100, 16, 700), (40, 50, 8, 60), (500, 30, 16, 90),
                                                 (1500, 64, 32, 31), (6, 9000, 64, 9000), (2000, 10, 8, 40),
                                                 (1, 5, 16, 50000), (5000, 9, 8, 7), (4500, 12, 8, 20)])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend_prompts(S, longest, page, most, in_place):
    check_extend(S, max(longest, most), page, S, most, in_place=in_place)


@pytest.mark.parametrize("S,most,padding", [(4, 3, 9), (700, 1, 40000), (2, 100, 5000), (3, 0, 17)])
def test_extend_padded_batches_and_wider_tables(S, most, padding):
    check_extend(S, 60, 16, S, most, padding=padding, wide=3)


def test_extend_the_most_sequences():
    check_extend(65535, 20, 8, 1, 1)


def check_truncate(S, longest, page, seed, how, in_place=False):
    rng, lens, table, free, width = make(S, longest, page, seed)
    if how == "ended":
        keep = np.where(rng.random(S) < 0.5, 0, lens)
    elif how == "drafts":
        keep = np.maximum(0, lens - rng.integers(0, 6, S))
    else:
        keep = rng.integers(0, lens + 1)
    want_lens, want = quantised.truncate(keep, lens, table, free, page)
    pages, count = stack(free, len(want) + 2)
    dl, dt = i32(lens), i32(table)
    out = dict(seqlens_out=dl, free_count_out=count) if in_place else {}
    seqlens, left = binding.paged_truncate(i32(keep), dl, dt, pages, count, page_size=page, **out)
    assert seqlens.tolist() == want_lens and left.tolist() == [len(want)]
    got = pages.tolist()
    assert got[:len(want)] == [int(x) for x in want] and got[len(want):] == [-7, -7]
    assert np.array_equal(dt.cpu().numpy(), table)


@pytest.mark.parametrize("S,longest,page", [(1, 100, 8), (1, 0, 16), (50, 300, 16), (1024, 40, 8), (1025, 40, 8),
                                            (3000, 200, 64), (4097, 30, 8),
                                            (20000, 9, 8)])
@pytest.mark.parametrize("how", ["ended", "drafts", "any"])
@pytest.mark.parametrize("in_place", [False, True])
def test_truncate(S, longest, page, how, in_place):
    check_truncate(S, longest, page, S + page, how, in_place)


REFUSED = {
    "negative length": (9, dict(lens=[5, -1, 3])),
    "negative count": (9, dict(new=[1, -2, 1])),
    "past the table": (9, dict(new=[1, 200, 1], total=202)),
    "more tokens than room": (9, dict(total=5)),
    "free count past its room": (9, dict(count=99)),
    "negative free count": (9, dict(count=-1)),
    "too few pages": (14, dict(count=2)),
}


@pytest.mark.parametrize("what", REFUSED)
@pytest.mark.parametrize("S", [3, 1500, 4500])
def test_a_step_that_does_not_fit_takes_nothing(what, S):
    code, bad = REFUSED[what]
    lens, new = np.full(S, 7), np.zeros(S, int)
    lens[:3], new[:3] = bad.get("lens", [5, 8, 3]), bad.get("new", [4, 9, 1])
    table = np.full((S, 8), -1)
    table[:, 0] = np.arange(S)
    pages, count = i32(np.arange(S, S + 20)), i32([bad.get("count", 20)])
    dt, T = i32(table), bad.get("total", 20)
    before = dt.clone()
    seqlens, cu, positions, slots, left = binding.paged_extend(i32(new), i32(lens), dt, pages, count, page_size=8,
                                                               total_tokens=T)
    assert binding.etattn_read_device_status(clear=True) == code
    assert torch.equal(dt, before) and seqlens.tolist() == list(lens) and torch.equal(left, count)
    assert not cu.any() and not positions.any() and bool((slots == -1).all())


@pytest.mark.parametrize("what,code", [("keep more than there is", 9), ("negative", 9), ("no room", 14)])
def test_a_truncation_that_does_not_fit_gives_nothing_back(what, code):
    lens, keep = [20, 9, 30], [0, 9, 8]
    if what == "negative":
        keep[1] = -1
    if what == "keep more than there is":
        keep[1] = 10
    table = np.arange(12).reshape(3, 4)
    pages, count = i32(np.full(9, -7)), i32([4 if what != "no room" else 5])
    seqlens, left = binding.paged_truncate(i32(keep), i32(lens), i32(table), pages, count, page_size=8)
    assert binding.etattn_read_device_status(clear=True) == code if what != "no room" else True
    if what == "no room":  # 3 + 3 pages go back, 4 places
        assert binding.etattn_read_device_status(clear=True) == code
    assert seqlens.tolist() == lens and torch.equal(left, count) and bool((pages == -7).all())


def test_no_sequences():
    none, pages, count = i32([]), i32([1, 2, 3]), i32([3])
    got = binding.paged_extend(none, none, i32(np.zeros((0, 4))), pages, count, page_size=8, total_tokens=0)
    assert [x.tolist() for x in got] == [[], [0], [], [], [3]]
    got = binding.paged_truncate(none, none, i32(np.zeros((0, 4))), pages, count, page_size=8)
    assert [x.tolist() for x in got] == [[], [3]]


@pytest.mark.parametrize("S", [5, 2000, 5000])
def test_a_captured_loop_hands_out_and_takes_back(S):
    """One graph with an extension and a truncation, both in place, replayed over
    changing amounts; the same by the definition, step by step."""
    page, rng = 8, np.random.default_rng(S)
    lens, table, free = np.zeros(S, int), np.full((S, 10), -1), list(rng.permutation(S * 10))
    dl, dt, new, keep = i32(lens), i32(table), i32(lens), i32(lens)
    pages, count = stack(free, S * 10)
    T = 4 * S
    cu, pos, slots = i32(np.zeros(S + 1)), i32(np.zeros(T)), torch.zeros(T, dtype=torch.int64).cuda()
    ws = torch.empty(binding.attn_paged_tables_workspace_size(S), dtype=torch.uint8, device="cuda")

    def step():
        binding.paged_extend(new, dl, dt, pages, count, page_size=page, total_tokens=T, seqlens_out=dl,
                             cu_seqlens_q=cu, positions=pos, slots=slots, free_count_out=count, workspace=ws)
        torch.sub(dl, keep, out=keep_len)
        binding.paged_truncate(keep_len, dl, dt, pages, count, page_size=page, seqlens_out=dl, free_count_out=count,
                               workspace=ws)

    keep_len = i32(lens)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for k in range(6):
            n, back = rng.integers(0, 4, S), rng.integers(0, 2, S)
            back = np.minimum(back, lens + n)
            new.copy_(i32(n)), keep.copy_(i32(back))
            graph.replay()
            stream.synchronize()
            table, lens, want_cu, want_pos, want_slots, free = quantised.extend(n, lens, table, free, page, T)
            lens, free = quantised.truncate(np.array(lens) - back, lens, table, free, page)
            lens = np.array(lens)
            assert dl.tolist() == list(lens) and count.tolist() == [len(free)] and cu.tolist() == want_cu
            assert pos.tolist() == want_pos and slots.tolist() == want_slots
            got, held = dt.cpu().numpy(), -(-lens // page)
            assert all(np.array_equal(got[s, :held[s]], table[s, :held[s]]) for s in range(S))
            assert pages.tolist()[:len(free)] == [int(x) for x in free]


def test_another_stream_owns_what_it_allocates():
    rng, lens, table, free, width = make(9, 40, 8, 3)
    pages, count = stack(free, len(free))
    stream = torch.cuda.Stream()
    args = (i32(np.ones(9)), i32(lens), i32(table), pages, count)
    torch.cuda.synchronize()
    got = binding.paged_extend(*args, page_size=8, total_tokens=9, stream=stream)
    stream.synchronize()
    want = quantised.extend(np.ones(9, int), lens, table, free, 8, 9)
    assert got[3].tolist() == want[4] and got[0].tolist() == want[1]


def test_a_16_bit_cache_takes_its_pages_too():
    """The table and lengths of an extension in the calls of the 16-bit cache: each new key
    is where the slots say, and attention over the pages is that over the keys in a row."""
    page, D, Hkv, S = 16, 64, 2, 3
    table, lens = i32(np.full((S, 5), -1)), i32([0, 0, 0])
    pages, count = stack(list(np.random.default_rng(1).permutation(15)), 15)
    k_pages, v_pages = (torch.zeros(15, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g, rows = torch.Generator().manual_seed(0), [[[], []] for _ in range(S)]
    for new in ([37, 5, 16], [1, 0, 1], [2, 12, 16]):
        k, v, q = (torch.randn(sum(new), h, D, generator=g).bfloat16().cuda() for h in (Hkv, Hkv, 4))
        _, cu, _, slots, _ = binding.paged_extend(i32(new), lens, table, pages, count, page_size=page,
                                                  total_tokens=sum(new), seqlens_out=lens, free_count_out=count)
        binding.paged_append(k, v, k_pages, v_pages, table, lens, cu_seqlens_q=cu)
        for x, y in ((k, k_pages), (v, v_pages)):
            assert torch.equal(y.transpose(1, 2).reshape(-1, Hkv, D)[slots], x)
        o, lse = binding.attention_paged(q, k_pages, v_pages, table, lens, cu_seqlens_q=cu, max_seqlen_q=max(new))
        at = cu.tolist()
        for s in range(S):
            for x, y in zip(rows[s], (k, v)):
                x.append(y[at[s]:at[s + 1]])
            if new[s] == 0:
                continue
            ks, vs = (torch.cat(x).double().repeat_interleave(2, 1) for x in rows[s])
            sc = torch.einsum("nhd,lhd->hnl", q[at[s]:at[s + 1]].double(), ks) / 8
            L, n = ks.shape[0], new[s]
            seen = torch.arange(L, device="cuda") <= torch.arange(n, device="cuda")[:, None] + L - n
            P = sc.masked_fill(~seen, -torch.inf).softmax(-1)
            want = torch.einsum("hnl,lhd->nhd", P, vs)
            # a rounding of the output, and one of 2^-16 of every weight (two parts)
            bound = 2.0 ** -8 * want.abs() + 2.0 ** -14 * torch.einsum("hnl,lhd->nhd", P, vs.abs()) + 1e-6
            assert bool(((o[at[s]:at[s + 1]].double() - want).abs() <= bound).all())
