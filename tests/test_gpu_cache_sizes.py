"""GPU tests: the helpers refuse tokens that do not divide among the sequences,
offsets that do not fit and a bound of new tokens that they do not keep are
recorded, and rows of no sequence are left out."""

import pytest
import torch

from exact_tiled_attention_19_gb300 import binding
from tests.test_gpu_paged import make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert binding.etattn_read_device_status(clear=True) == 0


@pytest.mark.parametrize("S,T", [(5, 3), (3, 5), (0, 3)])
def test_helpers_refuse_tokens_that_do_not_divide(S, T):
    k_pages, v_pages, table, seqlens = make_cache([20] * 5, 16, 2, 64, torch.bfloat16)
    table, seqlens = table[:S], seqlens[:S]
    q, k = (torch.zeros(T, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    for call in (lambda: binding.attention_paged(q, k_pages, v_pages, table, seqlens),
                 lambda: binding.paged_append(k, k, k_pages, v_pages, table, seqlens, q=q)):
        with pytest.raises(binding.EtattnError) as e:
            call()
        assert e.value.code == binding.ETATTN_ERR_BAD_SHAPE


@pytest.mark.parametrize("cu,code", [([0, 0, 0, 0], 0), ([0, 1, 2, 3], 9), ([0, 0, 0, 1], 9)])
def test_a_bound_of_zero_new_tokens(cu, code):
    """Nothing is written: no sequence keeps a token within the bound."""
    k_pages, v_pages, table, seqlens = make_cache([20, 30, 40], 16, 2, 64, torch.bfloat16)
    q = torch.randn(3, 4, 64).bfloat16().cuda()
    out, lse = torch.full_like(q, 5.0), torch.full((4, 3), 5.0, device="cuda")
    for shares in (None, 7):
        binding.attention_paged(q, k_pages, v_pages, table, seqlens, max_seqlen_q=0, num_shares=shares, out=out,
                                lse=lse, cu_seqlens_q=torch.tensor(cu, dtype=torch.int32).cuda())
        assert binding.etattn_read_device_status(clear=True) == code
        assert bool((out == 5).all()) and bool((lse == 5).all())


@pytest.mark.parametrize("cu", [
    [0, 5, 3],       # the last offset decreases
    [0, 3, 1, 4],    # every token has a sequence, and one sequence less than none
    [0, 2, 11],      # past the rows
    [0, 0, -1, 0],
])
def test_append_records_offsets_that_do_not_fit(cu):
    """Whether or not a token shows it; attention over the same offsets records
    them, too."""
    S, T = len(cu) - 1, 10
    k_pages, v_pages, table, seqlens = make_cache([40] * S, 16, 2, 64, torch.bfloat16)
    k, cu = torch.randn(T, 2, 64).bfloat16().cuda(), torch.tensor(cu, dtype=torch.int32).cuda()
    binding.paged_append(k, k, k_pages, v_pages, table, seqlens, cu_seqlens_q=cu)
    assert binding.etattn_read_device_status(clear=True) == binding.ETATTN_ERR_BAD_SEQLENS
    binding.attention_paged(k, k_pages, v_pages, table, seqlens, cu_seqlens_q=cu, max_seqlen_q=T)
    assert binding.etattn_read_device_status(clear=True) == binding.ETATTN_ERR_BAD_SEQLENS


@pytest.mark.parametrize("Hq", [2, 32])  # one and four heads a group
def test_append_with_many_rows_behind_the_last_sequence(Hq):
    """A call of a fixed size (a captured graph's) of which the offsets use a
    few rows: those are placed, and whatever the others hold is left out."""
    T, lens, cu = 1200, [40, 0, 25], [0, 3, 3, 8]
    k_pages, v_pages, table, seqlens = make_cache(lens, 16, 2, 64, torch.bfloat16)
    before = k_pages.clone(), v_pages.clone()
    x = torch.randn(T, Hq + 4, 64).bfloat16().cuda()
    x[8:] = float("nan")
    q, k, v = x[:, :Hq], x[:, Hq:Hq + 2], x[:, Hq + 2:]
    q_out = torch.full((T, Hq, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    binding.paged_append(k, v, k_pages, v_pages, table, seqlens, q=q, q_out=q_out, q_weight=w,
                         cu_seqlens_q=torch.tensor(cu, dtype=torch.int32).cuda())
    ref, _ = binding.qk_norm_rope(q[:8], k[:8], q_weight=w)
    assert torch.equal(q_out[:8], ref) and bool((q_out[8:] == 7).all())
    changed = set()
    for s, t, p in [(0, t, 37 + t) for t in range(3)] + [(2, t, 17 + t) for t in range(3, 8)]:
        page = int(table[s, p // 16]), p % 16
        changed.add(page)
        assert torch.equal(k_pages[page[0], :, page[1]], k[t]) and torch.equal(v_pages[page[0], :, page[1]], v[t])
    for now, then in ((k_pages, before[0]), (v_pages, before[1])):
        now = now.clone()
        for page, slot in changed:
            now[page, :, slot] = then[page, :, slot]
        assert torch.equal(now, then)
