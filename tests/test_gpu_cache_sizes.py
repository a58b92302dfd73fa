"""GPU tests: the helpers refuse tokens that do not divide among the sequences,
and a bound of new tokens that the offsets do not keep is recorded."""

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
