"""GPU tests of a step of no sequences: the tensors that a caller hands in for the
results are written, as those of a step with sequences are."""

import numpy as np
import pytest
import torch

from exact_tiled_attention_19_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert binding.etattn_read_device_status(clear=True) == 0


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


@pytest.mark.parametrize("total", [0, 5])
def test_results_handed_in_are_written(total):
    none, table, pages, count = i32([]), i32(np.zeros((0, 4))), i32([1, 2, 3]), i32([3])
    out = dict(seqlens_out=i32([]), cu_seqlens_q=i32([77]), positions=i32([77] * total),
               slots=torch.full((total,), 77, device="cuda"), free_count_out=i32([77]))
    got = binding.paged_extend(none, none, table, pages, count, page_size=8, total_tokens=total, **out)
    assert all(x is y for x, y in zip(got, out.values()))
    assert [x.tolist() for x in got] == [[], [0], [0] * total, [-1] * total, [3]]
    left = i32([77])
    got = binding.paged_truncate(none, none, table, pages, count, page_size=8, seqlens_out=none, free_count_out=left)
    assert got[1] is left and left.tolist() == [3]
    # in place, and new tensors
    got = binding.paged_extend(none, none, table, pages, count, page_size=8, total_tokens=total, seqlens_out=none,
                               free_count_out=count)
    assert got[4] is count and [x.tolist() for x in got] == [[], [0], [0] * total, [-1] * total, [3]]
    assert binding.paged_truncate(none, none, table, pages, count, page_size=8, free_count_out=count)[1].tolist() == [3]
    assert pages.tolist() == [1, 2, 3]


def test_invalid_calls_are_refused_without_sequences_too():
    none, table, pages, count = i32([]), i32(np.zeros((0, 4))), i32([1, 2, 3]), i32([3])
    for kw in (dict(page_size=12, total_tokens=0), dict(page_size=8, total_tokens=2 ** 30 + 1, positions=none, slots=none)):
        with pytest.raises((binding.EtattnError, ValueError, TypeError)):
            binding.paged_extend(none, none, table, pages, count, **kw)
    with pytest.raises(binding.EtattnError):
        binding.paged_truncate(none, none, table, pages, count, page_size=12)


@pytest.mark.parametrize("other", [False, True])
def test_a_captured_step_of_no_sequences(other):
    """Replayed with another count, on the capturing stream; or called on a stream of its own."""
    none, table, pages, count = i32([]), i32(np.zeros((0, 4))), i32([1, 2, 3]), i32([3])
    cu, left, stream = i32([77]), i32([77]), torch.cuda.Stream()
    torch.cuda.synchronize()

    def step(**kw):
        return binding.paged_extend(none, none, table, pages, count, page_size=8, total_tokens=0, cu_seqlens_q=cu,
                                    free_count_out=left, **kw)

    if other:
        step(stream=stream)
        stream.synchronize()
        assert cu.tolist() == [0] and left.tolist() == [3]
        return
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for n in (2, 1):
            cu.fill_(77), left.fill_(77), count.fill_(n)
            graph.replay()
            stream.synchronize()
            assert cu.tolist() == [0] and left.tolist() == [n]
