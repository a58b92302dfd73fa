"""GPU tests of how paged attention's work is cut, where the producer's search
for its sequences takes its other paths: more sequences than a warp has lanes,
runs of sequences without new tokens across the windows of 32 that the producer
loads, and units of 32 rows with any number of shares."""

import numpy as np
import pytest
import torch

from exact_tiled_attention_19_gb300 import binding
from tests.test_gpu_paged import DT, attend

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert binding.etattn_read_device_status(clear=True) == 0


@pytest.mark.parametrize("S", [31, 32, 33, 34, 63, 64, 65, 97])
@pytest.mark.parametrize("shares", [None, 1, 5, 304])
def test_sequence_counts_around_a_warp(S, shares):
    rng = np.random.default_rng(S)
    attend([int(x) for x in rng.integers(0, 200, S)], 1, 2, 1, 64, torch.bfloat16, 16, seed=S, shares=shares)


def ragged(counts):
    return [0] + [int(x) for x in np.cumsum(counts)]


@pytest.mark.parametrize("S,empty", [
    (100, [(20, 60)]),            # a run across the first reload
    (100, [(0, 33)]),             # the first window is empty
    (100, [(31, 33), (62, 97)]),
    (130, [(1, 129)]),            # three windows between two sequences
    (120, [(30, 64), (64, 119)]),
    (64, [(33, 64)]),             # the line ends inside the second window
])
@pytest.mark.parametrize("shares", [1, 2, 7, 60, 304])
def test_runs_of_sequences_without_new_tokens(S, empty, shares):
    rng = np.random.default_rng(S + shares)
    counts = rng.integers(1, 4, S)
    for a, b in empty:
        counts[a:b] = 0
    lens = [int(x) for x in rng.integers(3, 150, S)]
    attend(lens, 0, 4, 2, 32, torch.float16, 16, seed=shares, cu=ragged(counts), shares=shares)


@pytest.mark.parametrize("n,Hq", [(3, 12), (4, 16), (8, 8), (16, 8)])  # 18, 32, 32 and 64 rows for each of 2 KV heads
@pytest.mark.parametrize("shares", [2, 7, 304])
@pytest.mark.parametrize("page", [8, 128, 256])
@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "f16"), (32, "bf16")])
def test_units_of_32_rows(n, Hq, shares, page, D, dt):
    attend([500, n, 75 + n, 333], n, Hq, 2, D, DT[dt], page, seed=page + n, shares=shares, fill=float("nan"))


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
def test_units_of_32_rows_of_ragged_sequences(fill):
    """Some of whose rows fill one group of warps only."""
    counts = [1, 5, 0, 8, 2, 4]
    attend([40, 300, 10, 129, 2, 77], 0, 8, 2, 64, torch.bfloat16, 16, "nhd", seed=1, cu=ragged(counts), shares=9,
           fill=fill, window_left=33)
