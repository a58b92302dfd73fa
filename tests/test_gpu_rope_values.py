"""GPU tests of the norm and rotation at values where an element must not meet
another one: weights that are infinite or NaN, against the FP64 oracle."""

import numpy as np
import pytest
import torch

from exact_tiled_attention_19_gb300 import binding
from oracle import cache
from tests.test_gpu_rope import check_forward, f64, make, row_angles

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert binding.etattn_read_device_status(clear=True) == 0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("rope_dim,interleaved", [(0, False), (0, True), (32, False), (32, True), (64, False),
                                                  (64, True)])
@pytest.mark.parametrize("T", [3, 700, 16000])  # one, four and eight heads a group
def test_a_non_finite_weight_reaches_its_own_pair_alone(T, rope_dim, interleaved, bad):
    """n_d = x_d w_d r: the weight of one element past rope_dim reaches that
    element, one before it the two elements of its pair.  Every other element
    is that of the call with a weight of 1 in its place, bit for bit."""
    Hq, Hk, D, dtype = 33, 7, 64, torch.bfloat16
    q, k, kw = make(T, Hq, Hk, D, dtype, rope_dim, seed=T)
    hit = [3, 45]  # rope_dim = 32: one rotated, one not
    plain = dict(kw, q_weight=kw["q_weight"].clone(), k_weight=kw["k_weight"].clone())
    for w in (plain["q_weight"], plain["k_weight"]):
        w[hit] = 1.0
    odd = dict(plain, q_weight=plain["q_weight"].clone(), k_weight=plain["k_weight"].clone())
    for w in (odd["q_weight"], odd["k_weight"]):
        w[hit] = bad
    reached = set(hit)
    for d in hit:
        if d < rope_dim:
            reached.add(d ^ 1 if interleaved else (d + rope_dim // 2) % rope_dim)
    rest = [d for d in range(D) if d not in reached]
    ref = binding.qk_norm_rope(q, k, interleaved=interleaved, **plain)
    got = binding.qk_norm_rope(q, k, interleaved=interleaved, **odd)
    for a, b in zip(ref, got):
        assert torch.equal(a[..., rest], b[..., rest])
    if T == 3:
        cos, sin = row_angles(kw)
        with np.errstate(invalid="ignore"):
            want = cache.norm_rope(f64(q), f64(odd["q_weight"]), cos, sin, interleaved)
        assert np.array_equal(np.isfinite(want), np.isfinite(f64(got[0])))
        check_forward(ref[0], q, plain["q_weight"], plain, interleaved, 1e-6, dtype)
