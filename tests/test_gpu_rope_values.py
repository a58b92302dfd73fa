"""GPU tests of the norm and rotation at unusual values: weights that are
infinite or NaN reach nothing but their own pair, elements that neither norm
nor rotation touches keep their bits, and denormal inputs keep their size."""

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


def bits(t):
    return t.view(torch.int16)


def every_finite_value(dtype):
    """All finite 16-bit values, zeros of both signs and denormals among them."""
    x = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(dtype)
    return x[torch.isfinite(x.float())]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rope_dim,interleaved", [(0, False), (0, True), (32, False), (32, True)])
def test_what_is_neither_normed_nor_rotated_keeps_its_bits(dtype, rope_dim, interleaved):
    """Forward and backward, at one and at four heads a group."""
    D = 64
    x = every_finite_value(dtype).view(-1, 4, D).cuda()
    for q in (x[:5], x.repeat(20, 1, 1)):
        T = q.shape[0]
        kw = {}
        if rope_dim:
            cos, sin = binding.rope_tables(T, rope_dim)
            kw = dict(rope_cos=cos, rope_sin=sin, positions=torch.arange(T, dtype=torch.int32, device="cuda"))
        out, _ = binding.qk_norm_rope(q, q, interleaved=interleaved, **kw)
        assert torch.equal(bits(out[..., rope_dim:]), bits(q[..., rope_dim:]))
        dq, dk, _, _ = binding.qk_norm_rope_backward(q, q, q, q, interleaved=interleaved, **kw)
        for d in (dq, dk):
            assert torch.equal(bits(d[..., rope_dim:]), bits(q[..., rope_dim:]))


@pytest.mark.parametrize("weighted", [False, True])
def test_denormal_inputs_keep_their_size(weighted):
    """BF16 rows below 2^-126 under a rotation, and with a norm whose eps leaves
    them there or lifts them out (r = eps^-1/2 = 1000).  An output is off by half a
    step of its own size or half the smallest value, 2^-134.  In FP32 the two
    products of a row element are off by 2^-150 each, times r at most 2^-139;
    the other roundings, under 16 of 2^-24, of terms below 2^-116 make less
    than 2^-136."""
    T, H, D = 6, 3, 64
    g = torch.Generator().manual_seed(3)
    q = (torch.randn(T, H, D, generator=g) * 2.0 ** -128).to(torch.bfloat16).cuda()
    cos, sin = binding.rope_tables(T, D)
    kw = dict(rope_cos=cos, rope_sin=sin, positions=torch.arange(T, dtype=torch.int32, device="cuda"))
    if weighted:
        kw.update(q_weight=(1 + 0.2 * torch.randn(D, generator=g)).bfloat16().cuda())
    for eps in (1.0, 1e-6) if weighted else (1e-6,):
        out, _ = binding.qk_norm_rope(q, q, eps=eps, **kw)
        ref = cache.norm_rope(f64(q), f64(kw.get("q_weight")), f64(cos), f64(sin), False, eps)
        assert np.abs(ref).max() > 2.0 ** -128
        bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -134 + 2.0 ** -135
        assert np.all(np.abs(f64(out) - ref) <= bound)
