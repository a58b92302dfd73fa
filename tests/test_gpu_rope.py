"""GPU tests of the norm and rotation of queries and keys, forward and
backward, against the FP64 oracle.

Bounds, from the arithmetic.  u is the output type's half step
(finfo.eps / 2), e = 2^-24 the FP32 one.
Forward: r carries the sum of squares (8 products in a thread, then 4 additions
across threads: 12 roundings, halved by the root), the division by D, eps and
rsqrtf (2 steps); x r w two more; the rotation two products and one sum.  Under
16 roundings of the two terms: |dy| <= u |y| + 16 e (|n_a| + |n_b|).
Backward: g is a rotation of the upstream gradient (3 roundings), g w one, the
dot product with x 12, r^2 and the mean under 24, the difference 2: under 48
roundings of the terms: |ddx| <= u |dx| + 48 e r (|g w| + |x| r^2 mean|g w x|),
with |g| replaced by |dy_a| + |dy_b| for the rotated pairs.
dw: each term g x r under 24 roundings, summed in FP32 over the N rows in some
order: |ddw| <= (N + 24) e sum |g x r|.
FP16 outputs below the normal range are off by at most 2^-25 more."""

import numpy as np
import pytest
import torch

from exact_tiled_attention_19_gb300 import binding
from oracle import cache

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert binding.etattn_read_device_status(clear=True) == 0


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def make(T, Hq, Hk, D, dtype, rope_dim, seed=0, fused=True, start=0, weighted=True, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    fused_qkv = (torch.randn(T, Hq + 2 * Hk, D, generator=g) * scale).to(dtype).cuda()
    q, k = fused_qkv[:, :Hq], fused_qkv[:, Hq:Hq + Hk]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2))
    kw = dict(q_weight=wq, k_weight=wk) if weighted else {}
    if rope_dim:
        cos, sin = binding.rope_tables(start + max(T, 1), rope_dim)
        perm = torch.randperm(T, generator=g)
        kw.update(rope_cos=cos, rope_sin=sin, positions=(start + perm).to(torch.int32).cuda())
    return q, k, kw


def row_angles(kw):
    if "positions" not in kw:
        return None, None
    p = kw["positions"].cpu().numpy()
    return f64(kw["rope_cos"])[p], f64(kw["rope_sin"])[p]


def pair_sums(x, rope_dim, interleaved):
    """|x_a| + |x_b| at both elements of every rotated pair, |x| elsewhere."""
    a = np.abs(x)
    if rope_dim == 0:
        return a
    out = a.copy()
    i = np.arange(rope_dim // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rope_dim // 2)
    out[..., ia] = out[..., ib] = a[..., ia] + a[..., ib]
    return out


def check_forward(out, x, w, kw, interleaved, eps, dtype):
    cos, sin = row_angles(kw)
    ref = cache.norm_rope(f64(x), f64(w), cos, sin, interleaved, eps)
    terms = pair_sums(cache.norm_rope(f64(x), f64(w), None, None, False, eps),
                      0 if cos is None else 2 * cos.shape[-1], interleaved)
    bound = half_step(dtype) * np.abs(ref) + 16 * E * terms + (2.0 ** -25 if dtype == torch.float16 else 1e-38)
    err = np.abs(f64(out) - ref)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.2f} of the bound"


def check_backward(dx, dw, x, w, dy, kw, interleaved, eps, dtype):
    cos, sin = row_angles(kw)
    rope_dim = 0 if cos is None else 2 * cos.shape[-1]
    x64, w64, dy64 = f64(x), f64(w), f64(dy)
    ref, rw = cache.norm_rope_backward(x64, w64, dy64, cos, sin, interleaved, eps)
    g = pair_sums(dy64, rope_dim, interleaved)
    if w is not None:
        r = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + eps)
        gw = g * np.abs(w64)
        terms = r * (gw + np.abs(x64) * r * r * (gw * np.abs(x64)).mean(-1, keepdims=True))
    else:
        terms = g
    bound = half_step(dtype) * np.abs(ref) + 48 * E * terms + (2.0 ** -25 if dtype == torch.float16 else 1e-38)
    err = np.abs(f64(dx) - ref)
    assert np.all(err <= bound), f"dx: worst {np.max(err / bound):.2f} of the bound"
    if w is not None:
        rows = x64.shape[0] * x64.shape[1]
        bound = (rows + 24) * E * (g * np.abs(x64) * r).sum((0, 1)) + 1e-30
        err = np.abs(f64(dw) - rw)
        assert np.all(err <= bound), f"dw: worst {np.max(err / bound):.2f} of the bound"


SHAPES = [
    # T, Hq, Hk, D, type, rope_dim, interleaved, fused
    (1, 1, 1, 32, "f16", 32, False, True), (1, 1, 1, 128, "bf16", 128, False, True),
    (7, 4, 2, 64, "bf16", 64, False, True), (7, 4, 2, 64, "f16", 64, True, False),
    (33, 5, 1, 128, "bf16", 64, False, True), (33, 5, 1, 128, "f16", 16, True, True),
    (130, 8, 8, 32, "bf16", 16, False, False), (130, 3, 2, 32, "f16", 32, True, True),
    (257, 32, 8, 128, "bf16", 128, False, True), (64, 7, 0, 64, "bf16", 64, False, True),
    (64, 0, 3, 64, "f16", 48, False, True), (19, 4, 2, 128, "bf16", 0, False, True),
]


@pytest.mark.parametrize("T,Hq,Hk,D,dt,rope_dim,interleaved,fused", SHAPES)
@pytest.mark.parametrize("weighted", [True, False])
def test_forward_and_backward_match_the_oracle(T, Hq, Hk, D, dt, rope_dim, interleaved, fused, weighted):
    dtype = DT[dt]
    q, k, kw = make(T, Hq, Hk, D, dtype, rope_dim, seed=T + D, fused=fused, start=1000, weighted=weighted)
    qo, ko = binding.qk_norm_rope(q, k, interleaved=interleaved, eps=1e-5, **kw)
    check_forward(qo, q, kw.get("q_weight"), kw, interleaved, 1e-5, dtype)
    check_forward(ko, k, kw.get("k_weight"), kw, interleaved, 1e-5, dtype)
    g = torch.Generator().manual_seed(5)
    dqo, dko = (torch.randn(t.shape, generator=g).to(dtype).cuda() for t in (q, k))
    dq, dk, dwq, dwk = binding.qk_norm_rope_backward(q, k, dqo, dko, interleaved=interleaved, eps=1e-5, **kw)
    assert (dwq is None) == (not weighted) and (dwk is None) == (not weighted)
    check_backward(dq, dwq, q, kw.get("q_weight"), dqo, kw, interleaved, 1e-5, dtype)
    check_backward(dk, dwk, k, kw.get("k_weight"), dko, kw, interleaved, 1e-5, dtype)


@pytest.mark.parametrize("T", [1021, 5000])
def test_many_tokens(T):
    """More (token, head) rows than the backward launch has groups of threads:
    every group takes several."""
    q, k, kw = make(T, 16, 4, 64, torch.bfloat16, 32, seed=T)
    qo, ko = binding.qk_norm_rope(q, k, **kw)
    check_forward(qo, q, kw["q_weight"], kw, False, 1e-6, torch.bfloat16)
    check_forward(ko, k, kw["k_weight"], kw, False, 1e-6, torch.bfloat16)
    dq, dk, dwq, dwk = binding.qk_norm_rope_backward(q, k, qo, ko, **kw)
    check_backward(dq, dwq, q, kw["q_weight"], qo, kw, False, 1e-6, torch.bfloat16)
    check_backward(dk, dwk, k, kw["k_weight"], ko, kw, False, 1e-6, torch.bfloat16)


@pytest.mark.parametrize("Hq,Hk,D,rope_dim,interleaved", [(32, 8, 128, 128, False), (33, 7, 128, 64, True),
                                                            (61, 12, 64, 64, False)])
def test_more_than_the_l2_holds_equals_pieces_of_it(Hq, Hk, D, rope_dim, interleaved):
    """Every row is computed by itself, so a large call (whose groups take eight
    heads) gives the bits of small ones (one head a group)."""
    T = (140 << 20) // (4 * D * (Hq + Hk)) + 5
    q, k, kw = make(T, Hq, Hk, D, torch.bfloat16, rope_dim, seed=1)
    qo, ko = binding.qk_norm_rope(q, k, interleaved=interleaved, **kw)
    for a, b in ((0, 97), (T // 2, T // 2 + 130), (T - 101, T)):
        part = dict(kw, positions=kw["positions"][a:b])
        qp, kp = binding.qk_norm_rope(q[a:b], k[a:b], interleaved=interleaved, **part)
        assert torch.equal(qp, qo[a:b]) and torch.equal(kp, ko[a:b])
        check_forward(qp, q[a:b], kw["q_weight"], part, interleaved, 1e-6, torch.bfloat16)


def test_gradients_equal_differences_of_the_forward_pass():
    """Directional differences of sum(dy * y) in the oracle's own forward pass
    (64 bits) against the kernel's gradients: the gradients' rounding to FP16
    leaves |sum dx v - difference| <= sum (2^-11 |dx| + 48 e terms) |v|, taken
    with twice the first term."""
    q, k, kw = make(6, 3, 2, 64, torch.float16, 32, seed=9)
    cos, sin = row_angles(kw)
    g = torch.Generator().manual_seed(6)
    dqo, dko = (torch.randn(t.shape, generator=g).half().cuda() for t in (q, k))
    dq, _, dwq, _ = binding.qk_norm_rope_backward(q, k, dqo, dko, **kw)
    x, w, dy = f64(q), f64(kw["q_weight"]), f64(dqo)
    rng = np.random.default_rng(1)
    loss = lambda x_, w_: float((cache.norm_rope(x_, w_, cos, sin) * dy).sum())  # noqa: E731
    for _ in range(4):
        v = rng.standard_normal(x.shape)
        d = (loss(x + 1e-6 * v, w) - loss(x - 1e-6 * v, w)) / 2e-6
        assert abs(float((f64(dq) * v).sum()) - d) <= float((2 * 2.0 ** -11 * np.abs(f64(dq)) * np.abs(v)).sum()) + 1e-3
        v = rng.standard_normal(w.shape)
        d = (loss(x, w + 1e-6 * v) - loss(x, w - 1e-6 * v)) / 2e-6
        assert abs(float((f64(dwq) * v).sum()) - d) <= 1e-4 * np.abs(v).sum()


def test_far_positions_keep_their_angles():
    q, k, kw = make(16, 2, 1, 128, torch.bfloat16, 128, seed=3, start=1000000)
    qo, _ = binding.qk_norm_rope(q, k, **kw)
    check_forward(qo, q, kw["q_weight"], kw, False, 1e-6, torch.bfloat16)


def test_zero_rows_and_large_rows():
    """A row of zeros stays zero (eps keeps its norm finite) and has a finite
    gradient; rows of the largest magnitudes do not overflow in FP32."""
    q, k, kw = make(4, 2, 1, 64, torch.bfloat16, 64, seed=4, fused=False)
    q[1] = 0
    q[2] = 1e18
    qo, ko = binding.qk_norm_rope(q, k, **kw)
    check_forward(qo, q, kw["q_weight"], kw, False, 1e-6, torch.bfloat16)
    assert bool((qo[1] == 0).all())
    dq, dk, dwq, _ = binding.qk_norm_rope_backward(q, k, qo, ko, **kw)
    assert bool(torch.isfinite(dq).all()) and bool(torch.isfinite(dwq).all())


def test_nan_stays_in_its_row():
    q, k, kw = make(9, 4, 2, 64, torch.bfloat16, 64, seed=8, fused=False)
    ref, _ = binding.qk_norm_rope(q, k, **kw)
    q[3, 1, 5] = float("nan")
    out, _ = binding.qk_norm_rope(q, k, **kw)
    keep = torch.ones(9, 4, dtype=torch.bool, device="cuda")
    keep[3, 1] = False
    assert torch.equal(out[keep], ref[keep]) and bool(torch.isnan(out[3, 1]).all())


def test_positions_out_of_range_are_skipped_and_recorded():
    q, k, kw = make(5, 2, 1, 64, torch.bfloat16, 64, seed=1)
    kw["positions"] = torch.tensor([0, -1, 2, 5, 4], dtype=torch.int32, device="cuda")  # tables of 5 positions
    qo, ko = torch.full((5, 2, 64), 7.0, dtype=q.dtype, device="cuda"), torch.full((5, 1, 64), 7.0, dtype=q.dtype,
                                                                                  device="cuda")
    binding.qk_norm_rope(q, k, q_out=qo, k_out=ko, **kw)
    assert binding.etattn_read_device_status(clear=True) == binding.ETATTN_ERR_BAD_INDEX
    ok = [0, 2, 4]
    good = dict(kw, positions=kw["positions"][ok].contiguous())
    check_forward(qo[ok], q[ok], kw["q_weight"], good, False, 1e-6, q.dtype)
    assert bool((qo[[1, 3]] == 7).all()) and bool((ko[[1, 3]] == 7).all())
    dq, dk, dwq, dwk = binding.qk_norm_rope_backward(q, k, q, k, **kw)
    assert binding.etattn_read_device_status(clear=True) == binding.ETATTN_ERR_BAD_INDEX
    check_backward(dq[ok], dwq, q[ok], kw["q_weight"], q[ok], good, False, 1e-6, q.dtype)


def test_strided_outputs_and_untouched_neighbours():
    q, k, kw = make(12, 4, 2, 64, torch.bfloat16, 64, seed=2)
    buf = torch.full((12, 8, 64), 3.0, dtype=q.dtype, device="cuda")
    binding.qk_norm_rope(q, k, q_out=buf[:, 1:5], k_out=buf[:, 6:8], **kw)
    ref_q, ref_k = binding.qk_norm_rope(q, k, **kw)
    assert torch.equal(buf[:, 1:5], ref_q) and torch.equal(buf[:, 6:8], ref_k)
    assert bool((buf[:, 0] == 3).all()) and bool((buf[:, 5] == 3).all())
    # heads outermost: [H, T, D] storage
    ht = torch.empty((4, 12, 64), dtype=q.dtype, device="cuda").permute(1, 0, 2)
    binding.qk_norm_rope(q, k, q_out=ht, **kw)
    assert torch.equal(ht, ref_q)


def test_backward_without_tokens_gives_zero_weight_gradients():
    q, k, kw = make(0, 4, 2, 64, torch.bfloat16, 0)
    dq, dk, dwq, dwk = binding.qk_norm_rope_backward(q, k, torch.empty_like(q), torch.empty_like(k), **kw)
    assert bool((dwq == 0).all()) and bool((dwk == 0).all()) and dq.shape == (0, 4, 64)


def test_results_repeat_bit_for_bit_and_on_another_stream():
    q, k, kw = make(3001, 8, 2, 128, torch.bfloat16, 128, seed=11)
    a = binding.qk_norm_rope_backward(q, k, q, k, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = binding.qk_norm_rope_backward(q, k, q, k, **kw)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_a_given_stream_is_the_one_that_runs():
    q, k, kw = make(700, 8, 2, 128, torch.bfloat16, 128, seed=14)
    ref = binding.qk_norm_rope(q, k, **kw)
    ref_g = binding.qk_norm_rope_backward(q, k, q, k, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = binding.qk_norm_rope(q, k, stream=side, **kw)
        got_g = binding.qk_norm_rope_backward(q, k, q, k, stream=side, **kw)
    side.synchronize()
    for x, y in zip(ref + ref_g, got + got_g):
        assert torch.equal(x, y)


def test_captured_and_replayed_with_new_inputs():
    q, k, kw = make(40, 8, 2, 64, torch.bfloat16, 64, seed=12, fused=False)
    qo, ko = binding.qk_norm_rope(q, k, **kw)  # attributes set before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qo, ko = binding.qk_norm_rope(q, k, **kw)
        grads = binding.qk_norm_rope_backward(q, k, qo, ko, **kw)
    q2, k2, _ = make(40, 8, 2, 64, torch.bfloat16, 64, seed=13, fused=False)
    q.copy_(q2)
    k.copy_(k2)
    graph.replay()
    torch.cuda.synchronize()
    check_forward(qo, q, kw["q_weight"], kw, False, 1e-6, torch.bfloat16)
    check_backward(grads[0], grads[2], q, kw["q_weight"], qo, kw, False, 1e-6, torch.bfloat16)
