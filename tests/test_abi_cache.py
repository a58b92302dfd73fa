"""CPU tests of the calls on query/key norm and rotation and on the paged
cache: invalid calls return the documented status before any CUDA call, empty
work is a no-op, and the helpers refuse mismatched tensors."""

import pytest
import torch

from exact_tiled_attention_19_gb300 import binding as B

# Fake, aligned, far-apart device addresses: validation never dereferences them.
P = [0x100000000 * (i + 1) for i in range(16)]


def packed(H, D):
    return [H * D, D, 1]


def rope_call(**kw):
    a = dict(q=P[0], k=P[1], wq=P[2], wk=P[3], cos=P[4], sin=P[5], pos=P[6], qo=P[7], ko=P[8], T=10, Hq=4, Hk=2, D=64,
             dtype=1, rope=64, inter=0, maxpos=100, eps=1e-6)
    a.update(kw)
    st = a.get("strides") or packed(a["Hq"], a["D"]) + packed(a["Hk"], a["D"]) + packed(a["Hq"], a["D"]) + packed(
        a["Hk"], a["D"])
    return B.attn_qk_norm_rope(a["q"], a["k"], a["wq"], a["wk"], a["cos"], a["sin"], a["pos"], a["qo"], a["ko"],
                               a["T"], a["Hq"], a["Hk"], a["D"], a["dtype"], st, a["rope"], a["inter"], a["maxpos"],
                               a["eps"], 0)


COMMON = [
    (dict(dtype=5), 2), (dict(T=-1), 3), (dict(T=2 ** 30 + 1), 3), (dict(D=96), 3), (dict(Hq=-1), 3),
    (dict(Hq=65536), 3), (dict(rope=24), 3), (dict(rope=80), 3), (dict(rope=-16), 3), (dict(maxpos=0), 3),
    (dict(cos=0), 1), (dict(sin=0), 1), (dict(cos=P[4] + 4), 6), (dict(wq=P[2] + 2), 6), (dict(eps=0.0), 8),
    (dict(eps=float("nan")), 8), (dict(eps=float("inf")), 8), (dict(q=0), 1), (dict(k=0), 1), (dict(q=P[0] + 8), 6),
    (dict(k=P[1] + 8), 6),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(qo=0), 1), (dict(ko=0), 1), (dict(pos=0), 1), (dict(pos=P[6] + 2), 6), (dict(ko=P[8] + 4), 6),
    (dict(qo=P[0]), 7), (dict(ko=P[0] + 64), 7), (dict(ko=P[7]), 7),
    (dict(strides=[256, 64, 2, 128, 64, 1, 256, 64, 1, 128, 64, 1]), 5),
    (dict(strides=[256, 64, 1, 0, 64, 1, 256, 64, 1, 128, 64, 1]), 5),
    (dict(strides=[256, 64, 1, 128, 60, 1, 256, 64, 1, 128, 64, 1]), 5),
])
def test_rope_refusals(kw, code):
    assert rope_call(**kw) == code


def test_rope_empty_work_and_no_device():
    assert rope_call(T=0, q=0, k=0, qo=0, ko=0) == 0
    assert rope_call(Hq=0, Hk=0) == 0
    if not torch.cuda.is_available():
        assert rope_call() == 12
        assert rope_call(Hq=0, q=0, qo=0) == 12                # keys alone
        assert rope_call(rope=0, cos=0, sin=0, pos=0) == 12    # norm alone
        assert rope_call(wq=0, wk=0, eps=0.0) == 12            # rotation alone


def test_views_of_one_fused_buffer_are_told_apart():
    """q_out and k_out (4 and 2 heads of 64) in rows of 8 heads."""
    def call(q_at, k_at, q_stride=512, k_stride=512):
        st = packed(4, 64) + packed(2, 64) + [q_stride, 64, 1] + [k_stride, 64, 1]
        return rope_call(qo=P[7] + 128 * q_at, ko=P[7] + 128 * k_at, strides=st)

    if not torch.cuda.is_available():
        assert call(0, 4) == call(0, 6) == call(2, 0) == call(8, 4) == 12
    assert call(0, 3) == 7 and call(0, 7) == 7 and call(4, 7) == 7 and call(1, 8) == 7
    assert call(0, 4, k_stride=640) == 7  # other periods meet sooner or later


def bwd_call(**kw):
    a = dict(q=P[0], k=P[1], gq=P[2], gk=P[3], wq=P[4], wk=P[5], cos=P[6], sin=P[7], pos=P[8], dq=P[9], dk=P[10],
             dwq=P[11], dwk=P[12], T=10, Hq=4, Hk=2, D=64, dtype=1, rope=64, inter=0, maxpos=100, eps=1e-6, ws=P[13],
             wsb=1 << 24)
    a.update(kw)
    st = a.get("strides") or (packed(a["Hq"], a["D"]) + packed(a["Hk"], a["D"])) * 3
    return B.attn_qk_norm_rope_bwd(a["q"], a["k"], a["gq"], a["gk"], a["wq"], a["wk"], a["cos"], a["sin"], a["pos"],
                                   a["dq"], a["dk"], a["dwq"], a["dwk"], a["T"], a["Hq"], a["Hk"], a["D"], a["dtype"],
                                   st, a["rope"], a["inter"], a["maxpos"], a["eps"], a["ws"], a["wsb"], 0)


@pytest.mark.parametrize("kw,code", [c for c in COMMON if "cos" not in c[0] and "wq" not in c[0]] + [
    (dict(dq=0), 1), (dict(dk=0), 1), (dict(gq=0), 1), (dict(gk=0), 1), (dict(dwq=0), 1), (dict(dwk=0), 1),
    (dict(pos=0), 1), (dict(ws=0), 1), (dict(ws=P[13] + 16), 6), (dict(wsb=64), 3), (dict(dwq=P[11] + 2), 6),
    (dict(cos=P[6] + 4), 6), (dict(dq=P[0]), 7), (dict(dq=P[3]), 7), (dict(dk=P[9]), 7), (dict(dwq=P[1]), 7),
    (dict(dwk=P[11]), 7), (dict(ws=P[2]), 7), (dict(ws=P[9]), 7), (dict(ws=P[12]), 7),
    # a broadcast upstream gradient (stride 0) is refused
    (dict(strides=packed(4, 64) + packed(2, 64) + [0, 64, 1] + packed(2, 64) + packed(4, 64) + packed(2, 64)), 5),
])
def test_rope_backward_refusals(kw, code):
    assert bwd_call(**kw) == code


def test_rope_backward_workspace_and_empty_work():
    size = B.attn_qk_norm_rope_bwd_workspace_size
    assert size(0, 4, 2, 64) == 0 and size(10, 4, 2, 96) == 0 and size(-1, 4, 2, 64) == 0
    assert 0 < size(1, 1, 0, 32) <= size(100000, 32, 8, 128) <= 608 * 2 * 128 * 4
    assert bwd_call(wsb=size(10, 4, 2, 64) - 1) == 3
    assert bwd_call(T=0, wq=0, wk=0) == 0
    if not torch.cuda.is_available():
        assert bwd_call(wsb=size(10, 4, 2, 64)) == 12
        assert bwd_call(wq=0, wk=0, dwq=0, dwk=0, ws=0, wsb=0) == 12


def append_call(**kw):
    a = dict(q=P[0], k=P[1], v=P[2], wq=P[3], wk=P[4], cos=P[5], sin=P[6], qo=P[7], kp=P[8], vp=P[9], bt=P[10],
             lens=P[11], cu=0, S=5, T=10, Hq=4, Hkv=2, D=64, dtype=1, page=16, pages=30, width=6, ts=6, rope=64, inter=0,
             maxpos=100, eps=1e-6)
    a.update(kw)
    D, ps = a["D"], max(1, a["page"])
    st = a.get("strides") or (packed(a["Hq"], D) + packed(a["Hkv"], D) * 2 + packed(a["Hq"], D) +
                              [a["Hkv"] * ps * D, ps * D, D, 1] * 2)
    return B.attn_paged_append(a["q"], a["k"], a["v"], a["wq"], a["wk"], a["cos"], a["sin"], a["qo"], a["kp"], a["vp"],
                               a["bt"], a["lens"], a["cu"], a["S"], a["T"], a["Hq"], a["Hkv"], D, a["dtype"], st,
                               a["page"], a["pages"], a["width"], a["ts"], a["rope"], a["inter"], a["maxpos"], a["eps"],
                               0)


@pytest.mark.parametrize("kw,code", COMMON[:5] + COMMON[6:] + [
    (dict(Hkv=0), 4), (dict(S=-1), 3), (dict(S=65536), 3), (dict(page=12), 3), (dict(page=4), 3), (dict(page=8192), 3),
    (dict(pages=0), 3), (dict(width=0), 3), (dict(ts=5), 3), (dict(S=3), 3),  # 10 tokens do not split among 3
    (dict(v=0), 1), (dict(kp=0), 1), (dict(vp=0), 1), (dict(bt=0), 1), (dict(lens=0), 1), (dict(qo=0), 1),
    (dict(kp=P[8] + 8), 6), (dict(bt=P[10] + 1), 6), (dict(lens=P[11] + 2), 6), (dict(cu=P[12] + 2), 6),
    (dict(kp=P[1]), 7), (dict(vp=P[0]), 7), (dict(vp=P[8]), 7), (dict(qo=P[9]), 7), (dict(qo=P[2]), 7),
])
def test_append_refusals(kw, code):
    assert append_call(**kw) == code


def test_append_empty_work_and_layouts():
    assert append_call(T=0) == 0
    assert append_call(S=0, T=0) == 0
    if not torch.cuda.is_available():
        assert append_call() == 12
        assert append_call(S=3, cu=P[12]) == 12            # ragged
        assert append_call(Hq=0, q=0, qo=0) == 12          # keys and values alone
        # keys and values interleaved: [pages, 2, slot, head, d]
        page = [2 * 16 * 2 * 64, 64, 2 * 64, 1]
        st = packed(4, 64) + packed(2, 64) * 2 + packed(4, 64) + page * 2
        assert append_call(strides=st, vp=P[8] + 16 * 2 * 64 * 2) == 12


def paged_call(**kw):
    a = dict(q=P[0], kp=P[1], vp=P[2], o=P[3], lse=P[4], bt=P[5], lens=P[6], cu=0, S=5, mq=2, T=10, Hq=4, Hkv=2, D=64,
             dtype=1, page=16, pages=30, width=6, ts=6, causal=1, wl=-1, wr=-1, scale=0.125, shares=8, ws=P[7],
             wsb=1 << 24)
    a.update(kw)
    D, ps = a["D"], max(1, a["page"])
    st = a.get("strides") or (packed(a["Hq"], D) + [a["Hkv"] * ps * D, ps * D, D, 1] * 2 + packed(a["Hq"], D))
    return B.attn_fwd_paged(a["q"], a["kp"], a["vp"], a["o"], a["lse"], a["bt"], a["lens"], a["cu"], a["S"], a["mq"],
                            a["T"], a["Hq"], a["Hkv"], D, a["dtype"], st, a["page"], a["pages"], a["width"], a["ts"],
                            a["causal"], a["wl"], a["wr"], a["scale"], a["shares"], a["ws"], a["wsb"], 0)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 2), (dict(D=256), 3), (dict(T=-1), 3), (dict(mq=-1), 3), (dict(S=65536), 3), (dict(page=100), 3),
    (dict(page=4), 3), (dict(pages=-1), 3), (dict(pages=0), 3), (dict(width=0), 3), (dict(ts=1), 3), (dict(T=11), 3),
    (dict(shares=0), 3), (dict(shares=65536), 3), (dict(Hkv=3), 4), (dict(Hkv=0), 4), (dict(scale=0.0), 8),
    (dict(scale=float("nan")), 8), (dict(q=0), 1), (dict(kp=0), 1), (dict(vp=0), 1), (dict(o=0), 1), (dict(bt=0), 1),
    (dict(lens=0), 1), (dict(ws=0), 1), (dict(ws=P[7] + 128), 6), (dict(wsb=100), 3), (dict(q=P[0] + 2), 6),
    (dict(kp=P[1] + 8), 6), (dict(lse=P[4] + 2), 6), (dict(lens=P[6] + 1), 6), (dict(cu=P[8] + 2), 6),
    (dict(o=P[0]), 7), (dict(o=P[1] + 32), 7), (dict(lse=P[3]), 7), (dict(lse=P[2]), 7), (dict(ws=P[1]), 7),
    (dict(ws=P[3]), 7), (dict(ws=P[4]), 7), (dict(mq=2 ** 30, cu=P[8]), 3),
])
def test_paged_refusals(kw, code):
    assert paged_call(**kw) == code


def test_paged_empty_work_and_sizes():
    assert paged_call(S=0, T=0) == 0
    assert paged_call(T=0, mq=0) == 0
    size = B.attn_fwd_paged_workspace_size
    assert size(4, 2, 1, 64, 1) == 0 and size(4, 3, 1, 64, 2) == 0 and size(4, 2, 1, 100, 2) == 0
    assert size(4, 2, 0, 64, 2) == 0 and size(4, 2, 1, 64, 0) == 0
    assert size(32, 8, 1, 128, 304) >= 304 * 2 * 16 * 129 * 4
    assert size(32, 8, 8, 128, 304) >= 304 * 2 * 32 * 129 * 4
    assert paged_call(wsb=size(4, 2, 2, 64, 8) - 1) == 3
    if not torch.cuda.is_available():
        assert paged_call(wsb=size(4, 2, 2, 64, 8)) == 12
        assert paged_call(shares=1, ws=0, wsb=0) == 12
        assert paged_call(T=7, cu=P[8]) == 12
        assert B.attn_fwd_paged_plan(1, 4, 2, 1, 100, 64)[0] == 12
    assert B.attn_fwd_paged_plan(1, 4, 3, 1, 100, 64)[0] == 4
    assert B.attn_fwd_paged_plan(1, 4, 2, 1, -1, 64)[0] == 3


def test_status_string_of_the_bad_index():
    assert B.etattn_status_string(13) != "unknown status" and B.ETATTN_ERR_BAD_INDEX == 13


def test_helpers_refuse_mismatched_tensors():
    q, k = torch.zeros(6, 4, 64, dtype=torch.bfloat16), torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    cos, sin = B.rope_tables(32, 64, device="cpu")
    pos = torch.arange(6, dtype=torch.int32)
    with pytest.raises(TypeError):
        B.qk_norm_rope(q.float(), k)
    with pytest.raises(TypeError):
        B.qk_norm_rope(q, k.half())
    with pytest.raises(ValueError):
        B.qk_norm_rope(q, k[:5])
    with pytest.raises(ValueError):
        B.qk_norm_rope(q, k, q_weight=torch.ones(32, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        B.qk_norm_rope(q, k, rope_cos=cos, rope_sin=sin)  # no positions
    with pytest.raises(ValueError):
        B.qk_norm_rope(q, k, rope_cos=cos, positions=pos)  # half of the tables
    with pytest.raises(TypeError):
        B.qk_norm_rope(q, k, rope_cos=cos, rope_sin=sin, positions=pos.long())
    with pytest.raises(ValueError):
        B.qk_norm_rope(q, k, rope_cos=cos, rope_sin=sin, positions=pos[:5])
    with pytest.raises(TypeError):
        B.qk_norm_rope(q, k, rope_cos=cos.double(), rope_sin=sin.double(), positions=pos)
    with pytest.raises(ValueError):
        B.qk_norm_rope_backward(q, k, q[:5], k)
    pages = torch.zeros(9, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(6, 2, dtype=torch.int32), torch.zeros(6, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.paged_append(k, k, pages, pages[:8], table, lens)
    with pytest.raises(ValueError):
        B.paged_append(k, k, pages[:, :1], pages[:, :1], table, lens)
    with pytest.raises(TypeError):
        B.paged_append(k, k, pages, pages, table.long(), lens)
    with pytest.raises(ValueError):
        B.attention_paged(q, pages, pages, table, lens[:5])
    with pytest.raises(ValueError):
        B.attention_paged(q, pages, pages, table, lens, cu_seqlens_q=torch.zeros(7, dtype=torch.int32))
    with pytest.raises(ValueError):
        B.attention_paged(q[..., :32], pages, pages, table, lens)


def test_helpers_refuse_tensors_outside_the_gpu():
    q, k = torch.zeros(6, 4, 64, dtype=torch.bfloat16), torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(9, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(6, 2, dtype=torch.int32), torch.ones(6, dtype=torch.int32)
    for call in (lambda: B.qk_norm_rope(q, k), lambda: B.qk_norm_rope_backward(q, k, q, k),
                 lambda: B.paged_append(k, k, pages, pages.clone(), table, lens),
                 lambda: B.attention_paged(q, pages, pages, table, lens)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_rope_tables_are_exact_far_out():
    cos, sin = B.rope_tables(200000, 32, device="cpu")
    import math
    p, i = 199999, 3
    a = p * 10000.0 ** (-2 * i / 32)
    assert abs(float(cos[p, i]) - math.cos(a)) < 1e-7 and abs(float(sin[p, i]) - math.sin(a)) < 1e-7
