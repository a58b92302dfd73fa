"""CPU tests of the calls on the 4-bit paged cache and on its pages: invalid calls
return the documented status before any CUDA call, empty work is a no-op, and the
helpers refuse mismatched tensors."""

import pytest
import torch

from exact_tiled_attention_19_gb300 import binding as B

P = [0x100000000 * (i + 1) for i in range(16)]  # far apart and aligned; never dereferenced
NO_GPU = not torch.cuda.is_available()


def packed(H, D):
    return [H * D, D, 1]


def test_block_bytes():
    size = B.attn_paged_q4_block_bytes
    assert size(16, 128) == 16 * 72 and size(8, 64) == 8 * 36 and size(4096, 32) == 4096 * 20
    assert size(12, 128) == size(4, 128) == size(8192, 64) == size(16, 96) == size(0, 64) == 0
    for page in (8, 16, 4096):
        for D in (32, 64, 128):
            assert size(page, D) % 16 == 0


def append_call(**kw):
    a = dict(q=P[0], k=P[1], v=P[2], wq=P[3], wk=P[4], cos=P[5], sin=P[6], pos=P[7], slots=P[8], qo=P[9], kp=P[10],
             vp=P[11], T=10, Hq=4, Hkv=2, D=64, dtype=1, page=16, pages=30, rope=64, inter=0, maxpos=100, eps=1e-6)
    a.update(kw)
    D, block = a["D"], a["page"] * 36
    st = a.get("strides") or (packed(a["Hq"], D) + packed(a["Hkv"], D) * 2 + packed(a["Hq"], D) +
                              [a["Hkv"] * block, block] * 2)
    return B.attn_paged_append_q4(a["q"], a["k"], a["v"], a["wq"], a["wk"], a["cos"], a["sin"], a["pos"], a["slots"],
                                  a["qo"], a["kp"], a["vp"], a["T"], a["Hq"], a["Hkv"], D, a["dtype"], st, a["page"],
                                  a["pages"], a["rope"], a["inter"], a["maxpos"], a["eps"], 0)


BLOCK = 16 * 36
OUT = packed(4, 64) + packed(2, 64) * 2 + packed(4, 64)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), 2), (dict(T=-1), 3), (dict(T=2 ** 30 + 1), 3), (dict(D=96), 3), (dict(Hq=-1), 3),
    (dict(Hkv=65536), 3), (dict(Hkv=0), 4), (dict(rope=24), 3), (dict(rope=80), 3), (dict(page=12), 3),
    (dict(page=4), 3), (dict(pages=0), 3), (dict(pages=-1), 3), (dict(maxpos=0), 3), (dict(cos=0), 1),
    (dict(pos=0), 1), (dict(slots=0), 1), (dict(v=0), 1), (dict(kp=0), 1), (dict(qo=0), 1), (dict(eps=0.0), 8),
    (dict(eps=float("nan")), 8), (dict(k=P[1] + 8), 6), (dict(kp=P[10] + 8), 6), (dict(slots=P[8] + 4), 6),
    (dict(pos=P[7] + 2), 6), (dict(sin=P[6] + 4), 6),
    (dict(kp=P[1]), 7), (dict(vp=P[0] + 64), 7), (dict(vp=P[10]), 7), (dict(qo=P[10]), 7), (dict(qo=P[2]), 7),
    (dict(kp=P[8]), 7), (dict(vp=P[7]), 7), (dict(qo=P[5]), 7), (dict(kp=P[4]), 7),
    # keys and values meet where the strides differ
    (dict(vp=P[10] + 2 * BLOCK, strides=OUT + [2 * BLOCK, BLOCK] + [4 * BLOCK, BLOCK]), 7),
    # strides: not a multiple of 16 bytes, 0, or blocks that run into one another
    (dict(strides=OUT + [2 * BLOCK + 8, BLOCK] * 2), 5), (dict(strides=OUT + [0, BLOCK] * 2), 5),
    (dict(strides=OUT + [2 * BLOCK, BLOCK - 16] * 2), 5), (dict(strides=OUT + [BLOCK + 16, BLOCK] * 2), 5),
])
def test_append_refusals(kw, code):
    assert append_call(**kw) == code


def test_append_empty_work_and_layouts():
    assert append_call(T=0, k=0, v=0, q=0) == 0
    if NO_GPU:
        assert append_call() == 12
        assert append_call(Hq=0, q=0, qo=0) == 12                      # keys and values alone
        assert append_call(rope=0, cos=0, sin=0, pos=0) == 12          # no rotation
        assert append_call(wq=0, wk=0, eps=0.0) == 12                  # no norm
        # keys and values of a page beside each other; heads outside, pages inside
        assert append_call(vp=P[10] + 2 * BLOCK, strides=OUT + [4 * BLOCK, BLOCK] * 2) == 12
        assert append_call(strides=OUT + [BLOCK, 30 * BLOCK] * 2) == 12


def unpack_call(**kw):
    a = dict(pages=P[0], out=P[1], Hkv=2, D=64, dtype=0, page=16, num=30)
    a.update(kw)
    st = a.get("strides") or [2 * BLOCK, BLOCK, 2 * 16 * 64, 16 * 64, 64, 1]
    return B.attn_paged_unpack_q4(a["pages"], a["out"], a["Hkv"], a["D"], a["dtype"], st, a["page"], a["num"], 0)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 2), (dict(D=48), 3), (dict(page=24), 3), (dict(num=-1), 3), (dict(Hkv=0), 4), (dict(pages=0), 1),
    (dict(out=0), 1), (dict(out=P[1] + 8), 6), (dict(pages=P[0] + 4), 6), (dict(out=P[0]), 7),
    (dict(strides=[2 * BLOCK, BLOCK, 2048, 1024, 60, 1]), 5), (dict(strides=[2 * BLOCK, BLOCK, 2048, 1024, 64, 2]), 5),
    (dict(strides=[BLOCK, BLOCK, 2048, 1024, 64, 1]), 5),
])
def test_unpack_refusals(kw, code):
    assert unpack_call(**kw) == code


def test_unpack_empty_work():
    assert unpack_call(num=0, pages=0, out=0) == 0
    if NO_GPU:
        assert unpack_call() == 12


def paged_call(**kw):
    a = dict(q=P[0], kp=P[1], vp=P[2], o=P[3], lse=P[4], bt=P[5], lens=P[6], cu=0, S=5, n=2, T=10, Hq=4, Hkv=2, D=64,
             dtype=1, page=16, pages=30, width=6, ts=6, causal=1, wl=-1, wr=-1, scale=0.125, shares=7, ws=P[7],
             wsb=1 << 24)
    a.update(kw)
    st = a.get("strides") or packed(a["Hq"], a["D"]) + [2 * BLOCK, BLOCK] * 2 + packed(a["Hq"], a["D"])
    return B.attn_fwd_paged_q4(a["q"], a["kp"], a["vp"], a["o"], a["lse"], a["bt"], a["lens"], a["cu"], a["S"], a["n"],
                               a["T"], a["Hq"], a["Hkv"], a["D"], a["dtype"], st, a["page"], a["pages"], a["width"],
                               a["ts"], a["causal"], a["wl"], a["wr"], a["scale"], a["shares"], a["ws"], a["wsb"], 0)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), 2), (dict(D=80), 3), (dict(T=9), 3), (dict(n=-1), 3), (dict(Hq=5), 4), (dict(Hkv=0), 4),
    (dict(scale=0.0), 8), (dict(scale=float("inf")), 8), (dict(shares=0), 3), (dict(shares=65536), 3),
    (dict(page=10), 3), (dict(pages=0), 3), (dict(width=0), 3), (dict(ts=5), 3), (dict(S=65536), 3),
    (dict(q=0), 1), (dict(kp=0), 1), (dict(vp=0), 1), (dict(o=0), 1), (dict(bt=0), 1), (dict(lens=0), 1),
    (dict(ws=0), 1), (dict(ws=P[7] + 16), 6), (dict(wsb=64), 3), (dict(q=P[0] + 8), 6), (dict(kp=P[1] + 8), 6),
    (dict(lse=P[4] + 2), 6), (dict(bt=P[5] + 2), 6), (dict(o=P[0]), 7), (dict(o=P[1] + 64), 7), (dict(lse=P[2]), 7),
    (dict(lse=P[3]), 7), (dict(ws=P[1]), 7), (dict(ws=P[3]), 7), (dict(ws=P[4]), 7), (dict(o=P[5]), 7),
    (dict(ws=P[6]), 7),
    (dict(strides=packed(4, 64) + [2 * BLOCK, BLOCK, 2 * BLOCK, BLOCK - 16] + packed(4, 64)), 5),
    (dict(strides=[256, 64, 2] + [2 * BLOCK, BLOCK] * 2 + packed(4, 64)), 5),
])
def test_paged_refusals(kw, code):
    assert paged_call(**kw) == code


def test_paged_workspace_plan_and_empty_work():
    size = B.attn_fwd_paged_q4_workspace_size
    assert size(4, 2, 1, 64, 1) == 0 and size(4, 3, 1, 64, 8) == 0 and size(4, 2, 0, 64, 8) == 0
    assert 0 < size(32, 8, 1, 128, 456) < size(32, 8, 4, 128, 456) == size(32, 8, 8, 128, 456)
    assert paged_call(wsb=size(4, 2, 2, 64, 7) - 1) == 3
    assert paged_call(T=0, n=0) == 0 and paged_call(S=0, T=0, n=0) == 0
    assert B.attn_fwd_paged_q4_plan(1, 4, 3, 1, 100, 64)[0] == 4
    assert B.attn_fwd_paged_q4_plan(1, 4, 2, 1, -1, 64)[0] == 3
    assert B.attn_fwd_paged_q4_plan(1, 4, 2, 1, 100, 64, 9) == (0, 9, size(4, 2, 1, 64, 9))
    if NO_GPU:
        assert paged_call(wsb=size(4, 2, 2, 64, 7)) == 12
        assert paged_call(shares=1, ws=0, wsb=0, lse=0) == 12
        assert B.attn_fwd_paged_q4_plan(1, 4, 2, 1, 100, 64)[0] == 12


def extend_call(**kw):
    a = dict(n=P[0], L=P[1], bt=P[2], free=P[3], count=P[4], Lo=P[5], co=P[6], cu=P[7], pos=P[8], slots=P[9], S=5, T=10,
             page=16, width=6, ts=6, cap=30, ws=P[10], wsb=1 << 20)
    a.update(kw)
    return B.attn_paged_extend(a["n"], a["L"], a["bt"], a["free"], a["count"], a["Lo"], a["co"], a["cu"], a["pos"],
                               a["slots"], a["S"], a["T"], a["page"], a["width"], a["ts"], a["cap"], a["ws"], a["wsb"],
                               0)


def truncate_call(**kw):
    a = dict(n=P[0], L=P[1], bt=P[2], free=P[3], count=P[4], Lo=P[5], co=P[6], S=5, page=16, width=6, ts=6, cap=30,
             ws=P[10], wsb=1 << 20)
    a.update(kw)
    return B.attn_paged_truncate(a["n"], a["L"], a["bt"], a["free"], a["count"], a["Lo"], a["co"], a["S"], a["page"],
                                 a["width"], a["ts"], a["cap"], a["ws"], a["wsb"], 0)


COMMON = [
    (dict(S=-1), 3), (dict(S=65536), 3), (dict(page=4), 3), (dict(page=24), 3), (dict(width=-1), 3), (dict(ts=5), 3),
    (dict(cap=-1), 3), (dict(cap=2 ** 30 + 1), 3), (dict(n=0), 1), (dict(L=0), 1), (dict(bt=0), 1), (dict(free=0), 1),
    (dict(count=0), 1), (dict(Lo=0), 1), (dict(co=0), 1), (dict(S=4097, ws=0), 1), (dict(S=4097, ws=P[10] + 64), 6), (dict(S=4097, wsb=16388), 3),
    (dict(L=P[1] + 2), 6), (dict(free=P[3] + 1), 6), (dict(Lo=P[0]), 7), (dict(Lo=P[1] + 4), 7), (dict(co=P[1]), 7),
    (dict(bt=P[3] + 8), 7), (dict(free=P[0]), 7), (dict(S=4097, ws=P[2]), 7), (dict(co=P[5] + 8), 7), (dict(Lo=P[4]), 7),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(T=-1), 3), (dict(cu=0), 1), (dict(pos=0), 1), (dict(slots=0), 1), (dict(slots=P[9] + 4), 6),
    (dict(cu=P[5] + 16), 7), (dict(pos=P[9] + 8), 7), (dict(slots=P[2]), 7), (dict(S=0), 3),
])
def test_extend_refusals(kw, code):
    assert extend_call(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON)
def test_truncate_refusals(kw, code):
    assert truncate_call(**kw) == code


def test_tables_empty_work_and_in_place():
    size = B.attn_paged_tables_workspace_size
    assert size(0) == size(5) == size(4096) == size(65536) == 0 and size(4097) == 4 * 4098
    assert extend_call(S=0, T=0) == 0 and truncate_call(S=0) == 0
    if NO_GPU:
        for call in (extend_call, truncate_call):
            assert call() == call(ws=0, wsb=0) == call(S=4097, wsb=16392) == 12
            assert call(Lo=P[1], co=P[4]) == 12            # in place
            assert call(width=0, ts=0, bt=0) == 12         # no pages to hold
            assert call(cap=0, free=0) == 12
        assert extend_call(T=0, pos=0, slots=0) == 12


def test_status_string_of_missing_pages():
    assert B.etattn_status_string(14) != "unknown status" and B.ETATTN_ERR_NO_PAGES == 14


def cpu_cache(num=9, H=2, page=16, D=64):
    k = torch.zeros(num, H, page * {32: 20, 64: 36, 128: 72}[D], dtype=torch.uint8)
    return k, k.clone()


def test_helpers_refuse_mismatched_tensors():
    kp, vp = cpu_cache()
    k, q = torch.zeros(6, 2, 64, dtype=torch.bfloat16), torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    slots, pos = torch.zeros(6, dtype=torch.int64), torch.zeros(6, dtype=torch.int32)
    cos, sin = B.rope_tables(8, 64, device="cpu")
    table, lens = torch.zeros(6, 2, dtype=torch.int32), torch.zeros(6, dtype=torch.int32)
    for error, call in [
        (TypeError, lambda: B.paged_append_q4(k.float(), k, kp, vp, slots)),
        (TypeError, lambda: B.paged_append_q4(k, k.half(), kp, vp, slots)),
        (TypeError, lambda: B.paged_append_q4(k, k, kp.char(), vp, slots)),
        (TypeError, lambda: B.paged_append_q4(k, k, kp, vp, slots.int())),
        (ValueError, lambda: B.paged_append_q4(k, k, kp, vp, slots[:5])),
        (ValueError, lambda: B.paged_append_q4(k, k, kp, vp[:8], slots)),
        (ValueError, lambda: B.paged_append_q4(k, k, kp[:, :1], vp[:, :1], slots)),
        (ValueError, lambda: B.paged_append_q4(k, k, kp[..., :100], vp[..., :100], slots)),
        (ValueError, lambda: B.paged_append_q4(k, k, kp[..., ::2], vp[..., ::2], slots)),
        (ValueError, lambda: B.paged_append_q4(k, k, kp, vp, slots, rope_cos=cos, rope_sin=sin)),
        (ValueError, lambda: B.paged_append_q4(k, k, kp, vp, slots, q=q[:5])),
        (ValueError, lambda: B.paged_unpack_q4(kp, 48, torch.bfloat16)),
        (TypeError, lambda: B.paged_unpack_q4(kp.int(), 64, torch.bfloat16)),
        (ValueError, lambda: B.paged_unpack_q4(kp, 64, torch.bfloat16, out=k)),
        (ValueError, lambda: B.attention_paged_q4(q, kp, vp, table, lens[:5])),
        (TypeError, lambda: B.attention_paged_q4(q, kp, vp, table.long(), lens)),
        (ValueError, lambda: B.attention_paged_q4(q[..., :40], kp, vp, table, lens)),
        (ValueError, lambda: B.attention_paged_q4(q, kp, vp[:5], table, lens)),
        (ValueError, lambda: B.attention_paged_q4(q, kp, vp, table, lens, cu_seqlens_q=torch.zeros(7, dtype=torch.int32))),
        (ValueError, lambda: B.paged_extend(lens[:5], lens, table, pos, pos[:1], page_size=16, total_tokens=6)),
        (TypeError, lambda: B.paged_extend(lens.long(), lens, table, pos, pos[:1], page_size=16, total_tokens=6)),
        (ValueError, lambda: B.paged_extend(lens, lens, table, pos, pos[:2], page_size=16, total_tokens=6)),
        (ValueError, lambda: B.paged_extend(lens, lens, table.t().contiguous().t(), pos, pos[:1], page_size=16,
                                            total_tokens=6)),
        (TypeError, lambda: B.paged_extend(lens, lens, table, pos, pos[:1], page_size=16, total_tokens=6, slots=pos)),
        (ValueError, lambda: B.paged_truncate(lens, lens[:5], table, pos, pos[:1], page_size=16)),
        (TypeError, lambda: B.paged_truncate(lens, lens, table, pos.long(), pos[:1], page_size=16)),
    ]:
        with pytest.raises(error):
            call()


def test_helpers_refuse_tensors_outside_the_gpu():
    kp, vp = cpu_cache()
    k, i32 = torch.zeros(6, 2, 64, dtype=torch.bfloat16), torch.zeros(6, dtype=torch.int32)
    table = torch.zeros(6, 2, dtype=torch.int32)
    for call in (lambda: B.paged_append_q4(k, k, kp, vp, torch.zeros(6, dtype=torch.int64)),
                 lambda: B.paged_unpack_q4(kp, 64, torch.float16),
                 lambda: B.attention_paged_q4(k, kp, vp, table, i32),
                 lambda: B.paged_extend(i32, i32, table, i32, i32[:1], page_size=16, total_tokens=6),
                 lambda: B.paged_truncate(i32, i32, table, i32, i32[:1], page_size=16)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError):
        B.q4_pages(4, 2, 12, 64, device="cpu")
    k_pages, v_pages = B.q4_pages(4, 2, 16, 64, device="cpu")
    assert k_pages.shape == v_pages.shape == (4, 2, 16 * 36) and k_pages.stride(0) == 4 * 16 * 36
