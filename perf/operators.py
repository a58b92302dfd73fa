"""The cases on which the cache and query/key operators are measured.

``listed`` and ``draw`` name cases, ``prepare`` makes one's inputs on the GPU, ``run`` makes one pass
(with ``own`` false in elementary torch operations, with ``own`` true through the library), ``work``
counts what a pass cannot do without and ``exact`` computes it in 64 bits.

Operators ("op"):
  norm_rope      norm of every query and key head and their rotation, one pass
  norm_rope_bwd  its gradients: inputs and norm weights
  append         queries and keys normed and rotated; keys and values into a paged cache
  paged          attention of the new tokens over the paged cache
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def _norm(op, name, T, Hq, Hkv, D, dtype, rope, style, start):
    return {"name": name, "op": op, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype, "rope": rope,
            "style": style, "start": start}


def _cache(op, name, S, n, Hq, Hkv, D, dtype, page, layout, longest, lengths, **more):
    return {"name": name, "op": op, "S": S, "n": n, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page,
            "layout": layout, "longest": longest, "lengths": lengths, **more}


def listed():
    return [
        # The query/key step of one decode step of 8 sequences: a launch's latency.
        _norm("norm_rope", "norm_rope_t8", 8, 32, 8, 128, "bf16", 128, "half", 32760),
        # The same step over a prefill or training batch of 2 x 8192 tokens.
        _norm("norm_rope", "norm_rope_t16384", 16384, 32, 8, 128, "bf16", 128, "half", 0),
        # Gradients of a short FP16 fine-tuning batch: odd token count, part of the head rotated, pairs side by side.
        _norm("norm_rope_bwd", "norm_rope_bwd_t1021_d64", 1021, 16, 4, 64, "f16", 32, "interleaved", 0),
        # Gradients of the training batch.
        _norm("norm_rope_bwd", "norm_rope_bwd_t16384", 16384, 32, 8, 128, "bf16", 128, "half", 0),
        # One decode step of 8 sequences: latency.
        _cache("append", "append_s8_n1", 8, 1, 32, 8, 128, "bf16", 16, "nhd", 32768, "ragged"),
        # Prompts of 16 sequences written into the cache (an admission step).
        _cache("append", "append_s16_n1000", 16, 1000, 32, 8, 128, "bf16", 16, "nhd", 4096, "ragged"),
        # A single request's decode step over a short history: latency.
        _cache("paged", "paged_s1_k1000", 1, 1, 32, 8, 128, "bf16", 16, "nhd", 1000, "equal", window=-1),
        # A serving batch whose histories differ widely.
        _cache("paged", "paged_s64_ragged_k16384", 64, 1, 32, 8, 128, "bf16", 16, "nhd", 16384, "ragged", window=-1),
        # Drafted tokens checked together, FP16 heads of 64, local window.
        _cache("paged", "paged_s16_n4_d64_window", 16, 4, 16, 4, 64, "f16", 32, "hnd", 16384, "ragged", window=4095),
        # The decode step of the contiguous benchmark, on pages.
        _cache("paged", "paged_s8_k32768", 8, 1, 32, 8, 128, "bf16", 64, "hnd", 32768, "equal", window=-1),
        # One request with a very long history.
        _cache("paged", "paged_s1_k524288", 1, 1, 32, 8, 128, "bf16", 16, "nhd", 524288, "equal", window=-1),
        # Every query head with its own keys (no grouping).
        _cache("paged", "paged_s5_h16_k8191", 5, 1, 16, 16, 128, "bf16", 128, "hnd", 8191, "ragged", window=-1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "paged", "paged"])
    D = rng.choice([32, 64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("norm_rope", "norm_rope_bwd"):
        T = _log(rng, 1, 16384)
        return {"op": op, "T": T, "Hq": Hkv * group, "Hkv": Hkv, "D": D, "dtype": dtype,
                "rope": rng.choice([D, D // 2]), "style": rng.choice(["half", "interleaved"]),
                "start": rng.choice([0, _log(rng, 1, 100000)])}
    page = rng.choice([16, 32, 64, 128])
    layout = rng.choice(["nhd", "hnd"])
    if op == "append":
        S = _log(rng, 1, 64)
        n = rng.choice([1, _log(rng, 1, max(1, 16000 // S))])
        return {"op": op, "S": S, "n": n, "Hq": Hkv * group, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page,
                "layout": layout, "longest": n + _log(rng, 1, 8000), "lengths": "ragged"}
    S = _log(rng, 1, 64)
    n = rng.choice([1, 1, 1, rng.randint(2, 8)])
    longest = _log(rng, 1, 262144 // S)
    return {"op": op, "S": S, "n": n, "Hq": Hkv * group, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page,
            "layout": layout, "longest": max(n, longest), "lengths": rng.choice(["ragged", "equal"]),
            "window": rng.choice([-1, -1, _log(rng, 16, 8192)])}


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """Keys of every sequence, new tokens included: all the longest, or spread over the logarithm
    with the longest among them.  They go by the case alone, so that its work is known."""
    S, n, longest = case["S"], case["n"], max(case["longest"], case["n"])
    if case["lengths"] == "equal":
        return np.full(S, longest, dtype=np.int64)
    r = np.random.RandomState(S * 7919 + longest % 65521)
    lens = np.exp(r.uniform(math.log(n), math.log(longest + 1), S)).astype(np.int64)
    lens = np.clip(lens, n, longest)
    lens[r.randint(S)] = longest
    return lens


def _rotation_tables(positions, rope):
    """cos and sin of every position's angles, FP32, from angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64, device="cuda") / rope)
    ang = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    dt, D, Hq, Hkv, op = DTYPES[case["dtype"]], case["D"], case["Hq"], case["Hkv"], case["op"]

    def normal(*shape, scale=1.0, mean=0.0):
        x = torch.empty(shape, dtype=dt, device="cuda")
        return x.normal_(mean, scale, generator=g)

    T = case["T"] if "T" in case else case["S"] * case["n"]
    state = {"case": dict(case)}
    if op != "paged":
        # q, k and v as one projection leaves them: side by side in a row of each token.
        fused = normal(T, Hq + 2 * Hkv, D, scale=1.5)
        state["q"], state["k"], state["v"] = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
        state["wq"], state["wk"] = normal(D, scale=0.2, mean=1.0), normal(D, scale=0.2, mean=1.0)
    if op in ("norm_rope", "norm_rope_bwd"):
        state["cos"], state["sin"] = _rotation_tables(case["start"] + T, case["rope"])
        state["positions"] = torch.arange(case["start"], case["start"] + T, dtype=torch.int32, device="cuda")
        if op == "norm_rope_bwd":
            state["dq"], state["dk"] = normal(T, Hq, D), normal(T, Hkv, D)
        return state
    # The cache: every sequence's pages, in an order of their own, and some that nobody holds.
    lens, page, S = _lengths(case), case["page"], case["S"]
    width = int(-(-lens.max() // page))
    need = -(-lens // page)
    pool = int(need.sum()) + 7
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(width, device="cuda")[None, :] < torch.from_numpy(need).cuda()[:, None]
    table[held] = order[:int(need.sum())]
    state["table"] = table
    state["seqlens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    for name in ("k_pages", "v_pages"):  # logical [pages, Hkv, page, D]
        if case["layout"] == "hnd":
            state[name] = normal(pool, Hkv, page, D)
        else:
            state[name] = normal(pool, page, Hkv, D).permute(0, 2, 1, 3)
    if op == "append":
        state["cos"], state["sin"] = _rotation_tables(int(lens.max()), D)
    else:
        # Scores with a spread like that of trained heads, some of them peaked.
        state["q"] = normal(T, Hq, D, scale=2.0)
        state["max_seqlen_k"] = int(lens.max())
    return state


# ---------------------------------------------------------------- the plain forms, in 32 bits

def _halves(x, style):
    r = x.shape[-1] // 2
    return (x[..., :r], x[..., r:]) if style == "half" else (x[..., 0::2], x[..., 1::2])


def _joined(a, b, style):
    return torch.cat((a, b), -1) if style == "half" else torch.stack((a, b), -1).flatten(-2)


def _rotate(x, cos, sin, style, sign):
    """Rotates the first 2 * cos.shape[-1] elements of [T, H, D] by sign * angle."""
    rope = 2 * cos.shape[-1]
    c, s = cos[:, None], sign * sin[:, None]
    a, b = _halves(x[..., :rope], style)
    return torch.cat((_joined(a * c - b * s, b * c + a * s, style), x[..., rope:]), -1)


def _norm_rope(x, w, cos, sin, style):
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return _rotate(x * r * w.float(), cos, sin, style, 1.0)


def _norm_rope_bwd(x, w, dy, cos, sin, style):
    x, w = x.float(), w.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    g = _rotate(dy.float(), cos, sin, style, -1.0)
    dw = (g * x * r).sum((0, 1))
    gw = g * w
    return r * (gw - x * r.square() * (gw * x).mean(-1, keepdim=True)), dw


def _plain_append(s):
    case = s["case"]
    T, n, page = case["S"] * case["n"], case["n"], case["page"]
    t = torch.arange(T, device="cuda")
    seq = t // n
    pos = s["seqlens"].long()[seq] - n + t % n
    pages, slots = s["table"][seq, pos // page].long(), pos % page
    cos, sin = s["cos"][pos], s["sin"][pos]
    q = _norm_rope(s["q"], s["wq"], cos, sin, "half").to(s["q"].dtype)
    s["k_pages"][pages, :, slots] = _norm_rope(s["k"], s["wk"], cos, sin, "half").to(s["k"].dtype)
    s["v_pages"][pages, :, slots] = s["v"]
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_paged(s):
    case = s["case"]
    S, n, Hq, Hkv, D = case["S"], case["n"], case["Hq"], case["Hkv"], case["D"]
    table = s["table"].long().clamp(min=0)

    def gathered(pages):  # [S, Hkv, keys, D]
        x = pages[table].float()  # [S, width, Hkv, page, D]
        return x.transpose(1, 2).reshape(S, Hkv, -1, D)

    q = s["q"].float().view(S, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, D)
    scores = (q * D ** -0.5) @ gathered(s["k_pages"]).transpose(-1, -2)  # [S, Hkv, group * n, keys]
    scores = scores.view(S, Hkv, Hq // Hkv, n, -1)
    lens = s["seqlens"].long()
    at = (lens[:, None] - n + torch.arange(n, device="cuda"))[:, None, None, :, None]
    key = torch.arange(scores.shape[-1], device="cuda")
    out = key > at
    if case["window"] >= 0:
        out = out | (key < at - case["window"])
    scores = scores.masked_fill(out, -math.inf)
    m = scores.amax(-1, keepdim=True)
    e = (scores - m).exp()
    z = e.sum(-1, keepdim=True)
    v = gathered(s["v_pages"])
    o = (e / z).reshape(S, Hkv, -1, v.shape[2]) @ v
    o = o.view(S, Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(S * n, Hq, D)
    lse = (m + z.log()).reshape(S, Hq, n).permute(1, 0, 2).reshape(Hq, S * n)
    return {"o": o.to(s["q"].dtype), "lse": lse}


def _plain(s):
    op, style = s["case"]["op"], s["case"].get("style")
    if op == "append":
        return _plain_append(s)
    if op == "paged":
        return _plain_paged(s)
    pos = s["positions"].long()
    cos, sin = s["cos"][pos], s["sin"][pos]
    if op == "norm_rope":
        return {"q": _norm_rope(s["q"], s["wq"], cos, sin, style).to(s["q"].dtype),
                "k": _norm_rope(s["k"], s["wk"], cos, sin, style).to(s["k"].dtype)}
    dq, dwq = _norm_rope_bwd(s["q"], s["wq"], s["dq"], cos, sin, style)
    dk, dwk = _norm_rope_bwd(s["k"], s["wk"], s["dk"], cos, sin, style)
    return {"dq": dq.to(s["q"].dtype), "dk": dk.to(s["k"].dtype), "dwq": dwq, "dwk": dwk}


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from exact_tiled_attention_19_gb300 import binding
    case = s["case"]
    op = case["op"]
    if op == "paged":
        o, lse = binding.attention_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seqlens"],
                                         max_seqlen_k=s["max_seqlen_k"], window_left=case["window"])
        return {"o": o, "lse": lse}
    if op == "append":
        q = binding.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["seqlens"], q=s["q"],
                                 q_weight=s["wq"], k_weight=s["wk"], rope_cos=s["cos"], rope_sin=s["sin"], eps=EPS)
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    how = dict(q_weight=s["wq"], k_weight=s["wk"], rope_cos=s["cos"], rope_sin=s["sin"], positions=s["positions"],
               interleaved=case["style"] == "interleaved", eps=EPS)
    if op == "norm_rope":
        q, k = binding.qk_norm_rope(s["q"], s["k"], **how)
        return {"q": q, "k": k}
    dq, dk, dwq, dwk = binding.qk_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], **how)
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    Hq, Hkv, D, op = case["Hq"], case["Hkv"], case["D"], case["op"]
    if op in ("norm_rope", "norm_rope_bwd"):
        x = case["T"] * (Hq + Hkv) * D
        tables = case["T"] * (case["rope"] * 4 + 4)
        if op == "norm_rope":
            return {"bytes": 2 * 2 * x + tables + 4 * D, "flops": 10 * x}
        return {"bytes": 3 * 2 * x + tables + 12 * D, "flops": 18 * x}
    lens, S, n = _lengths(case), case["S"], case["n"]
    index = 4 * S + 4 * int((-(-lens // case["page"])).sum())
    if op == "append":
        T = S * n
        return {"bytes": 2 * 2 * T * (Hq + 2 * Hkv) * D + T * (D * 4 + 4) + 4 * S, "flops": 10 * T * (Hq + Hkv) * D}
    c = lens[:, None] - n + np.arange(n)[None, :]
    lo = np.maximum(c - case["window"], 0) if case["window"] >= 0 else np.zeros_like(c)
    pairs = int((c - lo + 1).sum())
    keys = int((lens - lo[:, 0]).sum())
    return {"bytes": 2 * 2 * keys * Hkv * D + 2 * 2 * S * n * Hq * D + 4 * S * n * Hq + index,
            "flops": 4 * D * pairs * Hq}


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_rows(x, w, cos, sin, style, dy=None):
    """One row set [T, H, D] in 64 bits: the rotation as a matrix product of complex numbers; with
    ``dy`` the gradients of x and w."""
    x, w = x.double(), w.double()
    rope = 2 * cos.shape[-1]
    turn = torch.complex(cos.double(), sin.double())[:, None]

    def turned(y, by):
        part = y[..., :rope]
        if style == "half":
            z = torch.complex(part[..., :rope // 2].contiguous(), part[..., rope // 2:].contiguous()) * by
            part = torch.cat((z.real, z.imag), -1)
        else:
            z = torch.view_as_complex(part.reshape(*part.shape[:-1], -1, 2).contiguous()) * by
            part = torch.view_as_real(z).flatten(-2)
        return torch.cat((part, y[..., rope:]), -1)

    inv = 1.0 / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / x.shape[-1] + EPS)
    unit = x * inv
    if dy is None:
        return turned(unit * w, turn)
    back = turned(dy.double(), turn.conj())
    dunit = back * w
    dot = torch.sum(dunit * unit, -1, keepdim=True) / x.shape[-1]
    return (dunit - unit * dot) * inv, torch.einsum("thd,thd->d", back, unit)


def exact(case, seed):
    s = prepare(case, seed)
    op, style = case["op"], case.get("style", "half")
    if op in ("norm_rope", "norm_rope_bwd"):
        at = s["positions"].long()
        cos, sin = s["cos"][at], s["sin"][at]
        if op == "norm_rope":
            return {"q": _exact_rows(s["q"], s["wq"], cos, sin, style),
                    "k": _exact_rows(s["k"], s["wk"], cos, sin, style)}
        dq, dwq = _exact_rows(s["q"], s["wq"], cos, sin, style, s["dq"])
        dk, dwk = _exact_rows(s["k"], s["wk"], cos, sin, style, s["dk"])
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    S, n, page, D, Hq, Hkv = case["S"], case["n"], case["page"], case["D"], case["Hq"], case["Hkv"]
    lens, table = s["seqlens"].tolist(), s["table"].long()
    if op == "append":
        at = torch.cat([torch.arange(L - n, L, device="cuda") for L in lens])
        cos, sin = s["cos"][at], s["sin"][at]
        k = _exact_rows(s["k"], s["wk"], cos, sin, style)
        k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
        for i, L in enumerate(lens):
            rows = slice(i * n, (i + 1) * n)
            p = torch.arange(L - n, L, device="cuda")
            k_pages[table[i, p // page], :, p % page] = k[rows]
            v_pages[table[i, p // page], :, p % page] = s["v"][rows].double()
        return {"q": _exact_rows(s["q"], s["wq"], cos, sin, style), "k_pages": k_pages, "v_pages": v_pages}
    o = torch.empty(S * n, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(Hq, S * n, dtype=torch.float64, device="cuda")
    for i, L in enumerate(lens):
        held = table[i, :-(-L // page)]
        for h in range(Hkv):
            K = s["k_pages"][held, h].double().reshape(-1, D)[:L]
            V = s["v_pages"][held, h].double().reshape(-1, D)[:L]
            for j in range(n):
                c = L - n + j
                lo = max(0, c - case["window"]) if case["window"] >= 0 else 0
                heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                z = s["q"][i * n + j, heads].double() @ K[lo:c + 1].T / math.sqrt(D)
                lse[heads, i * n + j] = torch.logsumexp(z, -1)
                o[i * n + j, heads] = torch.softmax(z, -1) @ V[lo:c + 1]
    return {"o": o, "lse": lse}
