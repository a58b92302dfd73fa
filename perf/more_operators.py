"""The cases on which the 4-bit paged cache and the calls that hand out its pages are measured.

``listed`` and ``draw`` name cases, ``prepare`` makes one's inputs on the GPU, ``run`` makes one pass
(with ``own`` false in elementary torch operations, with ``own`` true through the library), ``work``
counts what a pass cannot do without and ``exact`` computes it in 64 bits.

Operators ("op"):
  extend     pages, positions and slots for a step's new tokens, from the sequences' lengths
  truncate   pages past the kept lengths back on the free list
  append_q4  queries and keys normed and rotated; keys and values into the cache in 4 bits; the cache read back
  paged_q4   attention of the new tokens over the 4-bit cache

A cache's block of one page and head holds, for every group of min(D, 64) elements of its rows, the codes
[page, group / 2 bytes] (element e in half e % 2 of byte e / 2, the low half first) and then the scale and
the minimum [page, 2] in the type of the inputs.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def _tables(op, name, S, longest, page, step):
    return {"name": name, "op": op, "S": S, "longest": longest, "page": page, "step": step}


def _cache(op, name, S, n, Hq, Hkv, D, dtype, page, longest, lengths, **more):
    return {"name": name, "op": op, "S": S, "n": n, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page,
            "longest": longest, "lengths": lengths, **more}


def listed():
    return [
        # Pages for one decode step of 8 sequences: a launch's latency.
        _tables("extend", "extend_s8_decode", 8, 32768, 16, "decode"),
        # A step of a large batch that decodes most of its sequences and takes in some prompts, on odd lengths.
        _tables("extend", "extend_s1000_mixed", 1000, 8191, 16, "mixed"),
        # Drafted tokens of a batch rejected: the last few keys of each sequence go.
        _tables("truncate", "truncate_s64_drafts", 64, 16384, 16, "drafts"),
        # Requests that ended, among many that go on: whole sequences go.
        _tables("truncate", "truncate_s4000_ended", 4000, 4096, 32, "ended"),
        # One decode step of 8 sequences: latency.
        _cache("append_q4", "append_q4_s8_n1", 8, 1, 32, 8, 128, "bf16", 16, 128, "ragged"),
        # Prompts of 16 sequences written into the cache (an admission step).
        _cache("append_q4", "append_q4_s16_n1000", 16, 1000, 32, 8, 128, "bf16", 16, 1000, "equal"),
        # Odd FP16 prompts of heads of 64.
        _cache("append_q4", "append_q4_s3_n333_d64", 3, 333, 16, 4, 64, "f16", 32, 700, "ragged"),
        # A single request's decode step over a short history: latency.
        _cache("paged_q4", "paged_q4_s1_k1000", 1, 1, 32, 8, 128, "bf16", 16, 1000, "equal", window=-1),
        # A serving batch whose histories differ widely.
        _cache("paged_q4", "paged_q4_s64_ragged_k16384", 64, 1, 32, 8, 128, "bf16", 16, 16384, "ragged", window=-1),
        # Drafted tokens checked together, FP16 heads of 64, local window.
        _cache("paged_q4", "paged_q4_s16_n4_d64_window", 16, 4, 16, 4, 64, "f16", 32, 16384, "ragged", window=4095),
        # The decode step of the contiguous benchmark, on pages.
        _cache("paged_q4", "paged_q4_s8_k32768", 8, 1, 32, 8, 128, "bf16", 64, 32768, "equal", window=-1),
        # One request with a very long history.
        _cache("paged_q4", "paged_q4_s1_k524288", 1, 1, 32, 8, 128, "bf16", 16, 524288, "equal", window=-1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "truncate", "append_q4", "paged_q4", "paged_q4"])
    if op in ("extend", "truncate"):
        S = _log(rng, 1, 4000)
        return {"op": op, "S": S, "longest": _log(rng, 1, min(65536, (1 << 24) // S)),
                "page": rng.choice([8, 16, 32, 64, 256]),
                "step": rng.choice(["decode", "mixed"] if op == "extend" else ["drafts", "ended"])}
    D = rng.choice([32, 64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    dtype = rng.choice(["bf16", "f16"])
    page = rng.choice([8, 16, 32, 64, 128])
    S = _log(rng, 1, 64)
    if op == "append_q4":
        n = rng.choice([1, _log(rng, 1, max(1, 16000 // S))])
        return {"op": op, "S": S, "n": n, "Hq": Hkv * group, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page,
                "longest": n + rng.randint(0, 200), "lengths": "ragged"}
    n = rng.choice([1, 1, 1, rng.randint(2, 8)])
    longest = _log(rng, 1, 262144 // S)
    return {"op": op, "S": S, "n": n, "Hq": Hkv * group, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page,
            "longest": max(n, longest), "lengths": rng.choice(["ragged", "equal"]),
            "window": rng.choice([-1, -1, _log(rng, 16, 8192)])}


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """Keys of every sequence, new tokens included: all the longest, or spread over the logarithm
    with the longest among them.  They go by the case alone, so that its work is known."""
    S, n, longest = case["S"], case.get("n", 1), max(case["longest"], case.get("n", 1))
    if case.get("lengths") == "equal":
        return np.full(S, longest, dtype=np.int64)
    r = np.random.RandomState(S * 7919 + longest % 65521)
    lens = np.exp(r.uniform(math.log(n), math.log(longest + 1), S)).astype(np.int64)
    lens = np.clip(lens, n, longest)
    lens[r.randint(S)] = longest
    return lens


def _step(case):
    """(keys of every sequence before the step, new tokens or keys that stay), from the case alone."""
    S, lens = case["S"], _lengths(case)
    r = np.random.RandomState(S * 31 + case["longest"] % 8191)
    if case["step"] == "decode":
        return lens, np.ones(S, dtype=np.int64)
    if case["step"] == "mixed":  # four of five decode; the others wait, or bring a prompt into an unused slot
        kind = r.randint(10, size=S)
        lens = np.where(kind == 9, 0, lens)
        prompt = np.exp(r.uniform(0, math.log(2 * case["longest"] + 1), S)).astype(np.int64)
        return lens, np.where(kind == 9, np.minimum(prompt, case["longest"]), np.where(kind == 8, 0, 1))
    if case["step"] == "drafts":
        return lens, np.maximum(0, lens - r.randint(0, 8, size=S))
    return lens, np.where(r.randint(10, size=S) == 0, 0, lens)


def _rotation_tables(positions, rope):
    """cos and sin of every position's angles, FP32, from angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64, device="cuda") / rope)
    ang = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def _owned(lens, page, order, width):
    """A block table [S, width] whose sequences hold the pages of ``order`` one after the other."""
    need = -(-lens // page)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(width, device="cuda")[None, :] < torch.from_numpy(need).cuda()[:, None]
    table[held] = order[:int(need.sum())]
    return table


def _prepare_tables(case, g):
    lens, step = _step(case)
    page, S = case["page"], case["S"]
    after = lens + step if case["op"] == "extend" else lens
    width = int(-(-after.max() // page)) + 2
    used = int((-(-lens // page)).sum())
    pool = used + (int((-(-after // page) - -(-lens // page)).sum()) if case["op"] == "extend" else 0) + 200
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    free = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    free[:pool - used] = order[used:]
    device = lambda x: torch.from_numpy(x.astype(np.int32)).cuda()  # noqa: E731
    return {"case": dict(case), "table": _owned(lens, page, order, width), "lens": device(lens), "step": device(step),
            "free": free, "count": torch.tensor([pool - used], dtype=torch.int32, device="cuda"),
            "tokens": int(step.sum()) if case["op"] == "extend" else 0}


def _group(D):
    return min(D, 64)


def _fields(pages, D, page, dt):
    """The codes [pages, heads, groups, page, group / 2] and the scales and minima [..., page, 2] of a cache."""
    G = _group(D)
    x = pages.view(pages.shape[0], pages.shape[1], D // G, page * (G // 2 + 4))
    codes = x[..., :page * G // 2].unflatten(-1, (page, G // 2))
    return codes, x[..., page * G // 2:].unflatten(-1, (page, 4)).view(dt)


def _scale(span, dt):
    """The smallest value s of the 16-bit type with 15 s >= span, span >= 0."""
    s = (span / 15).to(dt)
    return torch.where(s.to(span.dtype) * 15 < span, (s.view(torch.int16) + 1).view(dt), s)


def _quantised(x):
    """Codes [..., group] and (scale, minimum) [..., 2] of rows x [..., group] of a 16-bit type."""
    y = x.float()
    low, high = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    s = _scale(high - low, x.dtype)
    c = torch.where(s > 0, ((y - low) / s.float()).round(), torch.zeros_like(y))
    return c.to(torch.uint8), torch.cat((s, low.to(x.dtype)), -1)


def _stored(pages, at, slot, x, D, page):
    """Rows x [T, heads, D] of a 16-bit type into the cache, row t at page at[t] and slot slot[t]."""
    codes, scales = _fields(pages, D, page, x.dtype)
    c, sm = _quantised(x.unflatten(-1, (-1, _group(D))))
    codes[at, :, :, slot] = c[..., 0::2] | (c[..., 1::2] << 4)
    scales[at, :, :, slot] = sm


def _values(pages, D, page, dt):
    """A cache's values [pages, heads, page, D] in 32 bits."""
    codes, scales = _fields(pages, D, page, dt)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    sm = scales.float()
    return (c * sm[..., :1] + sm[..., 1:]).transpose(2, 3).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    op = case["op"]
    if op in ("extend", "truncate"):
        return _prepare_tables(case, g)
    dt, D, Hq, Hkv, page, S, n = (DTYPES[case["dtype"]], *(case[k] for k in ("D", "Hq", "Hkv", "page", "S", "n")))
    T, lens = S * n, _lengths(case)

    def normal(*shape, scale=1.0, mean=0.0):
        x = torch.empty(shape, dtype=dt, device="cuda")
        return x.normal_(mean, scale, generator=g)

    # The cache: every sequence's pages, in an order of their own, and some that nobody holds.
    need = -(-lens // page)
    pool = int(need.sum()) + 7
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = _owned(lens, page, order, int(need.max()))
    G = _group(D)
    cache = torch.empty(pool, 2, Hkv, D // G * page * (G // 2 + 4), dtype=torch.uint8, device="cuda")
    state = {"case": dict(case), "table": table, "seqlens": torch.from_numpy(lens.astype(np.int32)).cuda(),
             "k_pages": cache[:, 0], "v_pages": cache[:, 1]}
    for name in ("k_pages", "v_pages"):
        for first in range(0, pool, 4096):
            part = state[name][first:first + 4096]
            x = normal(part.shape[0], Hkv, page, D)
            codes, scales = _fields(part, D, page, dt)
            c, sm = _quantised(x.unflatten(-1, (-1, G)).transpose(2, 3))
            codes.copy_(c[..., 0::2] | (c[..., 1::2] << 4))
            scales.copy_(sm)
    if op == "paged_q4":
        # Scores with a spread like that of trained heads, some of them peaked.
        state["q"] = normal(T, Hq, D, scale=2.0)
        state["max_seqlen_k"] = int(lens.max())
        return state
    # q, k and v as one projection leaves them: side by side in a row of each token.
    fused = normal(T, Hq + 2 * Hkv, D, scale=1.5)
    state["q"], state["k"], state["v"] = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    state["wq"], state["wk"] = normal(D, scale=0.2, mean=1.0), normal(D, scale=0.2, mean=1.0)
    state["cos"], state["sin"] = _rotation_tables(int(lens.max()), D)
    pos = (torch.from_numpy(lens - n).cuda()[:, None] + torch.arange(n, device="cuda")).flatten()
    seq = torch.arange(T, device="cuda") // n
    state["positions"] = pos.to(torch.int32)
    state["slots"] = table[seq, pos // page].long() * page + pos % page
    return state


# ---------------------------------------------------------------- the plain forms

def _plain_extend(s):
    page, lens, new = s["case"]["page"], s["lens"].long(), s["step"].long()
    before, after = (lens + page - 1) // page, (lens + new + page - 1) // page
    taken = (after - before).cumsum(0)
    base = taken - (after - before)
    count = s["count"].long()
    col = torch.arange(s["table"].shape[1], device="cuda")
    fresh = (col >= before[:, None]) & (col < after[:, None])
    which = (count - 1 - (base[:, None] + col - before[:, None])).clamp(0, s["free"].shape[0] - 1)
    s["table"].copy_(torch.where(fresh, s["free"][which], s["table"]))
    cu = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), new.cumsum(0)))
    t = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = lens[seq] + t - cu[seq]
    slots = s["table"][seq, pos // page].long() * page + pos % page
    return {"table": s["table"], "seqlens": (lens + new).int(), "cu_seqlens": cu.int(), "positions": pos.int(),
            "slots": slots, "count": (count - taken[-1]).int()}


def _plain_truncate(s):
    page, lens, keep = s["case"]["page"], s["lens"].long(), s["step"].long()
    have, stay = (lens + page - 1) // page, (keep + page - 1) // page
    given = (have - stay).cumsum(0)
    base = given - (have - stay)
    count = s["count"].long()
    col = torch.arange(s["table"].shape[1], device="cuda")
    back = (col >= stay[:, None]) & (col < have[:, None])
    place = count + base[:, None] + col - stay[:, None]
    # (What does not go back is written past the end, and cut off.)
    end = s["free"].shape[0]
    free = torch.cat((s["free"], s["free"][:1]))
    free = free.scatter(0, torch.where(back, place, end).flatten(), s["table"].flatten())
    s["free"].copy_(free[:end])
    return {"free": s["free"], "seqlens": keep.int(), "count": (count + given[-1]).int()}


def _norm_rope(x, w, cos, sin):
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = x * r * w
    half = y.shape[-1] // 2
    c, s, a, b = cos[:, None], sin[:, None], y[..., :half], y[..., half:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _rounded(x, dt):
    """64-bit values rounded once to the 16-bit type (a conversion by way of 32 bits rounds twice)."""
    bits, least = (8, -133) if dt == torch.bfloat16 else (11, -24)
    _, e = torch.frexp(x)
    unit = torch.ldexp(torch.ones_like(x), (e - bits).clamp(min=least))
    return ((x / unit).round() * unit).to(dt)


def _plain_append(s):
    case, dt = s["case"], s["k"].dtype
    page, D = case["page"], case["D"]
    at = s["positions"].long()
    cos, sin = s["cos"][at], s["sin"][at]
    q = _norm_rope(s["q"].float(), s["wq"].float(), cos, sin).to(dt)
    # Keys in 64 bits: a value next to a border of the roundings decides a code.
    k = _rounded(_norm_rope(s["k"].double(), s["wk"].double(), cos.double(), sin.double()), dt)
    where, slot = s["slots"] // page, s["slots"] % page
    _stored(s["k_pages"], where, slot, k, D, page)
    _stored(s["v_pages"], where, slot, s["v"], D, page)
    return {"q": q, "k": _values(s["k_pages"], D, page, dt).to(dt), "v": _values(s["v_pages"], D, page, dt).to(dt)}


def _plain_paged(s):
    case = s["case"]
    S, n, Hq, Hkv, D, page = (case[k] for k in ("S", "n", "Hq", "Hkv", "D", "page"))
    dt, table = s["q"].dtype, s["table"].long().clamp(min=0)

    def gathered(pages):  # [S, Hkv, keys, D]
        x = _values(pages[table.flatten()], D, page, dt).unflatten(0, table.shape)  # [S, width, Hkv, page, D]
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
    return {"o": o.to(dt), "lse": lse}


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from exact_tiled_attention_19_gb300 import binding
    case = s["case"]
    op = case["op"]
    if op == "extend":
        seqlens, cu, positions, slots, count = binding.paged_extend(
            s["step"], s["lens"], s["table"], s["free"], s["count"], page_size=case["page"], total_tokens=s["tokens"])
        return {"table": s["table"], "seqlens": seqlens, "cu_seqlens": cu, "positions": positions, "slots": slots,
                "count": count}
    if op == "truncate":
        seqlens, count = binding.paged_truncate(s["step"], s["lens"], s["table"], s["free"], s["count"],
                                                page_size=case["page"])
        return {"free": s["free"], "seqlens": seqlens, "count": count}
    if op == "append_q4":
        q = binding.paged_append_q4(s["k"], s["v"], s["k_pages"], s["v_pages"], s["slots"], q=s["q"],
                                    q_weight=s["wq"], k_weight=s["wk"], rope_cos=s["cos"], rope_sin=s["sin"],
                                    positions=s["positions"], eps=EPS)
        return {"q": q, "k": binding.paged_unpack_q4(s["k_pages"], case["D"], q.dtype),
                "v": binding.paged_unpack_q4(s["v_pages"], case["D"], q.dtype)}
    o, lse = binding.attention_paged_q4(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seqlens"],
                                        max_seqlen_k=s["max_seqlen_k"], window_left=case["window"])
    return {"o": o, "lse": lse}


PLAIN = {"extend": _plain_extend, "truncate": _plain_truncate, "append_q4": _plain_append, "paged_q4": _plain_paged}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    S, op, page = case["S"], case["op"], case["page"]
    if op in ("extend", "truncate"):
        lens, step = _step(case)
        if op == "extend":
            T, pages = int(step.sum()), int((-(-(lens + step) // page) - -(-lens // page)).sum())
            return {"bytes": 16 * S + 12 * T + 8 * pages, "flops": T + S}
        pages = int((-(-lens // page) - -(-step // page)).sum())
        return {"bytes": 12 * S + 8 * pages, "flops": S + pages}
    Hq, Hkv, D, n = case["Hq"], case["Hkv"], case["D"], case["n"]
    row = D // 2 + 4 * (D // _group(D))
    lens = _lengths(case)
    if op == "append_q4":
        T, read = S * n, (int((-(-lens // page)).sum()) + 7) * page * Hkv
        append = 2 * T * (2 * Hq + 2 * Hkv) * D + 2 * T * Hkv * row + T * (D * 4 + 12)
        return {"bytes": append + 2 * read * (row + 2 * D), "flops": 20 * T * (Hq + 2 * Hkv) * D + 4 * read * D}
    index = 4 * S + 4 * int((-(-lens // page)).sum())
    c = lens[:, None] - n + np.arange(n)[None, :]
    lo = np.maximum(c - case["window"], 0) if case["window"] >= 0 else np.zeros_like(c)
    pairs = int((c - lo + 1).sum())
    keys = int((lens - lo[:, 0]).sum())
    return {"bytes": 2 * keys * Hkv * row + 2 * 2 * S * n * Hq * D + 4 * S * n * Hq + index,
            "flops": 4 * D * pairs * Hq}


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_norm_rope(x, w, cos, sin):
    """One row set [T, H, D] in 64 bits: the rotation as a product of complex numbers."""
    x, w, half = x.double(), w.double(), x.shape[-1] // 2
    y = x * w / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / x.shape[-1] + EPS)
    turn = torch.complex(cos.double(), sin.double())[:, None]
    z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * turn
    return torch.cat((z.real, z.imag), -1)


def _exact_values(x):
    """What the cache holds for rows [..., group] of a 16-bit type, in 64 bits."""
    dt, x = x.dtype, x.double()
    low = x.min(-1, keepdim=True).values
    span = x.max(-1, keepdim=True).values - low
    s = (span / 15.0).to(dt).double()
    more = (s.to(dt).view(torch.int16) + 1).view(dt).double()
    s = torch.where(15.0 * s < span, more, s)
    return low + s * torch.where(s > 0, torch.round((x - low) / torch.where(s > 0, s, 1.0)), 0.0)


def _exact_cache(pages, D, page, dt):
    """A cache's values [pages, heads, page, D], byte by byte."""
    G = _group(D)
    out = torch.empty(pages.shape[0], pages.shape[1], page, D, dtype=torch.float64, device="cuda")
    block = page * (G // 2 + 4)
    for j in range(D // G):
        part = pages[..., j * block:(j + 1) * block]
        sm = part[..., page * G // 2:].contiguous().view(dt).double().view(*part.shape[:2], page, 2)
        c = part[..., :page * G // 2].reshape(*part.shape[:2], page, G // 2)
        for half in range(2):
            out[..., j * G + half:(j + 1) * G:2] = sm[..., 1:] + sm[..., :1] * ((c >> 4 * half) & 15).double()
    return out


def exact(case, seed):
    op = case["op"]
    if op in ("extend", "truncate"):  # whole numbers
        return None
    s = prepare(case, seed)
    S, n, page, D, Hq, Hkv = (case[k] for k in ("S", "n", "page", "D", "Hq", "Hkv"))
    dt, G = DTYPES[case["dtype"]], _group(D)
    if op == "append_q4":
        at = s["positions"].long()
        cos, sin = s["cos"][at], s["sin"][at]
        where, slot = s["slots"] // page, s["slots"] % page
        k = _rounded(_exact_norm_rope(s["k"], s["wk"], cos, sin), dt)
        out = {"q": _exact_norm_rope(s["q"], s["wq"], cos, sin)}
        for name, rows in (("k", k), ("v", s["v"])):
            out[name] = _exact_cache(s[name + "_pages"], D, page, dt)
            out[name][where, :, slot] = _exact_values(rows.reshape(S * n, Hkv, D // G, G)).reshape(S * n, Hkv, D)
        return out
    lens, table = s["seqlens"].tolist(), s["table"].long()
    o = torch.empty(S * n, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(Hq, S * n, dtype=torch.float64, device="cuda")
    for i, L in enumerate(lens):
        held = table[i, :-(-L // page)]
        for h in range(Hkv):
            K, V = (_exact_cache(s[x][held, h:h + 1], D, page, dt).reshape(-1, D)[:L] for x in ("k_pages", "v_pages"))
            for j in range(n):
                c = L - n + j
                lo = max(0, c - case["window"]) if case["window"] >= 0 else 0
                heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                z = s["q"][i * n + j, heads].double() @ K[lo:c + 1].T / math.sqrt(D)
                lse[heads, i * n + j] = torch.logsumexp(z, -1)
                o[i * n + j, heads] = torch.softmax(z, -1) @ V[lo:c + 1]
    return {"o": o, "lse": lse}
