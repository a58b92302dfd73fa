"""Definitions of the paged cache held in 4 bits and of the pages' bookkeeping:
rounding to a 16-bit type, a group's codes with its scale and minimum, a block's
bytes, and pages handed out and taken back one by one.

numpy arrays in and out; values in float64, types by name ("f16", "bf16").
"""

import numpy as np

# Bits of the significand, and the exponent of the smallest step.
_TYPES = {"f16": (11, -24), "bf16": (8, -133)}
_MAX = {"f16": 65504.0, "bf16": float.fromhex("0x1.fep127")}


def step(x, dtype):
    """The distance of neighbouring numbers of the type at x."""
    bits, least = _TYPES[dtype]
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    return np.ldexp(1.0, np.where(x == 0, least, np.maximum(e - bits, least)))


def rounded(x, dtype):
    """x rounded once to the type, to nearest and ties to even."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        y = np.where(np.isfinite(x), np.round(x / step(x, dtype)) * step(x, dtype), x)
    return np.where(np.isfinite(x) & (np.abs(y) > _MAX[dtype]), np.copysign(np.inf, x), y)


def to_bits(x, dtype):
    """The 16-bit patterns of numbers of the type (NaN: 0x7fff)."""
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        b = (x.astype(np.float16).view(np.uint16) if dtype == "f16"
             else (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16))
    return np.where(np.isnan(x), np.uint16(0x7fff), b)


def from_bits(b, dtype):
    b = np.asarray(b, np.uint16)
    with np.errstate(invalid="ignore"):  # (signalling NaN)
        x = b.view(np.float16) if dtype == "f16" else (b.astype(np.uint32) << 16).view(np.float32)
        return x.astype(np.float64)


def quantise(x, dtype):
    """(codes [..., G], scale [...], minimum [...]) of groups x [..., G] of numbers
    of the type."""
    x = np.asarray(x, np.float64)
    low, high = x.min(-1), x.max(-1)
    with np.errstate(invalid="ignore", over="ignore"):
        span = high - low
        bad = ~np.isfinite(x).all(-1) | ~np.isfinite(np.where(np.isfinite(span), span, np.inf).astype(np.float32))
        span = np.where(bad, 0.0, span)
        low, high = np.where(bad, 0.0, low), np.where(bad, 0.0, high)
        # The spread's own rounding to 64 bits (Knuth's error-free sum): 15 s is exact.
        back = high - span
        above = (high - (span + back)) + (back - low) > 0
        covers = lambda s: (15 * s > span) | ((15 * s == span) & ~above)  # noqa: E731
        s = rounded(span / 15, dtype)
        s = np.where(covers(s), s, s + step(s, dtype))
        below = s - step(s * (1 - 2.0 ** -20), dtype)
        assert np.all((s == 0) | ~covers(below))  # the smallest that does
        s = np.where(low > _MAX[dtype] - 15 * s, below, s)  # (the difference is exact where it decides)
        c = np.where(s[..., None] > 0, np.round((np.where(bad[..., None], 0.0, x) - low[..., None]) /
                                                np.where(s > 0, s, 1.0)[..., None]), 0.0)
    return c.astype(np.uint8), np.where(bad, np.nan, s), np.where(bad, np.nan, low)


def group_of(D):
    return min(D, 64)


def values(codes, s, m):
    return codes * s[..., None] + m[..., None]


def stored(x, dtype):
    """What a cache stands for after rows x [..., D] are stored."""
    G = group_of(x.shape[-1])
    return values(*quantise(x.reshape(*x.shape[:-1], -1, G), dtype)).reshape(x.shape)


def pack(x, dtype):
    """Blocks [..., bytes] of rows x [..., page, D]."""
    *lead, page, D = x.shape
    G = group_of(D)
    out = []
    for h in range(D // G):
        c, s, m = quantise(x[..., h * G:(h + 1) * G], dtype)
        out.append((c[..., 0::2] | (c[..., 1::2] << 4)).reshape(*lead, -1))
        sm = np.ascontiguousarray(np.stack((to_bits(s, dtype), to_bits(m, dtype)), -1))
        out.append(sm.view(np.uint8).reshape(*lead, -1))
    return np.concatenate(out, -1)


def parts(blocks, page, D, dtype):
    """(codes [..., page, D], scales [..., page, D / G], minima) of blocks [..., bytes]."""
    G = group_of(D)
    lead = blocks.shape[:-1]
    part = page * (G // 2 + 4)
    codes, scales, minima = [], [], []
    for h in range(D // G):
        b = blocks[..., h * part:(h + 1) * part]
        two = b[..., :page * G // 2].reshape(*lead, page, G // 2)
        codes.append(np.stack((two & 15, two >> 4), -1).reshape(*lead, page, G))
        sm = np.ascontiguousarray(b[..., page * G // 2:]).view(np.uint16).reshape(*lead, page, 2)
        scales.append(from_bits(sm[..., 0], dtype))
        minima.append(from_bits(sm[..., 1], dtype))
    return np.concatenate(codes, -1), np.stack(scales, -1), np.stack(minima, -1)


def unpack(blocks, page, D, dtype):
    """The values [..., page, D] that blocks stand for."""
    c, s, m = parts(blocks, page, D, dtype)
    G = group_of(D)
    return c * np.repeat(s, G, -1) + np.repeat(m, G, -1)


def extend(new_tokens, seqlens, table, free, page, capacity_tokens):
    """(table, seqlens, cu_seqlens, positions, slots, free pages left) of a step that
    fits: pages taken from the end of the list ``free``, one by one."""
    table, free = np.array(table), list(free)
    lens, cu, positions, slots = [], [0], [], []
    for s, (L, n) in enumerate(zip(seqlens, new_tokens)):
        for col in range(-(-int(L) // page), -(-int(L + n) // page)):
            table[s, col] = free.pop()
        for p in range(int(L), int(L + n)):
            positions.append(p)
            slots.append(int(table[s, p // page]) * page + p % page)
        lens.append(int(L + n))
        cu.append(cu[-1] + int(n))
    behind = capacity_tokens - len(slots)
    return table, lens, cu, positions + [0] * behind, slots + [-1] * behind, free


def truncate(keep, seqlens, table, free, page):
    """(seqlens, free pages): those past the kept keys appended one by one."""
    free = list(free)
    for s, (L, k) in enumerate(zip(seqlens, keep)):
        for col in range(-(-int(k) // page), -(-int(L) // page)):
            free.append(int(table[s, col]))
    return [int(k) for k in keep], free
