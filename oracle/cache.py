"""FP64 definitions of what surrounds attention: the norm and rotation of
queries and keys with their gradients, the append to a paged key-value cache
and attention over one.

Everything is written from the formulas, one row at a time where that is
plainest; numpy arrays in, float64 arrays out.
"""

import numpy as np

from .dense import attention_dense


def _pairs(rope_dim, interleaved):
    i = np.arange(rope_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rope_dim // 2)


def rotate(x, cos, sin, interleaved=False):
    """Rotates pairs of the first 2 * cos.shape[-1] elements of x [T, H, D] by
    the tokens' angles (cos, sin: [T, rope_dim / 2]); sin negated turns back."""
    y = np.array(x, dtype=np.float64)
    if cos is None:
        return y
    a, b = _pairs(2 * cos.shape[-1], interleaved)
    c, s = np.asarray(cos, np.float64)[:, None, :], np.asarray(sin, np.float64)[:, None, :]
    xa, xb = y[..., a].copy(), y[..., b].copy()
    y[..., a] = xa * c - xb * s
    y[..., b] = xb * c + xa * s
    return y


def norm_rope(x, weight, cos, sin, interleaved=False, eps=1e-6):
    """RMS norm of every head row of x [T, H, D] (weight None: no norm), then
    the rotation (cos None: none)."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return rotate(x, cos, sin, interleaved)


def norm_rope_backward(x, weight, dy, cos, sin, interleaved=False, eps=1e-6):
    """(dx, dweight) of sum(dy * norm_rope(x)); dweight None without a weight.

    y = R (n w) with n = x r: the rotation R is orthogonal, so the gradient of
    n w is g = R^-1 dy; dw = sum g n; and r's own gradient takes away the part
    of g w along x."""
    g = rotate(dy, cos, None if sin is None else -np.asarray(sin, np.float64), interleaved)
    if weight is None:
        return g, None
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    gw = g * w
    dx = r * gw - x * r ** 3 * np.mean(gw * x, axis=-1, keepdims=True)
    return dx, np.sum(g * x * r, axis=(0, 1))


def new_tokens(seqlens_k, cu_seqlens_q):
    """(sequence, token, position) of every new token that has a place."""
    out = []
    for s, L in enumerate(seqlens_k):
        first, end = int(cu_seqlens_q[s]), int(cu_seqlens_q[s + 1])
        for t in range(first, end):
            p = int(L) - (end - first) + (t - first)
            if p >= 0:
                out.append((s, t, p))
    return out


def paged_append(pages, rows, block_table, seqlens_k, cu_seqlens_q):
    """The pages [num_pages, H, page_size, D] after rows [T, H, D] are stored."""
    pages = np.array(pages, dtype=np.float64)
    page_size = pages.shape[2]
    for s, t, p in new_tokens(seqlens_k, cu_seqlens_q):
        pages[int(block_table[s][p // page_size]), :, p % page_size] = rows[t]
    return pages


def gather(pages, table_row, length):
    """The first ``length`` positions of one sequence: [H, length, D]."""
    page_size = pages.shape[2]
    out = np.zeros((pages.shape[1], length, pages.shape[3]))
    for j in range(length):
        out[:, j] = pages[int(table_row[j // page_size]), :, j % page_size]
    return out


def attention_paged(q, k_pages, v_pages, block_table, seqlens_k, cu_seqlens_q, causal=True, scale=1.0,
                    window_left=-1, window_right=-1):
    """(o [T, Hq, D], lse [Hq, T]): every sequence's rows against its gathered
    keys by the dense definition.  Tokens of no sequence stay NaN."""
    T, Hq, D = q.shape
    o, lse = np.full((T, Hq, D), np.nan), np.full((Hq, T), np.nan)
    for s, L in enumerate(seqlens_k):
        first, end = int(cu_seqlens_q[s]), int(cu_seqlens_q[s + 1])
        if end == first:
            continue
        k, v = (gather(pages, block_table[s], int(L)) for pages in (k_pages, v_pages))
        ro, rl = attention_dense(np.asarray(q[first:end], np.float64).transpose(1, 0, 2)[None], k[None], v[None],
                                 causal=causal, scale=scale, window_left=window_left, window_right=window_right)
        o[first:end] = ro[0].transpose(1, 0, 2)
        lse[:, first:end] = rl[0]
    return o, lse
